// Grouped differential attention decode over an 8-bit KV cache with a scale
// for each block of tokens and head (one new query token per sequence; format
// in gda_fp8_block.cuh), contiguous or paged, over all positions of a sequence
// or over the blocks that a list names; split over the cache length, plus a
// pass that joins the parts.  Short sequences take one launch: a cluster of
// thread blocks to each and unit of heads, joined through shared memory.
//
// The batch's positions, sequence after sequence, each rounded up to whole
// tiles of 16 (of a list: count * block), are cut into equal contiguous
// ranges.  A warp, which is a block of threads of its own, takes one range for
// one noise head and up to RH signal heads that share it: it copies a tile at a
// time into a ring in shared memory (TMA) and keeps the online softmax of
// all its maps and the accumulators O1, O2 in registers.  A tile lies in one
// block of tokens, so its rows follow one another in the cache and every head
// has one scale.  Each part of a range that lies in one sequence leaves (m, l)
// of both maps and (O1, O2) in workspace slot (range + sequence), which is
// unique because along the position axis neither index falls and one grows
// from part to part.
//
// The tensor cores multiply (mma.sync m16n8k16, f16 in, float32 out; a decode
// has one query row for a head, so the 128-row tcgen05 forms would sit idle for
// 127), because on the CUDA cores an element costs a widening and one (K) or
// two (V) multiply-adds, more than they can do at the copy rate.  e4m3 codes
// are exact in f16, and so is the query after a power of two.
//   - scores: A = codes of 16 positions x 16 dims, B = the query in every
//     column; the block's scale is a factor of the score.
//   - values: A = codes of 16 dims x 16 positions, B = four columns of weights,
//     the upper and the lower part of both maps', the other four zero, so that
//     two tiles of dims share one set of accumulators.  A weight is two f16
//     numbers, and the block's scale of V is in it, relative to a reference R of
//     its map, so that it keeps 22 bits down to 2^-18 R and 2^-40 R below that.
//     R is the largest such scale so far, but at most 2^12 times the largest
//     product of a scale and a weight, so that a scale far above the others'
//     whose keys have no weight does not take their digits; another R shrinks
//     the accumulators, as a larger score does.
// Step g of the loop copies K of tile g + A and V of the tile before that one,
// adds the values of tile g - 1 and scores tile g, so that no more than a tile
// is held while it is used.
//
// Measured (both kernels; of the 6793 GB/s of a copy): 64 sequences of 4096 to
// 8192, 12 + 4 heads of 64/128, 1007 MB: 157 us (95 %); one of 131072, 24 + 8
// heads, 671 MB: 109 us (91 %); 16 of up to 8191, 16 + 4 heads of 128/256, 437
// MB: 74 us (88 %); 16 listed blocks of 64 of each of the 64 sequences, 168 MB,
// one launch: 33.6 us (74 %; in two launches 38).  About 10 us of two launches are
// fixed: the chain of lengths, list, table and first tile (3), the joining (3),
// and the launches.  Copies alone take 95 % of the time.  By cp.async, a lane's
// 16 bytes each, the first two took 166 and 115 us: their issue was what the
// warps waited for.
#include <cuda_bf16.h>
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gda.h"
#include "gda_decode_join.cuh"
#include "gda_device.cuh"
#include "gda_fp8_block.cuh"
#include "gda_internal.h"

namespace cg = cooperative_groups;

namespace gda {
namespace {

constexpr int kTile = 16;              // positions of a tile
constexpr float kWeightBits = 15.f;    // weights carry a factor 2^15: the largest is within f16, the smallest far from its end
constexpr int kOneWarps = 8;           // at most, of a sequence in one launch
constexpr float kLowest = -3.0e38f;    // a maximum over no position
constexpr float kBand = 4096.f;        // a map's reference is at most that many times its largest product of scale and weight

// Signal heads of a warp: a noise head's group in equal parts of at most three
// (two at dv = 256).  Every part reads and scores the noise head for itself, and
// where the parts do not divide the group the last one does a head again, so a
// part costs about its heads and one more; the fewest of those are taken, of as
// many the smaller parts.  us of a call, 4 noise heads of 64/128, sequences of
// 4096 to 8192: groups of three as 3 166, as 2 + 2 234; of four as 2 + 2 209,
// as ones 307; of five as 3 + 3 195, as 2 + 2 + 2 232.  16 sequences of up to
// 8191, of 128/256: groups of four as 2 + 2 77, as ones 79.
struct Heads {
    int parts, each;   // parts of a group; signal heads of a part
};
Heads heads_of(int hs, int hn, int dv) {
    const int r = hs / hn, most = dv == 256 ? 2 : 3;
    Heads h{r, 1};
    for (int each = 2; each <= most && each <= r; ++each) {
        const int parts = (r + each - 1) / each;
        if (parts * (each + 1) < h.parts * (h.each + 1)) h = {parts, each};
    }
    return h;
}

// Shared memory of a warp, in bytes: tiles (codes of rh + 1 rows of K and rh of
// V for 16 positions), the first at a multiple of 1024, then queries, weights,
// and for each stage the tile's scales and a barrier.
constexpr int kMaxStages = 4;
__host__ __device__ constexpr int tile_bytes(int rh, int d, int dv) { return kTile * ((rh + 1) * d + rh * dv); }
__host__ __device__ constexpr int other_bytes(int rh, int d) { return (rh + 1) * d * 2 + rh * 128 + kMaxStages * 40; }
__host__ __device__ constexpr int stages_with(int warps, int rh, int d, int dv) {
    const int fit = (227 * 1024 / warps - 2048 - other_bytes(rh, d)) / tile_bytes(rh, d, dv);
    return fit > kMaxStages ? kMaxStages : fit;
}
// Warps that share an SM: the more signal heads a warp has, the more bytes it has in flight and the fewer warps it takes;
// as many on each of the four schedulers, and two stages for each.  us of a call, 8 / 12 / 16 warps: one signal head, 64
// sequences of 4096 to 8192, 4 + 4 heads of 64/128 86 / 76 / 72, 8 + 8 of 64/64 146 / 119 / 109; 32 of 8 + 8 of 128/128 104
// / 98 (as many as fit); two, 8 + 4 of 64/128 120 / 123, 16 + 4 209 / 218, but 28 + 4, four parts to a group, 205 / 177; 16
// + 4 of 64/64 175 / 159 / 160.  Three of 64/128, 12 + 4: 160 with eight, 167 with six of three stages, 173 with nine.
// Two of 128/256, 16 + 4: 76 with seven, 83 with four of three stages.
__host__ __device__ constexpr int warps_per_sm(int rh, int d, int dv) {
    int warps = rh == 1 ? 16 : (rh == 2 && dv == 64 ? 12 : 8);
    while (warps > 1 && stages_with(warps, rh, d, dv) < 2) warps -= warps > 8 ? 4 : 1;
    return warps;
}
__host__ __device__ constexpr int stages_of(int rh, int d, int dv) { return stages_with(warps_per_sm(rh, d, dv), rh, d, dv); }

struct Plan {
    Heads heads;
    int splits;        // ranges at most
    size_t ml_at, seg_at, bytes;
};

Plan plan_of(int B, int hs, int hn, int d, int dv) {
    Plan p;
    p.heads = heads_of(hs, hn, dv);
    p.splits = std::max(1, kSms * warps_per_sm(p.heads.each, d, dv) / (hn * p.heads.parts));
    const size_t slots = static_cast<size_t>(p.splits) + B;
    p.ml_at = (slots * hs * 2 * dv * sizeof(float) + 255) / 256 * 256;
    p.seg_at = p.ml_at + (slots * hs * 4 * sizeof(float) + 255) / 256 * 256;
    p.bytes = p.seg_at + static_cast<size_t>(B) * 2 * sizeof(int);
    return p;
}

struct Params {
    const __nv_bfloat16 *q1, *q2;
    const uint8_t *k1c, *k2c, *vc;
    const float *k1s, *k2s, *vs;
    const int *lens;
    const float *lambda;
    __nv_bfloat16 *out;
    float *ws_o;       // [slots][hs][2][dv]
    float *ws_ml;      // [slots][hs][4]: m1, l1, m2, l2
    int *ws_seg;       // [B][2]: first and last range of a sequence
    unsigned *err;
    float lambda_init, eps, scale_log2;
    int B, Lcap, hs, hn;
    int splits, parts;                       // ranges; parts of a noise head's group
    const int *block_table;
    int page_size, max_pages, num_pages;
    int shift;                               // log2 of a block's tiles
    uint32_t page_factor;                    // tile / (tiles of a page) = tile * page_factor >> page_shift, below 2^31
    int page_shift;
    const int *list, *count;                 // [B][hn][keep], [B], or nullptr: all blocks
    int keep;
};

// A sequence: its length, and its tiles along the axis that is cut into ranges.
struct Span {
    int len, tiles;
};

// A length outside [0, Lcap] and a count outside [0, keep] are clamped and reported.
template <bool LISTED>
__device__ __forceinline__ Span span_of(const Params &p, int b) {
    const int len = p.lens[b], count = LISTED ? p.count[b] : 0;
    const int l = min(max(len, 0), p.Lcap), c = LISTED ? min(max(count, 0), p.keep) : 0;
    if (l != len || c != count) atomicOr(p.err, GDA_DEVERR_BAD_LENGTH);
    return {l, LISTED ? (l == 0 ? 0 : c << p.shift) : (l + kTile - 1) / kTile};
}

__device__ __forceinline__ int positions_of(const Params &p, int b) {    // for the joining kernel: 0 if there are none
    return (p.list != nullptr ? span_of<true>(p, b) : span_of<false>(p, b)).tiles;
}

// The tiles [start, end) of a split on the axis of all sequences, and where it begins.  (There are fewer than 2^31.)
struct Range {
    int start, end, per, before;         // before: tiles of the sequences ahead of b
    int b;
    Span span;                           // of b
};

// Computed by a whole warp; false if the split has nothing to do.
template <bool LISTED>
__device__ __forceinline__ bool range_of(const Params &p, int split, Range &r) {
    const int lane = threadIdx.x & 31;
    int total = 0;
#pragma unroll 4
    for (int b = lane; b < p.B; b += 32) total += span_of<LISTED>(p, b).tiles;
    total = __reduce_add_sync(0xffffffffu, total);
    r.per = max(1, (total + p.splits - 1) / p.splits);
    if (static_cast<long long>(split) * r.per >= total) return false;
    r.start = split * r.per;
    r.end = min(total, r.start + r.per);
    int carry = 0;
    for (int base = 0; base < p.B; base += 32) {
        const int b = base + lane;
        const Span span = b < p.B ? span_of<LISTED>(p, b) : Span{0, 0};
        int incl = span.tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const int before = carry + incl - span.tiles;
        const unsigned hit = __ballot_sync(0xffffffffu, before <= r.start && r.start < before + span.tiles);
        if (hit) {
            const int src = __ffs(hit) - 1;
            r.b = base + src;
            r.before = __shfl_sync(0xffffffffu, before, src);
            r.span = {__shfl_sync(0xffffffffu, span.len, src), __shfl_sync(0xffffffffu, span.tiles, src)};
            return true;
        }
        carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;                         // not reached: start < total
}

// Notes the first and last range of every sequence that begins in range r of split `split`, for the joining kernel.
template <bool LISTED>
__device__ __forceinline__ void note_sequences(const Params &p, const Range &r, int split) {
    int before = r.before;
    for (int b = r.b; before < r.end; ++b) {
        const int tiles = span_of<LISTED>(p, b).tiles;
        if (tiles > 0 && before >= r.start && (threadIdx.x & 31) == 0) {
            p.ws_seg[2 * b] = split;
            p.ws_seg[2 * b + 1] = (before + tiles - 1) / r.per;
        }
        before += tiles;
    }
}

// Four bytes into shared memory, asynchronous; zeros in their place if `ok` is false.
__device__ __forceinline__ void copy_async4(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}

// A box of the tensor `map` into shared memory; its bytes count on the barrier `bar`.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap &map, uint32_t bar, int row, int head) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(&map)), "r"(0), "r"(row),
                 "r"(head), "r"(bar) : "memory");
}

// a * b + c: 16 x 16 (f16) times 16 x 8 (f16).
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A place in a warp's range: sequence b, tiles [tile, hi) of it, and the tiles of the range after those.
struct Cursor {
    int b, tile, hi, left;
};

__device__ __forceinline__ void enter(Cursor &c, int tile, int tiles) {
    const int n = min(tiles - tile, c.left);
    c.tile = tile;
    c.hi = tile + n;
    c.left -= n;
}

// To the next sequence with tiles; there is one while left > 0.  Returns its length.
template <bool LISTED>
__device__ __forceinline__ int next_sequence(const Params &p, Cursor &c) {
    Span span;
    do span = span_of<LISTED>(p, ++c.b);
    while (span.tiles == 0);
    enter(c, 0, span.tiles);
    return span.len;
}

// A tile in the cache: its page, its place there in tiles, and how many of its 16 positions exist.
struct Place {
    int page, tile, n;
};

// Tile `tile` (along the axis of ranges) of sequence b, whose length is len.
template <bool LISTED>
__device__ __forceinline__ Place place_of(const Params &p, int b, int g, int tile, int len) {
    // no branch on what is loaded: the loads are waited for when the tile's copies are started, a step later
    bool exists = true;
    if constexpr (LISTED) {
        const int id = p.list[(static_cast<size_t>(b) * p.hn + g) * p.keep + (tile >> p.shift)];
        exists = static_cast<unsigned>(id) <= static_cast<unsigned>(len / kTile >> p.shift);   // negative ones are not
        tile = exists ? (id << p.shift) + (tile & ((1 << p.shift) - 1)) : 0;
        exists = exists && tile * kTile < len;
        tile = exists ? tile : 0;
    }
    const int pg = static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(tile)) * p.page_factor >> p.page_shift);
    const int phys = p.block_table != nullptr ? p.block_table[static_cast<size_t>(b) * p.max_pages + pg] : b;
    return {phys, tile - pg * (p.page_size / kTile), exists ? min(kTile, len - tile * kTile) : 0};
}

// Cache row that a tile begins at.  A page outside the pool is read as page 0 and reported.  (Rows are below 2^31.)
__device__ __forceinline__ int row_of(const Params &p, const Place &at) {
    int phys = at.page;
    if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_pages)) {
        if (at.n > 0) atomicOr(p.err, GDA_DEVERR_BAD_PAGE);
        phys = 0;
    }
    return phys * p.page_size + at.tile * kTile;
}

// Places in a warp's shared memory, in bytes; a stage holds K of one tile and V of the tile before it.
template <int D, int DV, int RH>
struct Stage {
    static constexpr int NH = RH + 1;                    // heads with scores; the noise head is the last
    static constexpr int k = 0, v = NH * kTile * D, bytes = tile_bytes(RH, D, DV);
    static constexpr int k_bytes = v, v_bytes = bytes - v;
    static_assert(bytes % 1024 == 0 && v % 1024 == 0, "boxes change places by the bits of their addresses");
    static constexpr int count = stages_of(RH, D, DV);
    static_assert(count >= 2 && NH <= 4, "a tile is copied while another is used; four scales of K, three of V");
    static constexpr int queries = count * bytes, weights = queries + NH * D * 2, scales = weights + RH * 128;
    static constexpr int bars = scales + kMaxStages * 32, total = bars + kMaxStages * 8 + 1024;
    static constexpr int pitch = (bars + kMaxStages * 8 + 1023) / 1024 * 1024;   // of the warps of one block of threads
    static_assert(RH * (2 * DV * 4 + 16) <= count * bytes, "what a warp leaves has room in its ring");
    static constexpr int warps = warps_per_sm(RH, D, DV);
};

// The tensors of the caches, rows of heads: boxes of a head row (128 bytes of it at most) x 16 cache rows x heads.
struct Maps {
    CUtensorMap k1, k2, v;
};

template <typename V>
__device__ __forceinline__ V at(const uint8_t *smem) { return *reinterpret_cast<const V *>(smem); }

// The query rows of a warp's heads.
template <int D, int RH>
struct Queries {
    uint32_t words[RH + 1][D / 64];

    __device__ __forceinline__ void fetch(const Params &p, int b, int h0, int g) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j <= RH; ++j) {
            const __nv_bfloat16 *q = j == RH ? p.q2 + (static_cast<size_t>(b) * p.hn + g) * D
                                             : p.q1 + (static_cast<size_t>(b) * p.hs + h0 + j) * D;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) words[j][i] = reinterpret_cast<const uint32_t *>(q)[lane + 32 * i];
        }
    }

    // As f16 to shared memory, scaled by a power of two that brings a row's largest element to [2^14, 2^15) (f16 then
    // holds all of bf16's digits down to 2^-31 of that).  Returns this lane's factor from a product of codes to exp2
    // units: that of head lane % 4.
    __device__ __forceinline__ float place(const Params &p, uint8_t *dst) const {
        const int lane = threadIdx.x & 31;
        float mine = 0.f;
#pragma unroll
        for (int j = 0; j <= RH; ++j) {
            const uint32_t(&w)[D / 64] = words[j];
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) most = max(most, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
            most = __reduce_max_sync(0xffffffffu, most);
            const int up = min(268 - static_cast<int>(most >> 7), 253);   // biased exponent of the factor (254 has no inverse)
            const float f = __uint_as_float(static_cast<uint32_t>(up) << 23);
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
                reinterpret_cast<uint32_t *>(dst + j * D * 2)[lane + 32 * i] =
                    pack_half2(bf16_lo(w[i]) * f, bf16_hi(w[i]) * f);
            const float back = __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
            if ((lane & 3) == j) mine = p.scale_log2 * back;
        }
        return mine;
    }
};

// What a warp of RH heads from h0 on has come to, in its shared memory: sums [RH][2][DV], then m1, l1, m2, l2 of each.
template <int DV, int RH>
__device__ __forceinline__ float *left_sums(uint8_t *smem) { return reinterpret_cast<float *>(smem); }
template <int DV, int RH>
__device__ __forceinline__ float4 *left_stats(uint8_t *smem) { return reinterpret_cast<float4 *>(smem + RH * 2 * DV * 4); }

// The tiles of `range` (one at least) for noise head g and the signal heads from h0 on, `done` of which others do too.
// ONE: they are of one sequence, and what they come to is left in shared memory, else in slot split + sequence.
template <int D, int DV, int RH, bool LISTED, bool ONE>
__device__ __forceinline__ void run_range(const Params &p, const Maps &maps, const Range &range, uint8_t *const smem,
                                          const int split, const int g, const int h0, const int done) {
    using S = Stage<D, DV, RH>;
    constexpr int NH = S::NH, SLABS = DV < 128 ? 1 : DV / 128, WORDS = DV < 128 ? 2 : 4, A = S::count - 1;
    const int lane = threadIdx.x & 31, quad = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem);
    Cursor use{range.b, 0, 0, range.end - range.start};
    enter(use, range.start - range.before, range.span.tiles);
    Cursor get = use;                                    // the copies' place, ahead of the arithmetic's
    int get_len = range.span.len;
    Place next = place_of<LISTED>(p, get.b, g, get.tile, get_len);
    Queries<D, RH> q;
    q.fetch(p, use.b, h0, g);

    // scales of a tile: lanes 0 .. RH of K, 4 .. RH + 3 of V
    const int j_of = lane & 3, which = lane >= 4 ? 2 : (j_of < RH ? 0 : 1);
    const float *const scale_base = which == 0 ? p.k1s + h0 + j_of : (which == 1 ? p.k2s + g : p.vs + h0 + min(j_of, RH - 1));
    const uint32_t scale_pitch = which == 1 ? p.hn : p.hs;
    int last = 0, to = 0, counts[A + 1] = {};            // counts: positions of the last tiles copied, the latest at the end
    bool ready = true, pending = false;                  // K of `next`, V of the tile at row `last` are to be copied
    auto copy = [&]() {
        const uint32_t stage = ring + to * S::bytes, bar = ring + S::bars + to * 8;
        const int row = row_of(p, next), before = last;
        if (lane == 0 && (ready || pending)) {
            mbar_arrive_expect_tx(reinterpret_cast<uint64_t *>(smem + S::bars) + to,
                                  (ready ? S::k_bytes : 0) + (pending ? S::v_bytes : 0));
            if (pending) load_box(stage + S::v, maps.v, bar, before, h0 * (DV < 128 ? 1 : DV / 128));
            if (ready) {
                load_box(stage + S::k, maps.k1, bar, row, h0);
                load_box(stage + S::k + RH * kTile * D, maps.k2, bar, row, g);
            }
        }
        if (lane < 7 && ready)
            copy_async4(ring + S::scales + to * 32 + lane * 4,
                        scale_base + static_cast<size_t>(static_cast<uint32_t>(row) / kTile >> p.shift) * scale_pitch, next.n > 0);
        asm volatile("cp.async.commit_group;" ::: "memory");
        last = row;
#pragma unroll
        for (int i = 0; i < A; ++i) counts[i] = counts[i + 1];
        counts[A] = next.n;
        pending = ready;
        to = to == A ? 0 : to + 1;
        if (!ready) return;
        if (++get.tile >= get.hi) {
            if (get.left == 0) {
                ready = false;
                return;
            }
            get_len = next_sequence<LISTED>(p, get);
        }
        next = place_of<LISTED>(p, get.b, g, get.tile, get_len);
    };

    uint8_t *const queries = smem + S::queries, *const weights = smem + S::weights;
    float factor = 0.f;
    float acc[RH][SLABS * WORDS][4];                     // [w]: of tiles 2 w + t / 2 and map t % 2, see values_of
    float m = kLowest, l = 0.f;                          // of head t (both its lanes' positions; l of this lane's only)
    // of head t's two maps: what the scales of V in the weights are relative to, and 1 over it.  From 2^-126 on, whose
    // inverse is finite: smaller scales (or 0) are relative to that
    constexpr float kLeast = 0x1p-126f;
    float ref1 = 1.f, ref2 = 1.f, inverse1 = 1.f, inverse2 = 1.f;
    auto multiply = [](float (&a)[SLABS * WORDS][4], float f) {
#pragma unroll
        for (int i = 0; i < SLABS * WORDS; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) a[i][k] *= f;
    };
    auto clear = [&]() {
#pragma unroll
        for (int j = 0; j < RH; ++j)
#pragma unroll
            for (int i = 0; i < SLABS * WORDS; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[j][i][k] = 0.f;
    };
    // Where a tile's scale of V is above a map's reference or far below it: far above a tile the reference comes down as
    // what was added before has shrunk, and it goes up to the scale, or as far as the tile's largest weight `top` is worth.
    // (Where neither is looked at, R is at most kBand times the scale of a tile that raises the maximum.)  Powers of two
    // stay such where scales are within kBand of one another.
    auto refer = [](float &ref, float &inverse, float vs, float top, float by) {
        const float before = ref, worth = __uint_as_float(__float_as_uint(vs * (top * kBand)) & 0x7f800000u);
        ref = fmaxf(fmaxf(vs * kBand < ref ? ref * by : ref, top * kBand < 1.f ? worth : vs), kLeast);
        inverse = __frcp_rn(ref);
        return ref == before ? 1.f : fminf(before * inverse, 0x1p126f);   // (times `by` it is at most 1)
    };
    int have = kTile;                                    // positions of the tile scored last
    auto scores_of = [&](const uint8_t *const stage, const uint8_t *const scales) {
        // lane (quad, t) ends up with positions quad, quad + 8 of head t
        float sc0 = 0.f, sc1 = 0.f;
        const float ks = at<float>(scales + 4 * t), vs = at<float>(scales + 16 + 4 * t);
#pragma unroll
        for (int j = 0; j < NH; ++j) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {  // 16 dims of this lane
                // 16-byte chunks of rows of 128 bytes are exchanged by the row's low bits: two rows that eight lanes read
                // lie in different banks
                const int chunk = D == 64 ? t : 2 * t + half;
                const uint8_t *ka = stage + S::k + (j * kTile + quad) * D + (D == 64 ? chunk : chunk ^ quad) * 16;
                const uint8_t *qa = queries + j * D * 2 + chunk * 32;
                const uint4 lo = at<uint4>(ka), hi = at<uint4>(ka + 8 * D), b0 = at<uint4>(qa), b1 = at<uint4>(qa + 16);
                const uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, e[4] = {hi.x, hi.y, hi.z, hi.w};
                const uint32_t b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint2 x = e4m3x4_to_half2x2(a[i]), y = e4m3x4_to_half2x2(e[i]);
                    mma_16816(c, x.x, y.x, x.y, y.y, b[2 * i], b[2 * i + 1]);
                }
            }
            if (t == j) sc0 = c[0], sc1 = c[2];
        }
        have = counts[0];
        sc0 = sc0 * factor * ks, sc1 = sc1 * factor * ks;
        if (quad >= have) sc0 = -INFINITY;
        if (quad + 8 >= have) sc1 = -INFINITY;
        float tile = fmaxf(sc0, sc1);                    // the tile's largest score
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) tile = fmaxf(tile, __shfl_xor_sync(0xffffffffu, tile, o));
        const float mt = fmaxf(m, tile);
        const float shrink = fast_exp2(m - mt);
        const float p0 = fast_exp2(sc0 - mt + kWeightBits), p1 = fast_exp2(sc1 - mt + kWeightBits);
        m = mt;
        l = fmaf(l, shrink, p0 + p1);
        // what was added before shrinks by its scores, and by its references where this tile's scale of V is off them
        const bool off = t < RH && (vs > fminf(ref1, ref2) || vs * kBand < fmaxf(ref1, ref2));
        if (__any_sync(0xffffffffu, shrink != 1.f || off)) {
#pragma unroll
            for (int j = 0; j < RH; ++j) multiply(acc[j], __shfl_sync(0xffffffffu, shrink, t & 1 ? RH : j));
            if (__any_sync(0xffffffffu, off)) {
                const float top = fast_exp2(tile - mt);
                const float shrink1 = refer(ref1, inverse1, vs, top, shrink);
                const float shrink2 = refer(ref2, inverse2, vs, __shfl_sync(0xffffffffu, top, RH), __shfl_sync(0xffffffffu, shrink, RH));
#pragma unroll
                for (int j = 0; j < RH; ++j) {
                    const float by1 = __shfl_sync(0xffffffffu, shrink1, j), by2 = __shfl_sync(0xffffffffu, shrink2, j);
                    multiply(acc[j], t & 1 ? by2 : by1);
                }
            }
        }
        const float ratio1 = vs * inverse1, ratio2 = vs * inverse2;
        const float n0 = __shfl_sync(0xffffffffu, p0, (lane & ~3) | RH) * ratio2, n1 = __shfl_sync(0xffffffffu, p1, (lane & ~3) | RH) * ratio2;
        const float s0 = p0 * ratio1, s1 = p1 * ratio1;
        const uint32_t sh = pack_half2(s0, s1), nh = pack_half2(n0, n1);
        const float2 sf = half2_bits_to_float2(sh), nf = half2_bits_to_float2(nh);
        if (t < RH)
            *reinterpret_cast<uint4 *>(weights + t * 128 + quad * 16) =
                make_uint4(sh, pack_half2(s0 - sf.x, s1 - sf.y), nh, pack_half2(n0 - nf.x, n1 - nf.y));
    };

    auto values_of = [&](const uint8_t *const stage) {
        // k slots (2t, 2t + 1) are positions 2t, 2t + 8 and (2t + 8, 2t + 9) are 2t + 1, 2t + 9.  A lane has 4 WORDS dims
        // from 4 WORDS quad on (and 128 further, at DV = 256); tile 2 w has the first two of word w in its rows quad and
        // quad + 8, tile 2 w + 1 the others.  Columns 0 .. 3 are upper and lower parts of the signal map's weights and of
        // the noise map's for even tiles, 4 .. 7 for odd ones.
        constexpr int LOAD = 4 * WORDS, ROW = DV < 128 ? 64 : 128;
        // rows of 128 bytes: 16-byte chunks exchanged by the row's three low bits; of 64: by its bits 1 and 2
        uint32_t place[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t row = 2 * t + 8 * (k & 1) + (k >> 1);
            place[k] = row * ROW + (DV == 64 ? ((quad >> 1) ^ (row >> 1 & 3)) * 16 + (quad & 1) * 8 : (quad ^ (row & 7)) * 16);
        }
#pragma unroll
        for (int j = 0; j < RH; ++j) {
            const uint8_t *wa = weights + j * 128 + t * 32 + (quad & 3) * 4;
            const uint32_t w0 = at<uint32_t>(wa), w1 = at<uint32_t>(wa + 16);
            const uint32_t even0 = quad < 4 ? w0 : 0u, even1 = quad < 4 ? w1 : 0u;
            const uint32_t odd0 = quad < 4 ? 0u : w0, odd1 = quad < 4 ? 0u : w1;
            const uint8_t *va = stage + S::v + j * kTile * DV;
#pragma unroll
            for (int s = 0; s < SLABS; ++s) {
                uint32_t x[4][WORDS];                    // [2t, 2t + 8, 2t + 1, 2t + 9]
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint8_t *row = va + s * kTile * 128 + place[k];
                    if constexpr (LOAD == 8) {
                        const uint2 v = at<uint2>(row);
                        x[k][0] = v.x, x[k][1] = v.y;
                    } else {
                        const uint4 v = at<uint4>(row);
                        x[k][0] = v.x, x[k][1] = v.y, x[k][2] = v.z, x[k][3] = v.w;
                    }
                }
#pragma unroll
                for (int w = 0; w < WORDS; ++w) {
                    // bytes of two positions side by side: two dims, one in each half
                    const uint2 a = e4m3x4_to_half2x2(__byte_perm(x[0][w], x[1][w], 0x5140));
                    const uint2 c = e4m3x4_to_half2x2(__byte_perm(x[2][w], x[3][w], 0x5140));
                    mma_16816(acc[j][s * WORDS + w], a.x, a.y, c.x, c.y, even0, even1);
                    const uint2 e = e4m3x4_to_half2x2(__byte_perm(x[0][w], x[1][w], 0x7362));
                    const uint2 f = e4m3x4_to_half2x2(__byte_perm(x[2][w], x[3][w], 0x7362));
                    mma_16816(acc[j][s * WORDS + w], e.x, e.y, f.x, f.y, odd0, odd1);
                }
            }
        }
    };
    // Rows of V behind the last position of a tile are whatever the cache holds there, NaN codes too, which no weight of 0
    // takes away: they become zeros.
    auto drop_rows = [&](uint8_t *const stage) {
        constexpr int ROW = DV < 128 ? 64 : 128, ROWS = RH * kTile * DV / ROW;
        for (int i = lane; i < ROWS * ROW / 16; i += 32)
            if (i / (ROW / 16) % kTile >= have) *reinterpret_cast<uint4 *>(stage + S::v + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
    };
    // Leaves what the part that lies in sequence b has come to.
    auto leave = [&](int b) {
        if constexpr (ONE) __syncwarp();                 // it goes to where the tiles were
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        l *= 0x1p-15f;
        const float mn = __shfl_sync(0xffffffffu, m, RH), ln = __shfl_sync(0xffffffffu, l, RH);
        const size_t slot = static_cast<size_t>(split) + b;
#pragma unroll
        for (int j = 0; j < RH; ++j) {
            const float mj = __shfl_sync(0xffffffffu, m, j), lj = __shfl_sync(0xffffffffu, l, j);
            // sums over values from 2^64 on could leave float32: they and the sum of weights are left 2^64 smaller, and the
            // maximum, in powers of two, as much larger, which is the same to whoever joins the parts
            const float r1 = __shfl_sync(0xffffffffu, ref1, j), r2 = __shfl_sync(0xffffffffu, ref2, j);
            const float down1 = r1 > 0x1p64f ? 0x1p-64f : 1.f, up1 = r1 > 0x1p64f ? 64.f : 0.f;
            const float down2 = r2 > 0x1p64f ? 0x1p-64f : 1.f, up2 = r2 > 0x1p64f ? 64.f : 0.f;
            const float v = (t & 1 ? r2 * down2 : r1 * down1) * 0x1p-15f;
            if (j < done) continue;
            const size_t place = slot * p.hs + h0 + j;
            float4 *const stats = ONE ? left_stats<DV, RH>(smem) + j : reinterpret_cast<float4 *>(p.ws_ml) + place;
            if (lane == 0) *stats = make_float4(mj + up1, lj * down1, mn + up2, ln * down2);
            float *const o = (ONE ? left_sums<DV, RH>(smem) + j * 2 * DV : p.ws_o + place * 2 * DV) + (t & 1) * DV +
                             4 * WORDS * quad + 2 * (t >> 1);
#pragma unroll
            for (int i = 0; i < SLABS * WORDS; ++i) {
                const float(&c)[4] = acc[j][i];
                *reinterpret_cast<float2 *>(o + i / WORDS * 128 + i % WORDS * 4) = make_float2((c[0] + c[1]) * v, (c[2] + c[3]) * v);
            }
        }
    };

    // Step g: the values of tile g - 1, what ends with it and begins with tile g, and the scores of tile g.  Every piece
    // of the work stands in one place: a kernel starts with cold instructions, and what a first and a last step had of
    // their own cost more than the order of the pieces gains.
    int from = 0, ahead = A;                             // steps until the first tile is there
    uint32_t parity = 0;                                 // of each stage's barrier
    int part_of = -1;                                    // the sequence of the part that is under way
    bool ending = true, over = false;                    // the tile scored last was its part's last; the range's last
    for (;;) {
        __syncwarp();                                    // the readers of the stage to be written are done
        copy();
        if (ahead > 0) {
            --ahead;
            continue;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(A) : "memory");
        if (!mbar_wait_warp(ring + S::bars + from * 8, parity >> from & 1u)) {
            // it gives up; the copies of the other stages are waited for, as long again
            atomicOr(p.err, GDA_DEVERR_DECODE_TIMEOUT);
            for (int i = 0; i < S::count; ++i) mbar_wait_warp(ring + S::bars + i * 8, parity >> i & 1u);
            return;
        }
        parity ^= 1u << from;
        __syncwarp();                                    // every lane's copies of this stage have landed
        uint8_t *const stage = smem + from * S::bytes;
        const uint8_t *const scales = smem + S::scales + from * 32;
        from = from == A ? 0 : from + 1;
        if (part_of >= 0) {
            if (have < kTile) drop_rows(stage);
            values_of(stage);
        }
        if (ending) {
            if (part_of >= 0) leave(part_of);
            if (over) return;
            factor = q.place(p, queries);
            clear();
            m = kLowest, l = 0.f;
            ref1 = ref2 = fmaxf(at<float>(scales + 16 + 4 * t), kLeast);   // its largest weights are 1
            inverse1 = inverse2 = __frcp_rn(ref1);
            part_of = use.b;
        }
        __syncwarp();                                    // the weights have been read, the queries are there
        scores_of(stage, scales);
        ending = ++use.tile >= use.hi;
        if (ending) {
            over = use.left == 0;
            if (!over) {
                next_sequence<LISTED>(p, use);
                q.fetch(p, use.b, h0, g);
            }
        }
    }
}

// One warp: split u / units of the range, unit u % units = (noise head, part of its group).
template <int D, int DV, int RH, bool LISTED>
__global__ void __launch_bounds__(32, (Stage<D, DV, RH>::warps)) gda_decode_fp8_block_split_kernel(
    const Params p, const __grid_constant__ Maps maps) {
    using S = Stage<D, DV, RH>;
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t *const smem = raw + (-smem_u32(raw) & 1023u);
    const int lane = threadIdx.x, units = p.hn * p.parts, u = blockIdx.x;
    const int split = u / units, g = (u % units) / p.parts, part = u % p.parts;
    // every part is RH heads: the last begins early where they do not divide the group, and leaves what the parts
    // before it have done unwritten
    const int r = p.hs / p.hn, begin = min(part * RH, r - RH), done = part * RH - begin, h0 = g * r + begin;
    // a programmatic dependent of whatever is ahead in the stream: nothing is read or written before that has completed
    if (lane < S::count) mbar_init(reinterpret_cast<uint64_t *>(smem + S::bars) + lane, 1);
    fence_mbar_init();
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Range range;
    if (!range_of<LISTED>(p, split, range)) return;
    if (u % units == 0) note_sequences<LISTED>(p, range, split);
    run_range<D, DV, RH, LISTED, false>(p, maps, range, smem, split, g, h0, done);
}

// The statistics and sums of parts joined one after the other: a warp to a head, COLS of each map's columns to a lane.
template <int COLS>
struct Joined {
    float4 stats = make_float4(kLowest, 0.f, kLowest, 0.f);
    float o1[COLS] = {}, o2[COLS] = {};

    // sums: this lane's columns of the first map, those of the second DV behind them
    __device__ __forceinline__ void add(const float4 s, const float *sums, int dv) {
        const float t1 = fmaxf(stats.x, s.x), t2 = fmaxf(stats.z, s.z);
        const float f1 = fast_exp2(stats.x - t1), g1 = fast_exp2(s.x - t1), f2 = fast_exp2(stats.z - t2), g2 = fast_exp2(s.z - t2);
        stats = make_float4(t1, fmaf(s.y, g1, stats.y * f1), t2, fmaf(s.w, g2, stats.w * f2));
#pragma unroll
        for (int i = 0; i < COLS; i += 2) {
            const float2 x = *reinterpret_cast<const float2 *>(sums + i), y = *reinterpret_cast<const float2 *>(sums + dv + i);
            o1[i] = fmaf(x.x, g1, o1[i] * f1), o1[i + 1] = fmaf(x.y, g1, o1[i + 1] * f1);
            o2[i] = fmaf(y.x, g2, o2[i] * f2), o2[i + 1] = fmaf(y.y, g2, o2[i + 1] * f2);
        }
    }
};

// The row of sequence b and head h, by a whole warp.
template <int COLS>
__device__ __forceinline__ void write_row(const Params &p, Joined<COLS> &sum, int b, int h) {
    constexpr int DV = 32 * COLS;
    const int lane = threadIdx.x & 31;
    uint32_t *const out = reinterpret_cast<uint32_t *>(p.out + (static_cast<size_t>(b) * p.hs + h) * DV) + lane * COLS / 2;
    if (sum.stats.y == 0.f) {                                // no position (a NaN is not 0)
#pragma unroll
        for (int i = 0; i < COLS; i += 2) out[i / 2] = 0u;
        return;
    }
    const float i1 = 1.f / sum.stats.y, i2 = p.lambda[h] / sum.stats.w;
    float v[COLS], ss, early = 1.f, late = 1.f;
    for (int round = 0;; ++round) {
        const float e1 = i1 * early, e2 = i2 * early;
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < COLS; ++i) v[i] = (sum.o1[i] * e1 - sum.o2[i] * e2) * late, ss = fmaf(v[i], v[i], ss);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (round > 0 || norm_in_range(ss, p.eps, early, late)) break;
    }
    const float y = norm_factor(ss, DV, p.eps, p.lambda_init, early, late);
#pragma unroll
    for (int i = 0; i < COLS; i += 2) out[i / 2] = pack_bf16x2(v[i] * y, v[i + 1] * y);
}

// grid (units x ranks, B): a cluster of `ranks` blocks of threads to a sequence and unit, their warps to equal parts of
// the tiles, joined in shared memory, first within a block and then by the cluster's first.  One launch instead of two,
// for short sequences.
template <int D, int DV, int RH, bool LISTED>
__global__ void __launch_bounds__(32 * kOneWarps, 1) gda_decode_fp8_block_one_kernel(const Params p,
                                                                                     const __grid_constant__ Maps maps) {
    using S = Stage<D, DV, RH>;
    constexpr int COLS = DV / 32;                            // of a lane, in joining
    extern __shared__ __align__(1024) uint8_t raw[];
    __shared__ __align__(16) float joined[RH][2 * DV];
    __shared__ float4 joined_stats[RH];
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
    uint8_t *const all = raw + (-smem_u32(raw) & 1023u);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, b = blockIdx.y;
    const int u = blockIdx.x / ranks, g = u / p.parts, part = u % p.parts;
    const int r = p.hs / p.hn, begin = min(part * RH, r - RH), done = part * RH - begin, h0 = g * r + begin;
    uint8_t *const smem = all + warp * S::pitch;
    if (lane < S::count) mbar_init(reinterpret_cast<uint64_t *>(smem + S::bars) + lane, 1);
    fence_mbar_init();
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Span span = span_of<LISTED>(p, b);
    const int per = (span.tiles + warps * ranks - 1) / (warps * ranks);
    const int first = rank * warps * per, used = per > 0 ? min(warps, max(0, (span.tiles - first + per - 1) / per)) : 0;
    if (warp < used) {
        const int start = first + warp * per;
        const Range range{start, min(span.tiles, start + per), per, 0, b, span};
        run_range<D, DV, RH, LISTED, true>(p, maps, range, smem, 0, g, h0, done);
    }
    __syncthreads();
    for (int j = done + warp; j < RH; j += warps) {          // (four warps at least: one round)
        Joined<COLS> sum;
        for (int c = 0; c < used; ++c) {
            uint8_t *const left = all + c * S::pitch;
            sum.add(left_stats<DV, RH>(left)[j], left_sums<DV, RH>(left) + j * 2 * DV + lane * COLS, DV);
        }
        if (ranks > 1) {
            if (lane == 0) joined_stats[j] = sum.stats;
#pragma unroll
            for (int i = 0; i < COLS; i += 2) {
                *reinterpret_cast<float2 *>(&joined[j][lane * COLS + i]) = make_float2(sum.o1[i], sum.o1[i + 1]);
                *reinterpret_cast<float2 *>(&joined[j][DV + lane * COLS + i]) = make_float2(sum.o2[i], sum.o2[i + 1]);
            }
            continue;
        }
        write_row<COLS>(p, sum, b, h0 + j);
    }
    if (ranks == 1) return;
    cluster.sync();
    if (rank == 0)
        for (int j = done + warp; j < RH; j += warps) {
            Joined<COLS> sum;
#pragma unroll 4
            for (int c = 0; c < ranks; ++c)
                sum.add(*cluster.map_shared_rank(&joined_stats[j], c), cluster.map_shared_rank(&joined[j][lane * COLS], c), DV);
            write_row<COLS>(p, sum, b, h0 + j);
        }
    cluster.sync();                                          // no block goes while its sums are read
}

// Blocks of threads of a cluster and warps of a block for a sequence in one launch; ranks = 0: two launches.  `fit`: warps
// that an SM holds.
//
// Both are estimated in us, from the room in the block table or the lists, as the lengths are on the device (lists are
// taken to be full, caches for three quarters): two launches cost kTwoFixed and kStep for each step of their equal
// ranges; one costs kOneFixed, kWave for each further wave of blocks of threads, and for each step of a warp kOneStep, its
// tile's latency, or what the bytes take if that is more.  2 us of kTwoFixed stand for the host's 4 to 5.  us of a call from
// Python (graph replay, inputs in HBM), one / two launches, 12 + 4 heads of 64/128: one sequence of 256 23 (13.4) / 27
// (14.5); 16 of 512 24 (17.5) / 29 (19.6), of 2048 23 (30) / 28 (32); 64 of 256 23 (20) / 27 (24), of 512 24 (28) / 27 (32),
// of 1 to 1024 28 (36) / 27 (34), where the estimates are equal, of 2048 57 (75) / 61 (81), where they are 55.5 and 50.7, so
// that the slower two are taken; 256 of 512 74 (87) / 67 (87); lists of 16 blocks of 64 for 64 sequences 33.6 (46) / 37.8
// (54).  Sixteen clusters of eight do not run at once: four sequences of 1024 took 21.6 with those and 17.5 with two
// launches.
constexpr double kTwoFixed = 12.3, kOneFixed = 7.5, kOneCluster = 1.0, kWave = 2.0, kStep = 1.9, kOneStep = 1.5;
struct OneLaunch {
    int ranks = 0, warps = 0;
};
OneLaunch one_launch(const Params &p, int fit) {
    const long long reach = p.list != nullptr ? static_cast<long long>(p.keep) << p.shift : (p.Lcap + kTile - 1) / kTile;
    const long long blocks = static_cast<long long>(p.hn) * p.parts * p.B;
    const double bytes = kStep * (p.list != nullptr ? 1.0 : 0.75) * static_cast<double>(blocks) * reach / (kSms * fit);
    OneLaunch best;
    double least = kTwoFixed + bytes;
    for (int ranks = 1; ranks <= 8; ranks *= 2) {
        if (ranks > 1 && blocks * ranks > (ranks == 8 ? 64 : 128)) break;
        for (const int warps : {4, std::min(fit, kOneWarps)}) {
            if (warps < 4 || warps > fit) continue;
            const long long at_once = static_cast<long long>(kSms) * (fit / warps);
            const long long waves = (blocks * ranks + at_once - 1) / at_once, steps = (reach + warps * ranks - 1) / (warps * ranks);
            const double us = kOneFixed + (ranks > 1 ? kOneCluster : 0.0) + kWave * static_cast<double>(waves - 1) +
                              std::max(kOneStep * static_cast<double>(waves * steps), bytes);
            if (us < least) least = us, best = {ranks, warps};
        }
    }
    return best;
}

// Rows of `heads` heads of n bytes each, in boxes of (at most 128 bytes) x 16 cache rows x `box` of those.
// Where noise heads list blocks of their own, no other warp reads what lies beside a head's part of a row, so L2 is to
// fetch no more than that.
bool encode(CUtensorMap *map, const uint8_t *base, int n, int heads, long long rows, int box, int swizzle, bool listed) {
    const int piece = n < 128 ? n : 128;
    const uint64_t dims[3] = {static_cast<uint64_t>(piece), static_cast<uint64_t>(rows),
                              static_cast<uint64_t>(heads) * (n / piece)};
    const uint64_t strides[2] = {static_cast<uint64_t>(heads) * n, static_cast<uint64_t>(piece)};
    const uint32_t shape[3] = {static_cast<uint32_t>(piece), kTile, static_cast<uint32_t>(box * (n / piece))};
    return encode_tmap_3d_u8(map, base, dims, strides, shape, swizzle, listed);
}

template <int D, int DV, int RH, bool LISTED>
cudaError_t launch(const Params &p, cudaStream_t stream) {
    using S = Stage<D, DV, RH>;
    constexpr auto split = gda_decode_fp8_block_split_kernel<D, DV, RH, LISTED>;
    constexpr auto one = gda_decode_fp8_block_one_kernel<D, DV, RH, LISTED>;
    Maps maps;
    const long long rows = static_cast<long long>(p.num_pages) * p.page_size;
    constexpr int KS = D == 64 ? 0 : 128, VS = DV == 64 ? 64 : 128;
    if (!encode(&maps.k1, p.k1c, D, p.hs, rows, RH, KS, LISTED) || !encode(&maps.k2, p.k2c, D, p.hn, rows, 1, KS, LISTED) ||
        !encode(&maps.v, p.vc, DV, p.hs, rows, RH, VS, LISTED))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (const OneLaunch w = one_launch(p, S::warps); w.ranks > 0) {
        constexpr int most = S::warps < kOneWarps ? S::warps : kOneWarps;
        static_assert(most * S::pitch + 1024 + RH * (2 * DV * 4 + 16) + 64 <= 227 * 1024, "a block of threads fits an SM");
        const cudaError_t e = allow_shared_memory<one>(most * S::pitch + 1024);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(p.hn * p.parts * w.ranks, p.B);
        cfg.blockDim = dim3(32 * w.warps);
        cfg.dynamicSmemBytes = w.warps * S::pitch + 1024;
        if (w.ranks > 1) {
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = w.ranks;
            attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
            cfg.numAttrs = 2;
        }
        return cudaLaunchKernelEx(&cfg, one, p, maps);
    }
    cudaError_t e = allow_shared_memory<split>(S::total);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(p.splits * p.hn * p.parts);
    cfg.blockDim = dim3(32);
    cfg.dynamicSmemBytes = S::total;
    e = cudaLaunchKernelEx(&cfg, split, p, maps);
    return e == cudaSuccess ? launch_join<DV>(p, stream) : e;
}

template <int D, int DV, int RH>
cudaError_t launch(const Params &p, cudaStream_t stream) {
    return p.list != nullptr ? launch<D, DV, RH, true>(p, stream) : launch<D, DV, RH, false>(p, stream);
}

template <int D, int DV>
cudaError_t launch(const Params &p, int rh, cudaStream_t stream) {
    if (rh == 1) return launch<D, DV, 1>(p, stream);
    if constexpr (DV < 256)
        if (rh == 3) return launch<D, DV, 3>(p, stream);
    return launch<D, DV, 2>(p, stream);
}

}  // namespace

size_t decode_fp8_block_workspace_bytes(int B, int hs, int hn, int d, int dv) { return plan_of(B, hs, hn, d, dv).bytes; }

int launch_decode_fp8_block(const DecodeFp8BlockArgs &a, cudaStream_t stream) {
    const Plan pl = plan_of(a.B, a.hs, a.hn, a.d, a.dv);
    char *ws = static_cast<char *>(a.workspace);
    int shift = 0, page_shift = 31;
    while (kTile << shift < a.block) ++shift;
    const uint32_t page_tiles = a.page_size / kTile;     // factor = 2^(31 + l) / page_tiles, rounded up, 2^l >= page_tiles
    while (1ull << (page_shift - 31) < page_tiles) ++page_shift;
    const uint32_t page_factor = static_cast<uint32_t>(((1ull << page_shift) + page_tiles - 1) / page_tiles);
    const Params p{static_cast<const __nv_bfloat16 *>(a.q1),
                   static_cast<const __nv_bfloat16 *>(a.q2),
                   a.k1c, a.k2c, a.vc, a.k1s, a.k2s, a.vs, a.lens, a.lambda,
                   static_cast<__nv_bfloat16 *>(a.out),
                   reinterpret_cast<float *>(ws),
                   reinterpret_cast<float *>(ws + pl.ml_at),
                   reinterpret_cast<int *>(ws + pl.seg_at),
                   a.dev_err, a.lambda_init, a.eps,
                   static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a.d))),
                   a.B, a.Lcap, a.hs, a.hn, pl.splits, pl.heads.parts, a.block_table, a.page_size, a.max_pages,
                   a.num_pages, shift, page_factor, page_shift, a.list, a.count, a.keep};
    cudaError_t e = cudaErrorInvalidValue;
    switch (a.d * 1000 + a.dv) {
        case 64064: e = launch<64, 64>(p, pl.heads.each, stream); break;
        case 64128: e = launch<64, 128>(p, pl.heads.each, stream); break;
        case 64256: e = launch<64, 256>(p, pl.heads.each, stream); break;
        case 128064: e = launch<128, 64>(p, pl.heads.each, stream); break;
        case 128128: e = launch<128, 128>(p, pl.heads.each, stream); break;
        case 128256: e = launch<128, 256>(p, pl.heads.each, stream); break;
        default: return GDA_ERR_UNSUPPORTED;
    }
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

}  // namespace gda
