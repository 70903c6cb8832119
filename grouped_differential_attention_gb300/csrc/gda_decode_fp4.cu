// Grouped differential attention decode over a 4-bit KV cache (one new query
// token per sequence; format in gda_fp4.cuh), contiguous or paged, split over
// the cache length, plus a combine pass.
//
// The batch's cache positions, concatenated sequence after sequence, are cut
// into equal contiguous ranges.  A warp takes one range for one noise head
// and up to RH signal heads that share it, on its own: it copies 16 positions
// at a time into a ring of its own in shared memory (cp.async, one to four
// tiles ahead, so no thread of another warp is ever waited for), and keeps the
// online softmax of all its maps and the accumulators O1, O2 in registers.
// Each part of a range that lies in one sequence leaves (m, l) of both maps
// and (O1, O2) in workspace slot (range + sequence), which is unique because
// along the position axis neither index falls and one grows from part to
// part.  The combine kernel joins the parts of a sequence and applies the
// difference and the (1 - lambda_init) RMSNorm.
//
// Bytes are few (9/16 per element), so the arithmetic decides.  On the CUDA
// cores every element costs a widening and one (K) or two (V) multiply-adds:
// at the copy rate that is more than they can do (the fp8 decode, with half
// the elements per byte, already is bound by them).  Here the tensor cores
// multiply (mma.sync m16n8k16, f16 in, float32 out; a tile of a decode has
// one row of queries, so the 128-row tcgen05 forms would sit idle for 127),
// and the work left per element is half a conversion.  An mma has eight
// columns where a decode needs one or two; the others are put to use:
//   - scores: A = codes of 16 positions, B column n = the query with all but
//     its n-th block of 16 dims zeroed, so C holds the dot product of every
//     block by itself, and a score is sum_n scale[n] * C[n];
//   - values: A = code * scale of 16 dims x 16 positions, B = four columns of
//     weights, the upper and the lower part of both maps', the other four
//     zero, so that two tiles of dims share one set of accumulators.
// e2m1 codes, e4m3 scales and their products are exact in f16; the query is
// too, after a power of two.  A weight is two f16 numbers, its first 11 bits
// and what they leave, so that it keeps 22 bits down to 2^-18 of its map's
// largest and 2^-40 of that below (rounded to one f16, with the scale in B,
// the 64 sequences below took 115 us and not 120, but outputs were off by
// 2^-12 of their terms, and weights below 2^-32 were lost).  The weights are 2^15
// exp2(score - maximum); numerator and denominator share the factor.
//
// Measured (both kernels; of the 6793 GB/s of a copy): 64 sequences of 4096 to
// 8192, 12 + 4 heads of 64/128, 566 MB: 120 us (70 %); one of 131072, 24 + 8
// heads, 378 MB: 93 us (60 %); 16 of up to 8191, 16 + 4 heads of 128/256,
// 245 MB: 64 us (57 %).  The first one's split kernel takes 114 us; with the
// weights rounded it took 108, of which the copies alone 98 and the arithmetic
// alone 90: they overlap but for the start (a cold first tile arrives after
// several us) and the slowest warps, 10 % behind the mean.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gda.h"
#include "gda_decode_join.cuh"
#include "gda_device.cuh"
#include "gda_fp4.cuh"
#include "gda_internal.h"

namespace gda {
namespace {

constexpr int kWarpsPerBlock = 4;
constexpr int kTile = 16;              // positions of a tile
// Fewest positions of a range: a tile.  4 sequences of 37 to 600, us of both kernels: 15 with 16, 15.5 with 32, 17.2 with
// 64, 22.7 with 128.
constexpr int kMinRange = 16;
constexpr float kWeightBits = 15.f;    // weights carry a factor 2^15: the largest is within f16, the smallest far from its end

// Signal heads of a warp: a noise head's group in equal parts of at most three
// (two at dv = 256, where three tiles of three signal heads of 128 would leave an
// SM one block).  Every part reads and scores the noise head for itself, and where
// the parts do not divide the group the last one does a head again, so a part
// costs about its heads and one more; the fewest of those are taken, of as many
// the smaller parts.  us in the split kernel, 64 sequences of 4096 to 8192, 4
// noise heads of 64/128: groups of three as 3 113, as 2 + 2 153; of four as 2 +
// 2 163, as ones 202; of five as 3 + 3 217, as 2 + 2 + 2 225; of seven as three
// of 3 324, as four of 2 303.  16 sequences, 4 noise heads of 128/256: groups
// of three as 2 + 2 56, as ones 52; of four as 2 + 2 59, as ones 67.
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

// Blocks that share an SM, by the accumulator registers of a thread (DV / 8
// for each signal head).  us in the split kernel, this many / one fewer, 4
// noise heads, one signal head each: 64 sequences of 4096 to 8192 of 64/128
// 57.5 / 58, of 64/64 46.5 / 48.5; 32 of 128/128 38.5 / 38.5; two: 82 / 89 of
// 64/128, 53 / 57 of 128/128; three of 64/64 86 / 96.  One more makes no
// difference (three signal heads of 64/128 113 / 113 with one fewer tile in the
// ring, one of 131072 positions 94.4 / 94.5 with the joining of its parts).
// And as few as leave each warp a ring of three tiles, two of which are in use
// at a time; with four or more, two signal heads of 128/256 take 75 against 59,
// three of 128/128 92 against 73.
constexpr int kMinRing = 3, kMaxRing = 6;

// Bytes of shared memory of 16 positions: codes and block scales of rh + 1 rows of K and rh of V.
__host__ __device__ constexpr int tile_bytes(int rh, int d, int dv) {
    return kTile * ((rh + 1) * (d / 2 + d / 16) + rh * (dv / 2 + dv / 16));
}
// Tiles of a warp's ring; a block also has the f16 queries of its warps and as many zeros as those of one.
__host__ __device__ constexpr int ring_of(int blocks, int rh, int d, int dv) {
    const int queries = (rh + 1) * d * 2;
    const int fit = ((227 * 1024 / blocks - 1024 - queries) / kWarpsPerBlock - queries) / tile_bytes(rh, d, dv);
    return fit > kMaxRing ? kMaxRing : fit;
}
__host__ __device__ constexpr int blocks_per_sm(int rh, int d, int dv) {
    int blocks = rh * dv / 8 <= 16 ? 4 : (rh * dv / 8 <= 32 ? 3 : 2);
    while (blocks > 1 && ring_of(blocks, rh, d, dv) < kMinRing) --blocks;
    return blocks;
}

struct Fp4Plan {
    Heads heads;
    int splits;        // ranges at most
    size_t ml_at, seg_at, bytes;
};

Fp4Plan plan_of(int B, int hs, int hn, int d, int dv) {
    Fp4Plan p;
    p.heads = heads_of(hs, hn, dv);
    p.splits = std::max(1, kSms * blocks_per_sm(p.heads.each, d, dv) * kWarpsPerBlock / (hn * p.heads.parts));
    const size_t slots = static_cast<size_t>(p.splits) + B;
    p.ml_at = (slots * hs * 2 * dv * sizeof(float) + 255) / 256 * 256;
    p.seg_at = p.ml_at + (slots * hs * 4 * sizeof(float) + 255) / 256 * 256;
    p.bytes = p.seg_at + static_cast<size_t>(B) * 2 * sizeof(int);
    return p;
}

struct Params {
    const __nv_bfloat16 *q1, *q2;
    const uint8_t *k1c, *k2c, *vc, *k1b, *k2b, *vb;
    const float *k1_scale, *k2_scale, *v_scale;
    const int *lens;
    const float *lambda;
    __nv_bfloat16 *out;
    float *ws_o;       // [slots][hs][2][dv]
    float *ws_ml;      // [slots][hs][4]: m1, l1, m2, l2
    int *ws_seg;       // [B][2]: first and last range of a sequence
    unsigned *err;
    float lambda_init, eps, scale_log2;
    int B, Lcap, hs, hn;
    int splits, parts;   // ranges; parts of a noise head's group
    const int *block_table;
    int page_size, max_pages, num_pages;
};

// Length of sequence b; one outside [0, Lcap] is clamped and reported.
__device__ __forceinline__ int length_of(const Params &p, int b) {
    const int len = p.lens[b];
    if (len >= 0 && len <= p.Lcap) return len;
    atomicOr(p.err, GDA_DEVERR_BAD_LENGTH);
    return len < 0 ? 0 : p.Lcap;
}

__device__ __forceinline__ int positions_of(const Params &p, int b) { return length_of(p, b); }

// Cache row of position pos of sequence b.  A page outside the pool is read
// as page 0 and reported.  (The caches have 2^32 rows at most.)
__device__ __forceinline__ uint32_t row_of(const Params &p, int b, int pos) {
    if (p.block_table == nullptr) return static_cast<uint32_t>(b) * static_cast<uint32_t>(p.Lcap) + pos;
    const int pg = pos / p.page_size;
    int phys = p.block_table[static_cast<size_t>(b) * p.max_pages + pg];
    if (phys < 0 || phys >= p.num_pages) {
        atomicOr(p.err, GDA_DEVERR_BAD_PAGE);
        phys = 0;
    }
    return static_cast<uint32_t>(phys) * p.page_size + (pos - pg * p.page_size);
}

// The range [start, end) of a split in the concatenated positions, and where it begins.
struct Range {
    long long start, end, per, before;   // before: positions of the sequences ahead of b
    int b;
};

// Computed by a whole warp; false if the split has nothing to do.
__device__ __forceinline__ bool range_of(const Params &p, int split, Range &r) {
    const int lane = threadIdx.x & 31;
    long long total = 0;
#pragma unroll 4
    for (int b = lane; b < p.B; b += 32) total += length_of(p, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    r.per = max(static_cast<long long>(kMinRange), (total + p.splits - 1) / p.splits);
    r.per = (r.per + 15) / 16 * 16;
    r.start = split * r.per;
    r.end = min(total, r.start + r.per);
    if (r.start >= total) return false;
    long long carry = 0;
    for (int base = 0; base < p.B; base += 32) {
        const int b = base + lane;
        const long long len = b < p.B ? length_of(p, b) : 0;
        long long incl = len;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const long long before = carry + incl - len;
        const unsigned hit = __ballot_sync(0xffffffffu, before <= r.start && r.start < before + len);
        if (hit) {
            const int src = __ffs(hit) - 1;
            r.b = base + src;
            r.before = __shfl_sync(0xffffffffu, before, src);
            return true;
        }
        carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;                         // not reached: start < total
}

// Notes the first and last range of every sequence that begins in range r of split `split`, for the combine kernel.
__device__ __forceinline__ void note_sequences(const Params &p, const Range &r, int split) {
    long long before = r.before;
    for (int b = r.b; before < r.end; ++b) {
        const int len = length_of(p, b);
        if (len > 0 && before >= r.start && (threadIdx.x & 31) == 0) {
            p.ws_seg[2 * b] = split;
            p.ws_seg[2 * b + 1] = static_cast<int>((before + len - 1) / r.per);
        }
        before += len;
    }
}

// BYTES into shared memory, asynchronous; zeros in their place if `ok` is false, nothing at all if `there` is,
// (a predicate of the one instruction, not a branch around it).
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t *src, bool ok, bool there = true) {
    const int n = ok ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t"
                     "@p cp.async.cg.shared.global [%0], [%1], 16, %2;\n\t}" ::"r"(dst),
                     "l"(src), "r"(n), "r"(static_cast<int>(there)) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "@p cp.async.ca.shared.global [%0], [%1], %2, %3;\n\t}" ::"r"(dst),
                     "l"(src), "n"(BYTES), "r"(n), "r"(static_cast<int>(there)) : "memory");
}

// a * b + c: 16 x 16 (f16) times 16 x 8 (f16).
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

// A place in a warp's range: sequence b, positions [pos, hi) of it, and the positions of the range after those.
struct Cursor {
    int b, pos, hi, left;
};

__device__ __forceinline__ void enter(const Params &p, Cursor &c, int pos, int len) {
    const int n = min(len - pos, c.left);
    c.pos = pos;
    c.hi = pos + n;
    c.left -= n;
}

// To the next sequence with positions; there is one while left > 0.
__device__ __forceinline__ void next_sequence(const Params &p, Cursor &c) {
    int len = 0;
    do len = length_of(p, ++c.b);
    while (len == 0);
    enter(p, c, 0, len);
}

// Sizes of a warp's tile in shared memory, in bytes.
template <int D, int DV, int RH>
struct Tile {
    static constexpr int NH = RH + 1;                    // heads with scores; the noise head is the last
    static constexpr int KC = D / 2, KS = D / 16, VC = DV / 2, VS = DV / 16;   // codes and scales of a head row
    static constexpr int k_codes = 0;
    static constexpr int v_codes = k_codes + NH * kTile * KC;
    static constexpr int k_scales = v_codes + RH * kTile * VC;
    static constexpr int v_scales = k_scales + NH * kTile * KS;
    static constexpr int bytes = v_scales + RH * kTile * VS;
    static_assert(bytes == tile_bytes(RH, D, DV) && bytes % 16 == 0, "tiles follow one another");
    static constexpr int queries = NH * D * 2;           // f16; a block has as many bytes of zeros once more
    static constexpr int blocks = blocks_per_sm(RH, D, DV);
    static constexpr int ring = ring_of(blocks, RH, D, DV);   // tiles of the ring
    static_assert(ring >= 3, "a tile must be copied while two others are used");
    static constexpr int warp_bytes = ring * bytes + queries;
};

// V codes in shared memory: position pos is row v_row(pos), so that a lane's
// four positions 2t, 2t + 8, 2t + 1, 2t + 9 are rows t, t + 4, t + 8, t + 12;
// 16-byte chunks of a row change places by its low bits, so that the rows t =
// 0 .. 3 that one load reads lie in different banks.
__device__ __forceinline__ int v_row(int pos) { return (pos >> 1) | ((pos & 1) << 3); }
template <int DV>
__device__ __forceinline__ int v_chunk(int row, int chunk) {
    if constexpr (DV == 128) return chunk ^ (((row >> 1) & 1) << 1);
    if constexpr (DV == 256) return chunk ^ ((row & 3) << 1);
    return chunk;
}

// base + row * pitch, one multiply-add.
__device__ __forceinline__ const uint8_t *row_at(const uint8_t *base, uint32_t row, uint32_t pitch) {
    return base + static_cast<uint64_t>(row) * pitch;
}

// Starts the copies of a tile: positions whose cache rows are `row` of lanes
// 0 .. 15 (and again 16 .. 31), the first n of them; RH signal heads from h0 on.
template <int D, int DV, int RH>
__device__ __forceinline__ void issue_tile(const Params &p, uint32_t tile, uint32_t row, int n, uint32_t h0, uint32_t g) {
    using T = Tile<D, DV, RH>;
    const uint32_t lane = threadIdx.x & 31, hs = p.hs, hn = p.hn;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {                   // K codes: D / 32 chunks a row
        const uint32_t pos = lane / (D / 32) + i * (1024 / D), ch = lane % (D / 32);
        const uint32_t r = __shfl_sync(0xffffffffu, row, pos);
        const uint8_t *s1 = row_at(p.k1c, r, hs * T::KC) + (h0 * T::KC + ch * 16);
        const uint8_t *s2 = row_at(p.k2c, r, hn * T::KC) + (g * T::KC + ch * 16);
        const uint32_t dst = tile + T::k_codes + pos * T::KC + ch * 16;
        const bool ok = static_cast<int>(pos) < n;
#pragma unroll
        for (int j = 0; j < RH; ++j) copy_async<16>(dst + j * kTile * T::KC, s1 + j * T::KC, ok);
        copy_async<16>(dst + RH * kTile * T::KC, s2, ok);
    }
#pragma unroll
    for (int i = 0; i < DV / 64; ++i) {                  // V codes: DV / 32 chunks a row
        const uint32_t pos = lane / (DV / 32) + i * (1024 / DV), ch = lane % (DV / 32);
        const uint32_t r = __shfl_sync(0xffffffffu, row, pos);
        const uint8_t *s = row_at(p.vc, r, hs * T::VC) + (h0 * T::VC + ch * 16);
        const uint32_t vr = v_row(pos), dst = tile + T::v_codes + vr * T::VC + v_chunk<DV>(vr, ch) * 16;
        const bool ok = static_cast<int>(pos) < n;
#pragma unroll
        for (int j = 0; j < RH; ++j) copy_async<16>(dst + j * kTile * T::VC, s + j * T::VC, ok);
    }
    // scales: lanes 0 .. 15 take the first half of the heads, the others the rest
    constexpr int KH = (T::NH + 1) / 2, VH = (RH + 1) / 2;
    const uint32_t pos = lane & 15, upper = lane >> 4;
    const bool ok = static_cast<int>(pos) < n;
    const uint8_t *k1 = row_at(p.k1b, row, hs * T::KS) + (h0 + upper * KH) * T::KS;
    const uint8_t *k2 = row_at(p.k2b, row, hn * T::KS) + g * T::KS;
    const uint8_t *v = row_at(p.vb, row, hs * T::VS) + (h0 + upper * VH) * T::VS;
    const uint32_t kd = tile + T::k_scales + (upper * KH * kTile + pos) * T::KS;
    const uint32_t vd = tile + T::v_scales + (upper * VH * kTile + pos) * T::VS;
#pragma unroll
    for (int i = 0; i < KH; ++i) {
        // the upper lanes' last head is the noise head (or none, where NH is odd)
        const bool noise = upper && i + KH == RH;
        const bool some = i + KH <= RH || !upper;
        if (i + KH == RH) copy_async<T::KS>(kd + i * kTile * T::KS, noise ? k2 : k1 + i * T::KS, ok);
        else copy_async<T::KS>(kd + i * kTile * T::KS, k1 + i * T::KS, ok, some);
    }
#pragma unroll
    for (int i = 0; i < VH; ++i)
        copy_async<T::VS>(vd + i * kTile * T::VS, v + i * T::VS, ok, i + VH < RH || !upper);
}

template <typename V>
__device__ __forceinline__ V at(const uint8_t *smem) { return *reinterpret_cast<const V *>(smem); }

// The query rows of the warp's heads as f16 in shared memory, scaled by a
// power of two that brings their largest element to [2^14, 2^15) (f16 then
// holds all of bf16's digits down to 2^-31 of that).  Returns this lane's
// factor from a score head to exp2 units: that of head lane % 4.
template <int D, int RH>
__device__ __forceinline__ float load_queries(const Params &p, uint8_t *dst, int b, int h0, int g) {
    const int lane = threadIdx.x & 31;
    float mine = 0.f, scale[RH + 1];
    uint32_t words[RH + 1][D / 64];                      // all on their way before the first is used
#pragma unroll
    for (int j = 0; j <= RH; ++j) {
        const __nv_bfloat16 *q = j == RH ? p.q2 + (static_cast<size_t>(b) * p.hn + g) * D
                                         : p.q1 + (static_cast<size_t>(b) * p.hs + h0 + j) * D;
        scale[j] = j == RH ? p.k2_scale[g] : p.k1_scale[h0 + j];
#pragma unroll
        for (int i = 0; i < D / 64; ++i) words[j][i] = reinterpret_cast<const uint32_t *>(q)[lane + 32 * i];
    }
#pragma unroll
    for (int j = 0; j <= RH; ++j) {
        const uint32_t(&w)[D / 64] = words[j];
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) most = max(most, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
        most = __reduce_max_sync(0xffffffffu, most);
        const int up = min(268 - static_cast<int>(most >> 7), 253);       // biased exponent of the factor (254 has no inverse)
        const float f = __uint_as_float(static_cast<uint32_t>(up) << 23);
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
            reinterpret_cast<uint32_t *>(dst + j * D * 2)[lane + 32 * i] =
                pack_half2(bf16_lo(w[i]) * f, bf16_hi(w[i]) * f);
        const float back = __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
        if ((lane & 3) == j) mine = p.scale_log2 * scale[j] * back;
    }
    return mine;
}

// Sum over the blocks of head t's score, on lane t of a quad: lane t holds x[j] = the share of blocks 2t, 2t + 1 in
// head j's (D = 64: there are four blocks, and what lanes 2 and 3 hold is not used).
template <int D>
__device__ __forceinline__ float gather(const float (&x)[4], int t) {
    const bool odd = t & 1;
    if constexpr (D == 64) {
        const float a = (odd ? x[1] : x[0]) + __shfl_xor_sync(0xffffffffu, odd ? x[0] : x[1], 1);
        const float b = (odd ? x[3] : x[2]) + __shfl_xor_sync(0xffffffffu, odd ? x[2] : x[3], 1);
        const float c = __shfl_xor_sync(0xffffffffu, b, 2);
        return t < 2 ? a : c;
    } else {
        const float a = (t < 2 ? x[0] : x[2]) + __shfl_xor_sync(0xffffffffu, t < 2 ? x[2] : x[0], 2);
        const float b = (t < 2 ? x[1] : x[3]) + __shfl_xor_sync(0xffffffffu, t < 2 ? x[3] : x[1], 2);
        return (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
    }
}

// One warp: split u / units of the range, unit u % units = (noise head, part of its group).
template <int D, int DV, int RH>
__global__ void __launch_bounds__(kWarpsPerBlock * 32, (Tile<D, DV, RH>::blocks)) gda_decode_fp4_split_kernel(const Params p) {
    using T = Tile<D, DV, RH>;
    constexpr int NH = T::NH, SLABS = DV / 64, S = T::ring;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, quad = lane >> 2, t = lane & 3;
    uint8_t *const ring = smem + (threadIdx.x >> 5) * T::warp_bytes;
    uint8_t *const queries = ring + S * T::bytes, *const zeros = smem + kWarpsPerBlock * T::warp_bytes;
    for (int i = threadIdx.x; i < NH * D / 2; i += kWarpsPerBlock * 32) reinterpret_cast<uint32_t *>(zeros)[i] = 0u;
    __syncthreads();                                     // the only one: from here on every warp is on its own
    const int units = p.hn * p.parts;
    const int u = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
    const int split = u / units, g = (u % units) / p.parts, part = u % p.parts;
    if (split >= p.splits) return;
    // every part is RH heads: the last begins early where they do not divide the group, and leaves what the parts
    // before it have done unwritten
    const int r = p.hs / p.hn, begin = min(part * RH, r - RH), done = part * RH - begin, h0 = g * r + begin;
    Range range;
    if (!range_of(p, split, range)) return;

    if (u % units == 0) note_sequences(p, range, split);
    Cursor use{range.b, 0, 0, static_cast<int>(range.end - range.start)};
    enter(p, use, static_cast<int>(range.start - range.before), length_of(p, range.b));
    Cursor get = use;                                    // the copies' place, ahead of the arithmetic's
    bool more = true;
    uint32_t row = 0;
    int n = 0;
    // the rows of the next tile to copy, and the place behind it
    auto find = [&]() {
        n = min(kTile, get.hi - get.pos);
        row = row_of(p, get.b, get.pos + min(lane & 15, n - 1));
    };
    auto step = [&]() {
        get.pos += kTile;
        if (get.pos < get.hi) return;
        if (get.left > 0) next_sequence(p, get); else more = false;
    };
    find();
    int to = 0, from = 0, ahead = S - 2;                 // places of the ring; tiles to copy before the first is used
    // lane parts of places in shared memory
    const uint8_t *const qa0 = quad == (D == 64 ? t : 2 * t) ? queries + t * (D / 2) : zeros;
    const uint8_t *const qa1 = quad == 2 * t + 1 ? queries + t * (D / 2) + 32 : zeros;   // D = 128: the second block
    const int k_at = T::k_codes + quad * T::KC + t * (D / 8);
    const int ks_at = T::k_scales + quad * T::KS + (D == 64 ? t & 1 : t) * 2;

    float acc[RH][SLABS][2][4];                          // [u]: of tile 2 u + t / 2 and map t % 2, see values_of
    float m = -INFINITY, l = 0.f;                        // of head t (both its lanes' positions; l of this lane's only)
    float factor = load_queries<D, RH>(p, queries, use.b, h0, g);
#pragma unroll
    for (int j = 0; j < RH; ++j)
#pragma unroll
        for (int s = 0; s < SLABS; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[j][s][i][k] = 0.f;

    // of head t in the tile whose values are added next, as pairs of positions 8 apart: the upper parts of positions
    // quad & 6 and the next on a lane of an even quad, the lower parts of the same two on a lane of an odd one
    uint32_t weights[2] = {0u, 0u};
    float scale = 1.f;                                   // of what was added before them
    auto scores_of = [&](const uint8_t *const tile, uint32_t (&next)[2]) {
        // lane (quad, t) ends up with positions quad, quad + 8 of head t
        float x0[4] = {}, x1[4] = {};
#pragma unroll
        for (int j = 0; j < NH; ++j) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            const uint8_t *ka = tile + k_at + j * kTile * T::KC, *sa = tile + ks_at + j * kTile * T::KS;
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {  // 16 dims of this lane: a block
                const uint8_t *qa = (half ? qa1 : qa0) + j * D * 2;
                const uint4 b0 = at<uint4>(qa), b1 = at<uint4>(qa + 16);
                const uint2 lo = at<uint2>(ka + half * 8), hi = at<uint2>(ka + 8 * T::KC + half * 8);
                uint32_t a0[4], a1[4];
                e2m1x8_to_half2x4(a0, lo.x);
                e2m1x8_to_half2x4(a1, hi.x);
                mma_16816(c, a0[0], a1[0], a0[1], a1[1], b0.x, b0.y, c);
                mma_16816(c, a0[2], a1[2], a0[3], a1[3], b0.z, b0.w, c);
                e2m1x8_to_half2x4(a0, lo.y);
                e2m1x8_to_half2x4(a1, hi.y);
                mma_16816(c, a0[0], a1[0], a0[1], a1[1], b1.x, b1.y, c);
                mma_16816(c, a0[2], a1[2], a0[3], a1[3], b1.z, b1.w, c);
            }
            // columns 2t, 2t + 1 are blocks 2t, 2t + 1 (at D = 64 there are four: lanes 2, 3 hold nothing of use)
            const float2 s0 = half2_bits_to_float2(e4m3x2_to_half2(at<uint16_t>(sa)));
            const float2 s1 = half2_bits_to_float2(e4m3x2_to_half2(at<uint16_t>(sa + 8 * T::KS)));
            x0[j] = fmaf(c[1], s0.y, c[0] * s0.x);
            x1[j] = fmaf(c[3], s1.y, c[2] * s1.x);
        }
        const int have = use.hi - use.pos;               // positions of the tile, if below 16
        float sc0 = gather<D>(x0, t) * factor, sc1 = gather<D>(x1, t) * factor;
        if (quad >= have) sc0 = -INFINITY;
        if (quad + 8 >= have) sc1 = -INFINITY;
        float mt = max3f(m, sc0, sc1);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        scale = fast_exp2(m - mt);                       // m = -inf gives 0
        const float p0 = fast_exp2(sc0 - mt + kWeightBits), p1 = fast_exp2(sc1 - mt + kWeightBits);
        m = mt;
        l = fmaf(l, scale, p0 + p1);
        const uint32_t hi = pack_half2(p0, p1);
        const float2 h = half2_bits_to_float2(hi);
        const uint32_t lo = pack_half2(p0 - h.x, p1 - h.y), got = __shfl_xor_sync(0xffffffffu, quad & 1 ? hi : lo, 4);
        next[0] = quad & 1 ? got : hi;
        next[1] = quad & 1 ? lo : got;
    };
    auto rescale = [&]() {
        if (__any_sync(0xffffffffu, scale != 1.f)) {
#pragma unroll
            for (int j = 0; j < RH; ++j) {
                const float sj = __shfl_sync(0xffffffffu, scale, t & 1 ? RH : j);
#pragma unroll
                for (int s = 0; s < SLABS; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[j][s][i][k] *= sj;
            }
        }
    };
    auto values_of = [&](const uint8_t *const tile) {
        // k slots (2t, 2t + 1) are positions 2t, 2t + 8 and (2t + 8, 2t + 9) are 2t + 1, 2t + 9;
        // row `quad` of tile i is dim 8 quad + 2 i, row quad + 8 the next; columns 4 (i % 2) + 2 map and the next take the
        // upper and the lower part of that map's weights, the other four are zero, so that tiles 2 u and 2 u + 1 share
        // their accumulators
        const uint32_t pick = 0x40u + 0x11u * (quad >> 1);   // byte of block quad / 2 from either word
#pragma unroll
        for (int j = 0; j < RH; ++j) {
            const int src = 8 * t + 4 * (quad & 1) + (quad & 2 ? RH : j);
            const uint32_t w0 = __shfl_sync(0xffffffffu, weights[0], src), w1 = __shfl_sync(0xffffffffu, weights[1], src);
            const uint32_t b0[2] = {quad < 4 ? w0 : 0u, quad < 4 ? 0u : w0}, b1[2] = {quad < 4 ? w1 : 0u, quad < 4 ? 0u : w1};
            // scales of positions 2t, 2t + 1 and 2t + 8, 2t + 9: four blocks to a word
            const uint8_t *vs = tile + T::v_scales + (j * kTile + 2 * t) * T::VS;
            uint32_t e[4][SLABS];                        // [2t, 2t + 8, 2t + 1, 2t + 9][slab]
            if constexpr (DV == 64) {
                const uint2 u = at<uint2>(vs), v = at<uint2>(vs + 8 * T::VS);
                e[0][0] = u.x, e[2][0] = u.y, e[1][0] = v.x, e[3][0] = v.y;
            } else if constexpr (DV == 128) {
                const uint4 u = at<uint4>(vs), v = at<uint4>(vs + 8 * T::VS);
                e[0][0] = u.x, e[0][1] = u.y, e[2][0] = u.z, e[2][1] = u.w;
                e[1][0] = v.x, e[1][1] = v.y, e[3][0] = v.z, e[3][1] = v.w;
            } else {
                const int at_pos[4] = {0, 8, 1, 9};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 u = at<uint4>(vs + at_pos[k] * T::VS);
                    e[k][0] = u.x, e[k][1] = u.y, e[k][2] = u.z, e[k][3] = u.w;
                }
            }
            // codes of 8 dims of slab 0 in row t of the tile; slab s has bits 5, 6 of the place turned over
            const uint32_t lane_at = t * T::VC + (v_chunk<DV>(t, 0) + (quad >> 2)) * 16 + (quad & 3) * 4;
            const uint8_t *vc = tile + T::v_codes + j * kTile * T::VC;
#pragma unroll
            for (int s = 0; s < SLABS; ++s) {
                const uint32_t e0 = e4m3x2_to_half2(prmt(e[0][s], e[1][s], pick));
                const uint32_t e1 = e4m3x2_to_half2(prmt(e[2][s], e[3][s], pick));
                const uint8_t *row = vc + (lane_at ^ (32 * s));
                const uint32_t p0w = at<uint32_t>(row), p8w = at<uint32_t>(row + 4 * T::VC),
                               p1w = at<uint32_t>(row + 8 * T::VC), p9w = at<uint32_t>(row + 12 * T::VC);
                uint32_t a0[4], a1[4], a2[4], a3[4];
                // two positions' codes of one dim side by side in a byte: even dims, odd dims
                e2m1x8_to_half2x4(a0, (p0w & 0x0f0f0f0fu) | ((p8w << 4) & 0xf0f0f0f0u));
                e2m1x8_to_half2x4(a1, ((p0w >> 4) & 0x0f0f0f0fu) | (p8w & 0xf0f0f0f0u));
                e2m1x8_to_half2x4(a2, (p1w & 0x0f0f0f0fu) | ((p9w << 4) & 0xf0f0f0f0u));
                e2m1x8_to_half2x4(a3, ((p1w >> 4) & 0x0f0f0f0fu) | (p9w & 0xf0f0f0f0u));
#pragma unroll
                for (int k = 0; k < 4; ++k) {            // tiles 0, 2, 1, 3: the two that share accumulators are apart
                    const int i = 2 * (k & 1) + (k >> 1);
                    mma_16816(acc[j][s][i / 2], half2_mul(a0[i], e0), half2_mul(a1[i], e0), half2_mul(a2[i], e1),
                              half2_mul(a3[i], e1), b0[i % 2], b1[i % 2], acc[j][s][i / 2]);
                }
            }
        }
    };
    // The scores of a tile come with the values of the one before it, in one run of instructions without a branch: the
    // chain from scores to weights then has other work beside it (64 sequences, split kernel, weights of one f16: 114 -> 108 us).
    const uint8_t *before = ring;                        // the tile whose values are still to be added
    bool fresh = true;                                   // there is none: a part begins
    for (;;) {
        __syncwarp();                                    // the readers of place `to` are done
        if (more) {
            issue_tile<D, DV, RH>(p, smem_u32(ring) + to * T::bytes, row, n, h0, g);
            step();
            if (more) find();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        to = to + 1 == S ? 0 : to + 1;
        if (ahead > 0) {
            --ahead;
            continue;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncwarp();                                    // every lane's copies of this tile have landed
        const uint8_t *const tile = ring + from * T::bytes;
        from = from + 1 == S ? 0 : from + 1;
        uint32_t next[2];
        if (fresh) {
            scores_of(tile, next);
            fresh = false;
        } else {                                         // twice, so that these two are not parted by the test
            scores_of(tile, next);
            values_of(before);
            rescale();
        }
        weights[0] = next[0], weights[1] = next[1];
        before = tile;
        use.pos += kTile;
        if (use.pos < use.hi) continue;
        values_of(before);
        fresh = true;

        // ---- end of the part that lies in sequence use.b
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        const float mn = __shfl_sync(0xffffffffu, m, RH), ln = __shfl_sync(0xffffffffu, l, RH);
        const size_t slot = static_cast<size_t>(split) + use.b;
#pragma unroll
        for (int j = 0; j < RH; ++j) {
            if (j < done) continue;
            const float mj = __shfl_sync(0xffffffffu, m, j), lj = __shfl_sync(0xffffffffu, l, j);
            const size_t place = slot * p.hs + h0 + j;
            if (lane == 0) reinterpret_cast<float4 *>(p.ws_ml)[place] = make_float4(mj, lj, mn, ln);
            const float v = p.v_scale[h0 + j];
            float2 *o = reinterpret_cast<float2 *>(p.ws_o + (place * 2 + (t & 1)) * DV) + 4 * quad + (t >> 1);
#pragma unroll
            for (int s = 0; s < SLABS; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float(&c)[4] = acc[j][s][i];
                    o[32 * s + 2 * i] = make_float2((c[0] + c[1]) * v, (c[2] + c[3]) * v);
                }
        }
        if (use.left == 0) return;
        next_sequence(p, use);
        m = -INFINITY, l = 0.f;
        __syncwarp();                                    // the queries' last readers are done
        factor = load_queries<D, RH>(p, queries, use.b, h0, g);
#pragma unroll
        for (int j = 0; j < RH; ++j)
#pragma unroll
            for (int s = 0; s < SLABS; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[j][s][i][k] = 0.f;
    }
}

template <int D, int DV, int RH>
cudaError_t launch_split(const Params &p, cudaStream_t stream) {
    using T = Tile<D, DV, RH>;
    auto kern = gda_decode_fp4_split_kernel<D, DV, RH>;
    const int smem = T::warp_bytes * kWarpsPerBlock + T::queries;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int warps = p.splits * p.hn * p.parts;
    kern<<<(warps + kWarpsPerBlock - 1) / kWarpsPerBlock, kWarpsPerBlock * 32, smem, stream>>>(p);
    return cudaGetLastError();
}

template <int D, int DV>
cudaError_t launch_split(const Params &p, int rh, cudaStream_t stream) {
    if (rh == 1) return launch_split<D, DV, 1>(p, stream);
    if constexpr (DV < 256)
        if (rh == 3) return launch_split<D, DV, 3>(p, stream);
    return launch_split<D, DV, 2>(p, stream);
}

}  // namespace

size_t decode_fp4_workspace_bytes(int B, int hs, int hn, int d, int dv) {
    return plan_of(B, hs, hn, d, dv).bytes;
}

int launch_decode_fp4(const DecodeFp4Args &a, cudaStream_t stream) {
    const Fp4Plan pl = plan_of(a.B, a.hs, a.hn, a.d, a.dv);
    char *ws = static_cast<char *>(a.workspace);
    const Params p{static_cast<const __nv_bfloat16 *>(a.q1),
                   static_cast<const __nv_bfloat16 *>(a.q2),
                   a.k1c, a.k2c, a.vc, a.k1b, a.k2b, a.vb, a.k1_scale, a.k2_scale, a.v_scale, a.lens, a.lambda,
                   static_cast<__nv_bfloat16 *>(a.out),
                   reinterpret_cast<float *>(ws),
                   reinterpret_cast<float *>(ws + pl.ml_at),
                   reinterpret_cast<int *>(ws + pl.seg_at),
                   a.dev_err, a.lambda_init, a.eps,
                   static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a.d))),
                   a.B, a.Lcap, a.hs, a.hn, pl.splits, pl.heads.parts, a.block_table, a.page_size, a.max_pages,
                   a.num_pages};
    cudaError_t e = cudaErrorInvalidValue;
    switch (a.d * 1000 + a.dv) {
        case 64064: e = launch_split<64, 64>(p, pl.heads.each, stream); break;
        case 64128: e = launch_split<64, 128>(p, pl.heads.each, stream); break;
        case 64256: e = launch_split<64, 256>(p, pl.heads.each, stream); break;
        case 128064: e = launch_split<128, 64>(p, pl.heads.each, stream); break;
        case 128128: e = launch_split<128, 128>(p, pl.heads.each, stream); break;
        case 128256: e = launch_split<128, 256>(p, pl.heads.each, stream); break;
        default: return GDA_ERR_UNSUPPORTED;
    }
    if (e != cudaSuccess) return record_cuda_error(e);
    e = a.dv == 64    ? launch_join<64>(p, stream)
        : a.dv == 128 ? launch_join<128>(p, stream)
                      : launch_join<256>(p, stream);
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

}  // namespace gda
