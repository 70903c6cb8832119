// The blocks of tokens that a query is to attend, by a cheap score over the
// bounds that gda_cache_append_fp8_block keeps of every block's keys.
//
// For head h with query q, q8 = rint(q * (127 * (1 / amax))), amax = max |q|; a block
// b whose keys lie between lo and hi in every channel has, whatever its keys,
// a dot product of at most
//   ub_h(b) = sum over channels of q8 * hi where q8 > 0, of q8 * lo where q8 < 0
// (a whole number), and x_h(b) = ub * scale_h(b) * amax that bound in the units of
// a logit, up to one factor for all heads.  It bounds the products with q8: a
// channel of q below amax / 254 is 0 there, and where a block's keys are large
// in such channels its logits may be above it.  With t = (x_h(b) - max x_h) * 4 / (127
// ln 2 sqrt d) and w = 2^floor(t) (1 + t - floor(t)), 2^t with straight lines
// between the powers, block b has the share w / sum of w of head h if every
// block is as good as its x.  A block counts as much as for the head of the
// group (the signal heads that share a noise head, and that) that wants it
// most: the score is the largest share.  (The bounds themselves cannot be
// compared between heads: one whose logits are flat would outweigh one that
// attends to few blocks.)  A head whose amax is below 2^-100 or not finite, or
// whose largest x is past float32, takes no part.  Kept are the first and last blocks that the caller names, then the
// highest scores, of equal ones the lowest index.  The sums are over whole
// numbers, w in units of 2^-40, and the roundings have one order, so the choice
// is the same everywhere.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "gda.h"
#include "gda_device.cuh"
#include "gda_internal.h"

namespace gda {
namespace {

__device__ __forceinline__ int length_of(const BlockSelectArgs &a, int b) {
    const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
    const int len = a.lens[b];
    if (len >= 0 && len <= cap) return len;
    atomicOr(a.dev_err, GDA_DEVERR_BAD_LENGTH);
    return len < 0 ? 0 : static_cast<int>(cap);
}

// Index of block j of sequence b among the blocks of the pools.  A page outside the pool is read as page 0 and reported.
__device__ __forceinline__ size_t pool_block(const BlockSelectArgs &a, int b, int j) {
    const int per = a.page_size / a.block, pg = j / per;
    int phys = b;
    if (a.block_table != nullptr) {
        phys = a.block_table[static_cast<size_t>(b) * a.max_pages + pg];
        if (phys < 0 || phys >= a.num_pages) {
            atomicOr(a.dev_err, GDA_DEVERR_BAD_PAGE);
            phys = 0;
        }
    }
    return static_cast<size_t>(phys) * per + (j - pg * per);
}

// Blocks of tokens that a warp scores, in the two launches.  us of both with 8 / 16 / 32, in graphs: one sequence of 32768
// blocks, 3 + 1 heads of 64 138.8 / 137.9 / 138.2, 24 + 8 heads 164 / 161 / 157; four, 12 + 4 heads 199 / 192 / 191; one of
// 16384, 48 + 2 heads of 128 389 / 381 / 377.
constexpr int kChunk = 16;
constexpr int kScoreWarps = 4;
constexpr int kThreads = 512;          // of a block that selects

// Bytes of four whole numbers.
__device__ __forceinline__ uint32_t bytes_of(const int (&v)[4]) {
    return (static_cast<uint32_t>(v[0]) & 0xffu) | (static_cast<uint32_t>(v[1]) & 0xffu) << 8 |
           (static_cast<uint32_t>(v[2]) & 0xffu) << 16 | static_cast<uint32_t>(v[3]) << 24;
}

// Of a query row: its largest magnitude, and q8 of 16 channels as the lane `sub` of LANES needs it: the positive parts
// (the first half of the lanes) or the negative ones.
template <int LANES>
struct QueryPart {
    float amax;
    bool ok;
    uint32_t w[4];

    __device__ __forceinline__ QueryPart(const uint4 *row, int sub) {
        const uint4 q0 = row[sub % (LANES / 2) * 2], q1 = row[sub % (LANES / 2) * 2 + 1];
        const uint32_t v[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        uint32_t top = 0;                                    // magnitudes of bf16 order like their bits
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, max(v[k] << 16 & 0x7fff0000u, v[k] & 0x7fff0000u));
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        amax = __uint_as_float(top);
        ok = top < 0x7f800000u && amax >= 0x1p-100f;
        const float r = ok ? __fmul_rn(127.f, __frcp_rn(amax)) : 0.f;   // q / amax is often k + 1/2: each rounding counts
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            int c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t pair = v[2 * k + i / 2];
                c[i] = ok ? __float2int_rn(__fmul_rn(i & 1 ? bf16_hi(pair) : bf16_lo(pair), r)) : 0;
                c[i] = sub < LANES / 2 ? max(c[i], 0) : min(c[i], 0);
            }
            w[k] = bytes_of(c);
        }
    }
};

// x of kChunk blocks for as many heads as a warp's lanes hold bounds of, 16 bytes each: a lane has the greatest or the
// least of 16 channels, and the positive or the negative parts of q8 there.
template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32) gda_block_score_kernel(const BlockSelectArgs a, int most) {
    constexpr int LANES = D / 8, HEADS = 32 / LANES;         // lanes of a head's bounds, heads of a warp
    const int b = blockIdx.y, lane = threadIdx.x & 31, sub = lane % LANES;
    const int sig = (a.hs + HEADS - 1) / HEADS, units = sig + (a.hn + HEADS - 1) / HEADS;
    const int u = blockIdx.x * kScoreWarps + (threadIdx.x >> 5), unit = u % units, j0 = u / units * kChunk;
    const int n = (length_of(a, b) + a.block - 1) / a.block;
    if (n <= a.keep || j0 >= n) return;
    const bool noise = unit >= sig;
    const int heads = noise ? a.hn : a.hs, mine = (noise ? unit - sig : unit) * HEADS + lane / LANES;
    const int h = min(mine, heads - 1);
    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(noise ? a.q2 : a.q1) +
                                                     (static_cast<size_t>(b) * heads + h) * D);
    const QueryPart<LANES> part8(q, sub);
    const uint8_t *bounds = reinterpret_cast<const uint8_t *>(noise ? a.k2b : a.k1b) + h * 2 * D + sub * 16;
    const float *scales = (noise ? a.k2s : a.k1s) + h;
    const size_t pitch = static_cast<size_t>(heads) * 2 * D;

    float *out = a.scores + (static_cast<size_t>(b) * (a.hs + a.hn) + (noise ? a.hs + h : h)) * most;
    const int j1 = min(n, j0 + kChunk);
#pragma unroll 1
    for (int j = j0; j < j1; j += 4) {
        uint4 v[4];
        float s[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {                        // (the last one again where there are fewer)
            const size_t at = pool_block(a, b, min(j + k, j1 - 1));
            v[k] = *reinterpret_cast<const uint4 *>(bounds + at * pitch);
            s[k] = scales[at * heads];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            int ub = __dp4a(static_cast<int>(v[k].x), static_cast<int>(part8.w[0]), 0);
            ub = __dp4a(static_cast<int>(v[k].y), static_cast<int>(part8.w[1]), ub);
            ub = __dp4a(static_cast<int>(v[k].z), static_cast<int>(part8.w[2]), ub);
            ub = __dp4a(static_cast<int>(v[k].w), static_cast<int>(part8.w[3]), ub);
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1) ub += __shfl_xor_sync(0xffffffffu, ub, o);
            if (sub == 0 && mine < heads && j + k < j1)
                out[j + k] = part8.ok ? __fmul_rn(__fmul_rn(static_cast<float>(ub), s[k]), part8.amax) + 0.f : -INFINITY;
        }
    }
}

// 2^t, straight lines between whole t, for t = (x - most) * unit <= 0; at least 2^-126.
__device__ __forceinline__ float weight(float x, float most, float unit) {
    const float t = fmaxf(__fmul_rn(__fsub_rn(x, most), unit), -126.f), e = floorf(t);
    const int line = __float2int_rn(__fmul_rn(__fsub_rn(t, e), 0x1p23f));
    return __int_as_float(((static_cast<int>(e) + 127) << 23) + line);
}

// In whole units of 2^-40.
__device__ __forceinline__ unsigned long long units(float w) { return __float2ull_rz(w * 0x1p40f); }

// 1 / the sum of w, from the largest x of a head and that sum in units; 0 for a head without a part.
__device__ __forceinline__ float inverse_of(float most, unsigned long long sum) {
    return most > -INFINITY && most < INFINITY ? __frcp_rn(__fmul_rn(__ull2float_rn(sum), 0x1p-40f)) : 0.f;
}

// Block j's key: its share, which is at least 0 and orders like its bits.
__device__ __forceinline__ uint32_t key_of(const BlockSelectArgs &a, float share, int j, int n) {
    return j < a.first || j >= n - a.last ? 0xffffffffu : __float_as_uint(share);
}

// The place of the k-th highest of a histogram of 256, computed by a whole warp: its bin, how many are left of k there,
// and how many there are.
__device__ __forceinline__ uint3 bin_of(const uint32_t *hist, uint32_t k) {
    const int lane = threadIdx.x & 31;
    uint32_t own[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += own[i] = hist[255 - 8 * lane - i];    // from the top
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    uint32_t above = incl - sum;
    uint32_t bin = 0, left = 0, count = 0;
    const bool here = above < k && k <= incl;
    if (here) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (left == 0 && above + own[i] >= k) bin = 255 - 8 * lane - i, left = k - above, count = own[i];
            above += own[i];
        }
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    return make_uint3(__shfl_sync(0xffffffffu, bin, src), __shfl_sync(0xffffffffu, left, src),
                      __shfl_sync(0xffffffffu, count, src));
}

constexpr int kCountKeys = 256;        // at most the threads of a block

// The indices of the `kept` < n highest of n keys in shared memory, of equal ones the lowest, ascending; a whole block.
__device__ __forceinline__ void list_highest(const uint32_t *keys, int n, int kept, int *list, uint32_t (&hist)[kThreads / 32][256],
                                             uint2 (&sums)[kThreads / 32]) {
    constexpr int WARPS = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (n <= kCountKeys) {                                   // few: EACH lanes to a key count those ahead of it
        constexpr int EACH = kThreads / kCountKeys;
        const int j = threadIdx.x / EACH;
        uint32_t lanes = 0;
        if (warp * (32 / EACH) < n) {
            const uint32_t own = keys[min(j, n - 1)];
            int ahead = 0;
#pragma unroll 8
            for (int i = lane % EACH; i < n; i += EACH) {
                const uint32_t k = keys[i];
                ahead += k > own || (k == own && i < j);
            }
#pragma unroll
            for (int o = 1; o < EACH; o <<= 1) ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
            lanes = __ballot_sync(0xffffffffu, j < n && ahead < kept && lane % EACH == 0);
            if (lane == 0) sums[warp].x = __popc(lanes);
        }
        __syncthreads();
        if (lanes >> lane & 1u) {
            int at = __popc(lanes & ((1u << lane) - 1));
            for (int w = 0; w < warp; ++w) at += sums[w].x;
            list[at] = j;
        }
        return;
    }
    // the kept-th highest key, eight bits at a time, a histogram to a warp: most keys share their first digits
    uint32_t prefix = 0, need = kept;
    for (int at = 24; at >= 0; at -= 8) {
        for (int i = lane; i < 256; i += 32) hist[warp][i] = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += kThreads) {
            const uint32_t k = keys[j];
            if (at == 24 || k >> (at + 8) == prefix >> (at + 8)) atomicAdd(&hist[warp][k >> at & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x < 256) {
            uint32_t sum = 0;
#pragma unroll 8
            for (int w = 0; w < WARPS; ++w) sum += hist[w][threadIdx.x];
            hist[0][threadIdx.x] = sum;
        }
        __syncthreads();
        const uint3 bin = bin_of(hist[0], need);             // every warp for itself
        prefix |= bin.x << at, need = bin.y;
        __syncthreads();
        if (bin.y == bin.z) {                                // all that begin like it: what is above the least of those
            --prefix, need = 0;                              // (there are n > kept keys, so it is not 0)
            break;
        }
    }
    // all keys above it, and the first `need` equal to it, in order
    const int per = (n + kThreads - 1) / kThreads, j0 = min(n, static_cast<int>(threadIdx.x) * per), j1 = min(n, j0 + per);
    uint2 mine = make_uint2(0u, 0u);
    for (int j = j0; j < j1; ++j) mine.x += keys[j] > prefix, mine.y += keys[j] == prefix;
    uint2 incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t p = __shfl_up_sync(0xffffffffu, incl.x, o), q = __shfl_up_sync(0xffffffffu, incl.y, o);
        if (lane >= o) incl.x += p, incl.y += q;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    uint32_t gt = incl.x - mine.x, eq = incl.y - mine.y;
    for (int w = 0; w < warp; ++w) gt += sums[w].x, eq += sums[w].y;
    for (int j = j0; j < j1; ++j) {
        if (keys[j] > prefix) list[gt++ + min(eq, need)] = j;
        else if (keys[j] == prefix && eq++ < need) list[gt + eq - 1] = j;
    }
}

// grid (hn, B): keeps the blocks of one (sequence, noise head).
__global__ void __launch_bounds__(kThreads) gda_block_select_kernel(const BlockSelectArgs a, int most) {
    constexpr int WARPS = kThreads / 32;
    extern __shared__ uint32_t keys[];
    __shared__ float best[128], inverse[128];                // of the heads: the largest x, 1 / the sum of w
    __shared__ float part_most[WARPS];
    __shared__ unsigned long long part_sum[WARPS];
    __shared__ uint32_t hist[WARPS][256];
    __shared__ uint2 sums[WARPS];
    // a programmatic dependent of the scoring kernel: this wait, of every block, returns once its writes are visible
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int g = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = (length_of(a, b) + a.block - 1) / a.block, kept = min(n, a.keep), r = a.hs / a.hn;
    int *list = a.list + (static_cast<size_t>(b) * a.hn + g) * a.keep;
    if (g == 0 && threadIdx.x == 0) a.count[b] = kept;
    for (int i = threadIdx.x + (n <= a.keep ? 0 : kept); i < a.keep; i += kThreads) list[i] = i < kept ? i : -1;
    if (n <= a.keep) return;
    const float *x = a.scores + static_cast<size_t>(b) * (a.hs + a.hn) * most;
    auto row_of = [&](int i) { return x + static_cast<size_t>(i == r ? a.hs + g : g * r + i) * most; };

    // the heads' maxima and sums: `team` warps to a head
    const int team = max(1, WARPS / (r + 1)), teams = WARPS / team, member = warp % team, first = warp / team;
    for (int i0 = 0; i0 <= r; i0 += teams) {                 // the same for all threads
        const int i = i0 + first;
        const bool here = first < teams && i <= r;
        const float *xh = row_of(min(i, r));
        float m = -INFINITY;
        if (here)
#pragma unroll 4
            for (int j = member * 32 + lane; j < n; j += team * 32) m = fmaxf(m, xh[j]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) part_most[warp] = m;
        __syncthreads();
        for (int k = 0; k < team; ++k) m = fmaxf(m, part_most[min(warp - member + k, WARPS - 1)]);
        unsigned long long total = 0;
        if (here)
#pragma unroll 4
            for (int j = member * 32 + lane; j < n; j += team * 32) total += units(weight(xh[j], m, a.unit));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane == 0) part_sum[warp] = total;
        __syncthreads();
        if (here && member == 0 && lane == 0) {
            for (int k = 1; k < team; ++k) total += part_sum[warp + k];
            best[i] = m, inverse[i] = inverse_of(m, total);
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kThreads) {
        float s = 0.f;
#pragma unroll 4
        for (int i = 0; i <= r; ++i) s = fmaxf(s, __fmul_rn(weight(row_of(i)[j], best[i], a.unit), inverse[i]));
        keys[j] = key_of(a, s, j, n);
    }
    __syncthreads();
    list_highest(keys, n, kept, list, hist, sums);
}

cudaError_t launch_select(const BlockSelectArgs &a, int most, cudaStream_t stream) {
    const cudaError_t e = allow_shared_memory<gda_block_select_kernel>(kBlockSelectMaxBlocks * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.hn, a.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = most * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gda_block_select_kernel, a, most);
}

// ---- one launch ----
//
// A cluster of thread blocks to one (sequence, noise head): each scores its part of the sequence's blocks for all heads of
// the group, x stays in shared memory, maxima and sums are exchanged, and the first one selects.  Measured (graph replay):
// 64 sequences of 64 to 128 blocks, 12 + 4 heads of 64, 13 MB 12.5 us (the two launches above 17.9), of which 4.4 an
// empty launch, 4 the bounds and 2 the ranking; one of 2048, 24 + 8 heads, 9 MB 16.6 (20.7), 4 the bounds and 4 the
// search.  It is bound by its chain of short phases, not by the bytes (1.9 and 1.3 us).  256 / 512 threads: 11.9 / 12.5
// and 16.6 / 16.6, but 17.6 / 16.5 and 23.7 / 20.6 with the bounds in HBM.
constexpr int kMaxCluster = 8;
constexpr int kSharedLimit = 200 * 1024;

__host__ __device__ constexpr int part_of(int most, int ranks) { return ((most + ranks - 1) / ranks + 3) / 4 * 4; }
// Shared memory of a thread block, at the longest head dim: q8's parts, places of its blocks, x, keys of all blocks.
__host__ __device__ constexpr long long fused_bytes(int most, int heads, int ranks) {
    return heads * 256LL + 4LL * part_of(most, ranks) * (heads + 1) + 4LL * (most + 3);
}

__device__ __forceinline__ uint32_t remote(const void *p, int rank) {    // that address in another block of the cluster
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int product(uint4 a, uint4 b, int c) {       // of 16 whole numbers each, added to c
    c = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), c);
    c = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), c);
    c = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), c);
    return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), c);
}

template <int D>
__global__ void __launch_bounds__(kThreads) gda_block_select_fused_kernel(const BlockSelectArgs a, int part) {
    constexpr int WARPS = kThreads / 32, LANES = D / 16, PAIRS = 32 / LANES, STEP = WARPS * PAIRS;   // 32 bytes to a lane
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ float amax[128], best[128], own_best[128], inverse[128];
    __shared__ unsigned long long own_sum[128];
    __shared__ uint32_t hist[WARPS][256];
    __shared__ uint2 sums[WARPS];
    asm volatile("griddepcontrol.wait;" ::: "memory");       // a programmatic dependent of whatever is ahead in the stream
    uint32_t rank_, ranks_;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank_));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks_));
    const int rank = static_cast<int>(rank_), ranks = static_cast<int>(ranks_);
    const int g = blockIdx.x / ranks, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LANES;
    const int r = a.hs / a.hn, heads = r + 1;
    uint4 *const parts = reinterpret_cast<uint4 *>(raw);     // [heads][D / 8]
    for (int h = WARPS - 1 - warp; h < heads; h += WARPS) {   // while the first warps look up places
        const uint4 *q = reinterpret_cast<const uint4 *>(
            h == r ? static_cast<const __nv_bfloat16 *>(a.q2) + (static_cast<size_t>(b) * a.hn + g) * D
                   : static_cast<const __nv_bfloat16 *>(a.q1) + (static_cast<size_t>(b) * a.hs + g * r + h) * D);
        const QueryPart<D / 8> part8(q, lane % (D / 8));
        if (lane < D / 8) parts[h * (D / 8) + lane] = make_uint4(part8.w[0], part8.w[1], part8.w[2], part8.w[3]);
        if (lane == 0) amax[h] = part8.ok ? part8.amax : -1.f;
    }
    const int n = (length_of(a, b) + a.block - 1) / a.block, kept = min(n, a.keep);
    int *list = a.list + (static_cast<size_t>(b) * a.hn + g) * a.keep;
    if (rank == 0) {
        if (g == 0 && threadIdx.x == 0) a.count[b] = kept;
        for (int i = threadIdx.x + (n <= a.keep ? 0 : kept); i < a.keep; i += kThreads) list[i] = i < kept ? i : -1;
    }
    if (n <= a.keep) return;                                 // the whole cluster
    const int per = (n + ranks - 1) / ranks, j0 = min(n, rank * per), own = min(n, j0 + per) - j0;   // per <= part
    int *const places = reinterpret_cast<int *>(raw + heads * 256);
    float *const x = reinterpret_cast<float *>(places + part);   // [heads][part]
    uint32_t *const keys = reinterpret_cast<uint32_t *>(x + heads * part);

    for (int j = threadIdx.x; j < own; j += kThreads) places[j] = static_cast<int>(pool_block(a, b, j0 + j));
    __syncthreads();

    // (block, head) pairs, a block's heads side by side as their bounds are
    const int total = own * heads;
    int first = warp * PAIRS, j = (first + lane / LANES) / heads, h = (first + lane / LANES) % heads;
    const int dj = STEP / heads, dh = STEP % heads;
    while (first < total) {
        constexpr int K = 4;
        uint4 v[K], w[K];
        float s[K];
        int to[K], head[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {                        // (the last block again past the end)
            const size_t at = static_cast<size_t>(places[min(j, own - 1)]);
            const bool noise = h == r;
            const size_t place = noise ? at * a.hn + g : at * a.hs + g * r + h;
            const uint4 *bounds = reinterpret_cast<const uint4 *>((noise ? a.k2b : a.k1b) + place * 2 * D) + sub * 2;
            v[k] = bounds[0], w[k] = bounds[1];
            s[k] = (noise ? a.k2s : a.k1s)[place];
            head[k] = h;
            to[k] = j < own ? h * part + j : -1;
            j += dj, h += dh;
            if (h >= heads) h -= heads, ++j;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint4 *q8 = parts + head[k] * (D / 8) + sub * 2;
            int ub = product(v[k], q8[0], 0);
            ub = product(w[k], q8[1], ub);
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1) ub += __shfl_xor_sync(0xffffffffu, ub, o);
            const float top = amax[head[k]];
            if (sub == 0 && to[k] >= 0)
                x[to[k]] = top >= 0.f ? __fmul_rn(__fmul_rn(static_cast<float>(ub), s[k]), top) + 0.f : -INFINITY;
        }
        first += K * STEP;
    }
    __syncthreads();

    for (int i = warp; i < heads; i += WARPS) {              // the same warp for a head's maximum and sum
        float m = -INFINITY;
        for (int k = lane; k < own; k += 32) m = fmaxf(m, x[i * part + k]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) own_best[i] = m;
    }
    if (ranks > 1) cluster_barrier();
    __syncwarp();
    for (int i = warp; i < heads; i += WARPS) {
        float m = own_best[i];
        if (ranks > 1) {
            if (lane < ranks) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(m) : "r"(remote(own_best + i, lane)) : "memory");
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        }
        unsigned long long sum = 0;
        for (int k = lane; k < own; k += 32) sum += units(weight(x[i * part + k], m, a.unit));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) best[i] = m, own_sum[i] = sum;
    }
    if (ranks > 1) cluster_barrier();
    __syncwarp();
    for (int i = warp; i < heads; i += WARPS) {
        unsigned long long sum = own_sum[i];
        if (ranks > 1) {
            if (lane >= ranks) sum = 0;
            else asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(sum) : "r"(remote(own_sum + i, lane)) : "memory");
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        if (lane == 0) inverse[i] = inverse_of(best[i], sum);
    }
    __syncthreads();
    const uint32_t keys_to = remote(keys, 0);
    for (int k = threadIdx.x; k < own; k += kThreads) {
        float s = 0.f;
#pragma unroll 4
        for (int i = 0; i < heads; ++i) s = fmaxf(s, __fmul_rn(weight(x[i * part + k], best[i], a.unit), inverse[i]));
        const uint32_t key = key_of(a, s, j0 + k, n);
        if (rank == 0) keys[k] = key;
        else asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(keys_to + 4 * (j0 + k)), "r"(key) : "memory");
    }
    if (ranks > 1) cluster_barrier();
    else __syncthreads();
    if (rank == 0) list_highest(keys, n, kept, list, hist, sums);
}

// Thread blocks of a cluster: as many as it takes to keep the SMs busy, not fewer than 128 blocks of tokens each, and not
// so few that x does not fit.  0: it does not fit at all.
int cluster_of(int B, int most, int hs, int hn) {
    const int heads = hs / hn + 1;
    int ranks = 1;
    while (ranks < kMaxCluster &&
           (fused_bytes(most, heads, ranks) > kSharedLimit || (static_cast<long long>(B) * hn * ranks < 152 && most > 128 * ranks)))
        ranks *= 2;
    return fused_bytes(most, heads, ranks) <= kSharedLimit ? ranks : 0;
}

template <int D>
cudaError_t launch_fused(const BlockSelectArgs &a, int most, int ranks, cudaStream_t stream) {
    const cudaError_t e = allow_shared_memory<gda_block_select_fused_kernel<D>>(kSharedLimit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.hn * ranks, a.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(fused_bytes(most, a.hs / a.hn + 1, ranks));
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ranks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, gda_block_select_fused_kernel<D>, a, part_of(most, ranks));
}

}  // namespace

size_t block_select_workspace_bytes(int B, int most, int hs, int hn) {
    return cluster_of(B, most, hs, hn) > 0 ? 0 : static_cast<size_t>(B) * most * (hs + hn) * sizeof(float);
}

int launch_block_select(const BlockSelectArgs &a, cudaStream_t stream) {
    const int most = a.max_pages * (a.page_size / a.block), heads = a.d == 64 ? 4 : 2;
    const int warps = ((a.hs + heads - 1) / heads + (a.hn + heads - 1) / heads) * ((most + kChunk - 1) / kChunk);
    if (const int ranks = cluster_of(a.B, most, a.hs, a.hn)) {
        const cudaError_t e = a.d == 64 ? launch_fused<64>(a, most, ranks, stream) : launch_fused<128>(a, most, ranks, stream);
        return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
    }
    const dim3 grid((warps + kScoreWarps - 1) / kScoreWarps, a.B);
    if (a.d == 64) gda_block_score_kernel<64><<<grid, kScoreWarps * 32, 0, stream>>>(a, most);
    else gda_block_score_kernel<128><<<grid, kScoreWarps * 32, 0, stream>>>(a, most);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return record_cuda_error(e);
    e = launch_select(a, most, stream);
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

}  // namespace gda
