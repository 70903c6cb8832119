// The blocks of tokens that a query is to attend, by a cheap score over the
// bounds that gda_cache_append_fp8_block keeps of every block's keys.
//
// For head h with query q, q8 = rint(q * (127 * (1 / amax))), amax = max |q|; a block
// b whose keys lie between lo and hi in every channel has, whatever its keys,
// a dot product of at most
//   ub_h(b) = sum over channels of q8 * hi where q8 > 0, of q8 * lo where q8 < 0
// (a whole number), and x_h(b) = ub * scale_h(b) * amax is that bound on the
// logit up to one factor for all heads.  With t = (x_h(b) - max x_h) * 4 / (127
// ln 2 sqrt d) and w = 2^floor(t) (1 + t - floor(t)), 2^t with straight lines
// between the powers, block b has the share w / sum of w of head h if every
// block is as good as its bound.  A block counts as much as for the head of the
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

// Blocks of tokens that a warp scores.  us of both kernels with 8 / 16 / 32, cold: 64 sequences of 64 to 128 blocks, 12 +
// 4 heads 22.7 / 23.7 / 27.8; one of 2048, 24 + 8 heads 28.8 / 31.9 / 35.0.
constexpr int kChunk = 8;
constexpr int kScoreWarps = 4;

// Bytes of four whole numbers.
__device__ __forceinline__ uint32_t bytes_of(const int (&v)[4]) {
    return (static_cast<uint32_t>(v[0]) & 0xffu) | (static_cast<uint32_t>(v[1]) & 0xffu) << 8 |
           (static_cast<uint32_t>(v[2]) & 0xffu) << 16 | static_cast<uint32_t>(v[3]) << 24;
}

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
    const bool noise = unit >= sig, upper = sub < LANES / 2;
    const int heads = noise ? a.hn : a.hs, mine = (noise ? unit - sig : unit) * HEADS + lane / LANES;
    const int h = min(mine, heads - 1);
    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(noise ? a.q2 : a.q1) +
                                                     (static_cast<size_t>(b) * heads + h) * D + sub % (LANES / 2) * 16);
    const uint4 q0 = q[0], q1 = q[1];
    const uint8_t *bounds = reinterpret_cast<const uint8_t *>(noise ? a.k2b : a.k1b) + h * 2 * D + sub * 16;
    const float *scales = (noise ? a.k2s : a.k1s) + h;
    const size_t pitch = static_cast<size_t>(heads) * 2 * D;

    const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
    uint32_t top = 0;                                        // magnitudes of bf16 order like their bits
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, max(w[k] << 16 & 0x7fff0000u, w[k] & 0x7fff0000u));
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float amax = __uint_as_float(top);
    const bool ok = top < 0x7f800000u && amax >= 0x1p-100f;
    const float r = ok ? __fmul_rn(127.f, __frcp_rn(amax)) : 0.f;   // q / amax is often k + 1/2: each rounding counts
    uint32_t part[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        int v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t pair = w[2 * k + i / 2];
            const int c = ok ? __float2int_rn(__fmul_rn(i & 1 ? bf16_hi(pair) : bf16_lo(pair), r)) : 0;
            v[i] = upper ? max(c, 0) : min(c, 0);
        }
        part[k] = bytes_of(v);
    }
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
            int ub = __dp4a(static_cast<int>(v[k].x), static_cast<int>(part[0]), 0);
            ub = __dp4a(static_cast<int>(v[k].y), static_cast<int>(part[1]), ub);
            ub = __dp4a(static_cast<int>(v[k].z), static_cast<int>(part[2]), ub);
            ub = __dp4a(static_cast<int>(v[k].w), static_cast<int>(part[3]), ub);
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1) ub += __shfl_xor_sync(0xffffffffu, ub, o);
            if (sub == 0 && mine < heads && j + k < j1)
                out[j + k] = ok ? __fmul_rn(__fmul_rn(static_cast<float>(ub), s[k]), amax) + 0.f : -INFINITY;
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

// The place of the k-th highest of a histogram of 256, computed by a whole warp: its bin, and how many are left of k there.
__device__ __forceinline__ uint2 bin_of(const uint32_t *hist, uint32_t k) {
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
    uint32_t bin = 0, left = 0;
    const bool here = above < k && k <= incl;
    if (here) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (left == 0 && above + own[i] >= k) bin = 255 - 8 * lane - i, left = k - above;
            above += own[i];
        }
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    return make_uint2(__shfl_sync(0xffffffffu, bin, src), __shfl_sync(0xffffffffu, left, src));
}

// grid (hn, B): keeps the blocks of one (sequence, noise head).
template <int THREADS>
__global__ void __launch_bounds__(THREADS) gda_block_select_kernel(const BlockSelectArgs a, int most) {
    constexpr int WARPS = THREADS / 32;
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
    for (int i = threadIdx.x + (n <= a.keep ? 0 : kept); i < a.keep; i += THREADS) list[i] = i < kept ? i : -1;
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
            best[i] = m, inverse[i] = m > -INFINITY && m < INFINITY ? __frcp_rn(__fmul_rn(__ull2float_rn(total), 0x1p-40f)) : 0.f;
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += THREADS) {
        float s = 0.f;
#pragma unroll 4
        for (int i = 0; i <= r; ++i) s = fmaxf(s, __fmul_rn(weight(row_of(i)[j], best[i], a.unit), inverse[i]));
        // a share is at least 0 and orders like its bits
        keys[j] = j < a.first || j >= n - a.last ? 0xffffffffu : __float_as_uint(s);
    }
    // the kept-th highest key, eight bits at a time, a histogram to a warp: most keys share their first digits
    uint32_t prefix = 0, need = kept;
    for (int at = 24; at >= 0; at -= 8) {
        for (int i = lane; i < 256; i += 32) hist[warp][i] = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += THREADS) {
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
        const uint2 bin = bin_of(hist[0], need);             // every warp for itself
        prefix |= bin.x << at, need = bin.y;
        __syncthreads();
    }
    // all keys above it, and the first `need` equal to it, in order
    const int per = (n + THREADS - 1) / THREADS, j0 = min(n, static_cast<int>(threadIdx.x) * per), j1 = min(n, j0 + per);
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

template <int THREADS>
cudaError_t launch_select(const BlockSelectArgs &a, int most, cudaStream_t stream) {
    const cudaError_t e = allow_shared_memory<gda_block_select_kernel<THREADS>>(kBlockSelectMaxBlocks * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.hn, a.B);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = most * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gda_block_select_kernel<THREADS>, a, most);
}

}  // namespace

int launch_block_select(const BlockSelectArgs &a, cudaStream_t stream) {
    const int most = a.max_pages * (a.page_size / a.block), heads = a.d == 64 ? 4 : 2;
    const int warps = ((a.hs + heads - 1) / heads + (a.hn + heads - 1) / heads) * ((most + kChunk - 1) / kChunk);
    const dim3 grid((warps + kScoreWarps - 1) / kScoreWarps, a.B);
    if (a.d == 64) gda_block_score_kernel<64><<<grid, kScoreWarps * 32, 0, stream>>>(a, most);
    else gda_block_score_kernel<128><<<grid, kScoreWarps * 32, 0, stream>>>(a, most);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return record_cuda_error(e);
    // 2048 blocks, us of both kernels, cold: 31.9 with 1024 threads, 27.8 with 512 or 256
    e = most > 512 ? launch_select<512>(a, most, stream) : launch_select<256>(a, most, stream);
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

}  // namespace gda
