// The blocks of tokens that a query is to attend, by a cheap score over the
// bounds that gda_cache_append_fp8_block keeps of every block's keys.
//
// For head h with query q, q8 = rint(q * (127 / amax)), amax = max |q|; a block
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
// attends to few blocks.)  A head whose amax is below 2^-100 or not finite takes
// no part.  Kept are the first and last blocks that the caller names, then the
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

constexpr int kThreads = 256;

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

// grid (chunks of blocks, heads, B): x of one head, a warp to a block.
__global__ void __launch_bounds__(kThreads) gda_block_score_kernel(const BlockSelectArgs a, int most) {
    __shared__ int pos[32], neg[32];                         // q8 by its sign, four channels to a word
    __shared__ float amax_of;
    const int head = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
    const int n = (length_of(a, b) + a.block - 1) / a.block;
    if (n <= a.keep) return;
    const bool noise = head >= a.hs;
    const int h = noise ? head - a.hs : head, heads = noise ? a.hn : a.hs;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(noise ? a.q2 : a.q1) +
                             (static_cast<size_t>(b) * heads + h) * a.d;
    if (threadIdx.x < 32) {
        float v[4], amax = 0.f;
        bool nan = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = 4 * lane + k < a.d ? __bfloat162float(q[4 * lane + k]) : 0.f;
            nan |= v[k] != v[k];
            amax = fmaxf(amax, fabsf(v[k]));
        }
        amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
        nan = __any_sync(0xffffffffu, nan);
        const bool ok = !nan && amax >= 0x1p-100f && amax < INFINITY;
        const float r = ok ? __fdiv_rn(127.f, amax) : 0.f;
        uint32_t p = 0, m = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = ok ? __float2int_rn(__fmul_rn(v[k], r)) : 0;
            p |= static_cast<uint32_t>(max(i, 0)) << 8 * k;
            m |= (static_cast<uint32_t>(min(i, 0)) & 0xffu) << 8 * k;
        }
        pos[lane] = static_cast<int>(p), neg[lane] = static_cast<int>(m);
        if (lane == 0) amax_of = ok ? amax : -1.f;
    }
    __syncthreads();
    const float amax = amax_of;
    const int8_t *bounds = noise ? a.k2b : a.k1b;
    const float *scale = noise ? a.k2s : a.k1s;
    float *out = a.scores + (static_cast<size_t>(b) * (a.hs + a.hn) + head) * most;
    for (int j = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); j < n; j += gridDim.x * (kThreads / 32)) {
        const size_t at = pool_block(a, b, j) * heads + h;
        int ub = 0;
        if (4 * lane < a.d) {
            const int *w = reinterpret_cast<const int *>(bounds + at * 2 * a.d);
            ub = __dp4a(w[lane], pos[lane], __dp4a(w[a.d / 4 + lane], neg[lane], 0));
        }
        ub = __reduce_add_sync(0xffffffffu, ub);
        if (lane == 0)
            out[j] = amax < 0.f ? -INFINITY : __fmul_rn(__fmul_rn(static_cast<float>(ub), scale[at]), amax) + 0.f;
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

// grid (hn, B): keeps the blocks of one (sequence, noise head).
__global__ void __launch_bounds__(kThreads) gda_block_select_kernel(const BlockSelectArgs a, int most) {
    extern __shared__ uint32_t keys[];
    __shared__ float best[128], inverse[128];                // of the heads: the largest x, 1 / the sum of w
    __shared__ uint32_t hist[256];
    __shared__ uint32_t digit, left;
    __shared__ uint2 sums[kThreads / 32];
    const int g = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = (length_of(a, b) + a.block - 1) / a.block, kept = min(n, a.keep), r = a.hs / a.hn;
    int *list = a.list + (static_cast<size_t>(b) * a.hn + g) * a.keep;
    if (g == 0 && threadIdx.x == 0) a.count[b] = kept;
    for (int i = threadIdx.x + (n <= a.keep ? 0 : kept); i < a.keep; i += kThreads) list[i] = i < kept ? i : -1;
    if (n <= a.keep) return;
    const float *x = a.scores + static_cast<size_t>(b) * (a.hs + a.hn) * most;
    for (int i = warp; i <= r; i += kThreads / 32) {
        const float *xh = x + static_cast<size_t>(i == r ? a.hs + g : g * r + i) * most;
        float m = -INFINITY;
        for (int j = lane; j < n; j += 32) m = fmaxf(m, xh[j]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        unsigned long long total = 0;
        for (int j = lane; j < n; j += 32) total += units(weight(xh[j], m, a.unit));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane == 0) best[i] = m, inverse[i] = m > -INFINITY ? __frcp_rn(__fmul_rn(__ull2float_rn(total), 0x1p-40f)) : 0.f;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kThreads) {
        float s = 0.f;
        for (int i = 0; i <= r; ++i) {
            const float w = weight(x[static_cast<size_t>(i == r ? a.hs + g : g * r + i) * most + j], best[i], a.unit);
            s = fmaxf(s, __fmul_rn(w, inverse[i]));
        }
        // a share is at least 0 and orders like its bits
        keys[j] = j < a.first || j >= n - a.last ? 0xffffffffu : __float_as_uint(s);
    }
    // the kept-th highest key, eight bits at a time
    uint32_t prefix = 0, need = kept;
    for (int at = 24; at >= 0; at -= 8) {
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += kThreads) {
            const uint32_t k = keys[j];
            if (at == 24 || k >> (at + 8) == prefix >> (at + 8)) atomicAdd(&hist[k >> at & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            uint32_t above = 0;
            int dgt = 255;
            while (above + hist[dgt] < need) above += hist[dgt--];
            digit = dgt, left = need - above;
        }
        __syncthreads();
        prefix |= digit << at, need = left;
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

}  // namespace

int launch_block_select(const BlockSelectArgs &a, cudaStream_t stream) {
    const int most = a.max_pages * (a.page_size / a.block);
    const int chunks = (most + kThreads / 32 - 1) / (kThreads / 32);
    cudaError_t e = cudaFuncSetAttribute(gda_block_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kBlockSelectMaxBlocks * 4);
    if (e != cudaSuccess) return record_cuda_error(e);
    gda_block_score_kernel<<<dim3(chunks, a.hs + a.hn, a.B), kThreads, 0, stream>>>(a, most);
    e = cudaGetLastError();
    if (e != cudaSuccess) return record_cuda_error(e);
    gda_block_select_kernel<<<dim3(a.hn, a.B), kThreads, most * 4, stream>>>(a, most);
    e = cudaGetLastError();
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

}  // namespace gda
