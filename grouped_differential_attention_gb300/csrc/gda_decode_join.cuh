// The second kernel of the split decodes: what the ranges of a sequence left
// (maximum, sum and value sums of both maps) joined, the difference, and the
// (1 - lambda_init) RMSNorm.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "gda_device.cuh"

namespace gda {
namespace {

constexpr int kSms = 152;              // SMs that the plans of the split decodes count on

// Whether a row's sum of squares is of use for its norm.  Those of elements from about 2^64 on are past float32, and those
// below 2^-63 are lost, which tells where eps is as small.  The row is then taken once more, times early in the two maps'
// sums and late in their difference, powers of two that the norm takes out again: its squares are then at most 2^124, and at
// least 2^-118 for an element of 2^-149.
__device__ __forceinline__ bool norm_in_range(float squares, float eps, float &early, float &late) {
    if (squares <= 0x1p100f && (squares >= 0x1p-80f || eps >= 0x1p-60f)) return true;
    if (squares < 1.f) late = 0x1p90f;
    else early = 0x1p-70f;                 // (a NaN stays one)
    return false;
}

// The factor of a row that was taken times early * late.
__device__ __forceinline__ float norm_factor(float squares, int dv, float eps, float lambda_init, float early, float late) {
    const float f = early * late;
    return (1.f - lambda_init) * rsqrtf(squares * (1.f / dv) + eps * f * f);
}

// grid (h_s, B): joins the parts of one (sequence, head).  DV / 2 threads
// hold the DV + DV columns of (O1, O2), four each, with the maximum and sum of
// their map; THREADS / (DV / 2) such groups share the parts, each joining its
// own as it reads them (a part's statistics and values are fetched together),
// and are joined with one another at the end.  Params: out [B, hs, dv] bf16,
// ws_seg [B][2] (first and last range of a sequence), ws_ml [slots][hs][4] (m1,
// l1, m2, l2), ws_o [slots][hs][2][dv], splits, hs, B, lambda, lambda_init, eps;
// positions_of(p, b) is 0 for a sequence without a part.
template <int DV, int THREADS, class Params>
__global__ void __launch_bounds__(THREADS) gda_decode_join_kernel(const Params p) {
    constexpr int COLS = DV / 2, GROUPS = THREADS / COLS, HALF = COLS / 2;
    __shared__ float4 sums[GROUPS][COLS];
    __shared__ float2 stats[GROUPS][2];
    // a programmatic dependent of the split kernel: this wait returns once that grid has completed and its writes are visible
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = threadIdx.x % COLS, group = threadIdx.x / COLS;
    const bool second = col >= HALF;
    __nv_bfloat16 *out = p.out + (static_cast<size_t>(b) * p.hs + h) * DV;
    const int2 seg = reinterpret_cast<const int2 *>(p.ws_seg)[b];
    if (positions_of(p, b) == 0) {       // no position: the row is zero
        if (threadIdx.x < DV / 2) reinterpret_cast<uint32_t *>(out)[threadIdx.x] = 0u;
        return;
    }
    // ranges c0 .. c1 left a part in slots c + b (clamped so that a damaged workspace cannot send the reads astray)
    const int c0 = min(max(seg.x, 0), p.splits - 1), c1 = min(max(seg.y, c0), p.splits - 1);
    const size_t at0 = (static_cast<size_t>(c0) + b) * p.hs + h;
    const int parts = c1 - c0 + 1;
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml) + at0 * 2 + second;
    const float4 *o = reinterpret_cast<const float4 *>(p.ws_o) + at0 * COLS + col;

    float m = -INFINITY, l = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = group; c < parts; c += GROUPS) {
        const size_t at = static_cast<size_t>(c) * p.hs;
        const float2 s = ml[at * 2];
        const float4 v = o[at * COLS];
        const float top = fmaxf(m, s.x), f = fast_exp2(m - top), g = fast_exp2(s.x - top);
        m = top;
        l = fmaf(s.y, g, l * f);
        sum.x = fmaf(v.x, g, sum.x * f);
        sum.y = fmaf(v.y, g, sum.y * f);
        sum.z = fmaf(v.z, g, sum.z * f);
        sum.w = fmaf(v.w, g, sum.w * f);
    }
    sums[group][col] = sum;
    if (col % HALF == 0) stats[group][second] = make_float2(m, l);
    __syncthreads();
    if (threadIdx.x >= HALF) return;       // whole warps from here on, or half a warp (DV = 64)
    // groups beyond the parts hold (-inf, 0); the first one has at least one part
    const int used = min(GROUPS, parts);
    float M1 = -INFINITY, M2 = -INFINITY, L1 = 0.f, L2 = 0.f;
    for (int g = 0; g < used; ++g) M1 = fmaxf(M1, stats[g][0].x), M2 = fmaxf(M2, stats[g][1].x);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), d = a;
    for (int g = 0; g < used; ++g) {
        const float f1 = fast_exp2(stats[g][0].x - M1), f2 = fast_exp2(stats[g][1].x - M2);
        const float4 x = sums[g][col], y = sums[g][col + HALF];
        L1 = fmaf(stats[g][0].y, f1, L1), L2 = fmaf(stats[g][1].y, f2, L2);
        a.x = fmaf(x.x, f1, a.x), a.y = fmaf(x.y, f1, a.y), a.z = fmaf(x.z, f1, a.z), a.w = fmaf(x.w, f1, a.w);
        d.x = fmaf(y.x, f2, d.x), d.y = fmaf(y.y, f2, d.y), d.z = fmaf(y.z, f2, d.z), d.w = fmaf(y.w, f2, d.w);
    }
    if (L1 == 0.f) {                       // parts, but no position in any of them (a NaN is not 0)
        reinterpret_cast<uint2 *>(out)[col] = make_uint2(0u, 0u);
        return;
    }
    const float i1 = 1.f / L1, i2 = p.lambda[h] / L2;
    constexpr unsigned mask = HALF >= 32 ? 0xffffffffu : 0xffffu;
    float v[4], ss, early = 1.f, late = 1.f;
    for (int round = 0;; ++round) {        // the same for all threads: they have the same sum
        const float e1 = i1 * early, e2 = i2 * early;
        v[0] = (a.x * e1 - d.x * e2) * late, v[1] = (a.y * e1 - d.y * e2) * late;
        v[2] = (a.z * e1 - d.z * e2) * late, v[3] = (a.w * e1 - d.w * e2) * late;
        ss = v[0] * v[0] + v[1] * v[1] + v[2] * v[2] + v[3] * v[3];
#pragma unroll
        for (int off = (HALF >= 32 ? 32 : HALF) / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(mask, ss, off);
        if constexpr (HALF > 32) {         // DV = 256: two warps
            __shared__ float both[2][2];
            if (lane == 0) both[round][warp] = ss;
            named_bar_sync(1, HALF);
            ss = both[round][0] + both[round][1];
        }
        if (round > 0 || norm_in_range(ss, p.eps, early, late)) break;
    }
    const float y = norm_factor(ss, DV, p.eps, p.lambda_init, early, late);
    reinterpret_cast<uint2 *>(out)[col] = make_uint2(pack_bf16x2(v[0] * y, v[1] * y), pack_bf16x2(v[2] * y, v[3] * y));
}

template <int DV, int THREADS, class Params>
cudaError_t launch_join(const Params &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.hs, p.B);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, gda_decode_join_kernel<DV, THREADS, Params>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// The fewer the rows, the more parts each has and the more threads an SM can
// give it.  us with 256 / 512 / 1024 threads: 24 rows of 152 parts 22.6 / 15.0
// / 8.1, of up to 38 8.3 / 6.8 / 5.8; 256 rows 9.2 / 6.7 / 8.5; 768 rows 5.8 /
// 7.6 / 13.6.  So 1024 up to a row an SM, 512 up to two, 256 beyond.
template <int DV, class Params>
cudaError_t launch_join(const Params &p, cudaStream_t stream) {
    const int rows = p.hs * p.B;
    if (rows <= kSms) return launch_join<DV, 1024>(p, stream);
    return rows <= 2 * kSms ? launch_join<DV, 512>(p, stream) : launch_join<DV, 256>(p, stream);
}

}  // namespace
}  // namespace gda
