// RMSNorm of every query and key head row and its rotation by position, in
// one pass over the four projections, and the gradients of both.
//
// Row x of d values (one token, one head), weight row w of its tensor,
// rotated pairs (a, b) i = 0 .. rot/2 - 1, angle = position * inv_freq[i]:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r w
//   y_a = n_a cos - n_b sin,  y_b = n_b cos + n_a sin;  y = n beyond rot
// and, given dy, with dn the rotation of dy by -angle:
//   dw = sum over tokens and heads of dn x r
//   dx = r (dn w - x r^2 mean(dn w x))
// All of it in float32, one rounding at the end.
//
// Angles: position * inv_freq grows to hundreds of thousands of radians,
// where a float32 product has lost the phase.  inv_freq / (2 pi) is held as
// two floats (48 bits); the product with the position is split exactly by a
// fused multiply-add, whole turns drop out without rounding, and the rest
// goes to sincospif.  Positions of 2^24 and beyond, which float32 does not
// hold exactly, take the same steps in double.
//
// Memory-bound: a head row is read and written once (and dy read, for the
// gradients).  d/8 lanes hold a row, eight values a lane, in two groups of
// four that are partners in the rotation (a pair is never split over lanes,
// so only the mean needs shuffles): dims 4l.. and rot/2 + 4l.. when pairs
// are half a row apart, 8l.. and 8l + 4.. otherwise.  The tokens of a block
// share one table of sines in shared memory, which serves all their heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "gda.h"
#include "gda_device.cuh"
#include "gda_internal.h"

namespace gda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = 8;       // tokens of a block's sine table

// Four consecutive values of a row.
template <typename T>
__device__ __forceinline__ void load4(float (&f)[4], const T *p) {
    if constexpr (sizeof(T) == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    } else {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    }
}

template <typename T>
__device__ __forceinline__ void store4(T *p, const float (&f)[4]) {
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    else
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

// Frequency in turns as hi + lo.
struct Turns {
    float hi, lo;
};

__device__ __forceinline__ Turns turns_of(float inv_freq) {
    const double t = static_cast<double>(inv_freq) * 0.15915494309189533577;   // 1 / (2 pi)
    const float hi = static_cast<float>(t);
    return {hi, static_cast<float>(t - static_cast<double>(hi))};
}

// (cos, sin) of position * frequency.
__device__ __forceinline__ float2 angle(int pos, Turns f) {
    float turn;
    if (pos > -(1 << 24) && pos < (1 << 24)) {
        const float p = static_cast<float>(pos);
        const float whole = p * f.hi;
        const float rest = fmaf(p, f.hi, -whole);
        turn = (whole - rintf(whole)) + fmaf(p, f.lo, rest);
    } else {
        const double t = static_cast<double>(pos) * (static_cast<double>(f.hi) + static_cast<double>(f.lo));
        turn = static_cast<float>(t - rint(t));
    }
    float s, c;
    sincospif(2.f * turn, &s, &c);
    return make_float2(c, s);
}

// Where a lane's two groups of four dims start, and its four rotated pairs.
struct Lane {
    int a, b;      // first dims of the two groups
    int pair;      // table index of its first pair, -1: nothing to rotate
    bool apart;    // pairs are (a[i], b[i]); else (a[0], a[1]), (a[2], a[3]), (b[0], b[1]), (b[2], b[3])
};

__device__ __forceinline__ Lane lane_of(const NormRopeArgs &p, int l) {
    const bool rotated = 8 * l < p.rot;
    if (rotated && !p.interleaved) return {4 * l, p.rot / 2 + 4 * l, 4 * l, true};
    return {8 * l, 8 * l + 4, rotated ? 4 * l : -1, false};
}

__device__ __forceinline__ void turn_pair(float &x, float &y, float2 cs, float sign) {
    const float u = x, v = y, sn = sign * cs.y;
    x = u * cs.x - v * sn;
    y = v * cs.x + u * sn;
}

// Rotates the lane's four pairs by the table's angles (by the negative ones for sign = -1).
__device__ __forceinline__ void rotate(float (&a)[4], float (&b)[4], const Lane &ln, const float2 *cs, float sign) {
    if (ln.pair < 0) return;
    cs += ln.pair;
    if (ln.apart) {
#pragma unroll
        for (int i = 0; i < 4; ++i) turn_pair(a[i], b[i], cs[i], sign);
    } else {
        turn_pair(a[0], a[1], cs[0], sign);
        turn_pair(a[2], a[3], cs[1], sign);
        turn_pair(b[0], b[1], cs[2], sign);
        turn_pair(b[2], b[3], cs[3], sign);
    }
}

__device__ __forceinline__ float dot8(const float (&a)[4], const float (&b)[4], const float (&c)[4],
                                      const float (&d)[4]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fmaf(a[i], c[i], s);
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fmaf(b[i], d[i], s);
    return s;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float s) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// The block's sine table: pairs of `n` tokens from t0 on.
__device__ __forceinline__ void fill_table(const NormRopeArgs &p, float2 *table, long long t0, int n) {
    const int half = p.rot / 2;
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const int tok = i / half, pair = i - tok * half;
        table[i] = angle(p.positions[t0 + tok], turns_of(p.inv_freq[pair]));
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) gda_qk_norm_rope_kernel(const NormRopeArgs p, int tokens) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES;     // lanes of a row, rows of a warp
    __shared__ float2 table[kMaxTokens * D / 2];
    __shared__ float w[4 * D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Lane ln = lane_of(p, lane % LANES);
    for (int i = threadIdx.x; i < 4 * D; i += kThreads) w[i] = p.weight[i];
    const int per_token = 2 * (p.hs + p.hn);
    const long long t0 = static_cast<long long>(blockIdx.x) * tokens;
    const int n = static_cast<int>(min(static_cast<long long>(tokens), p.T - t0));
    fill_table(p, table, t0, n);
    __syncthreads();
    for (int base = warp * ROWS; base < n * per_token; base += kWarps * ROWS) {
        const int row = base + lane / LANES;
        const bool live = row < n * per_token;
        const int tok = live ? row / per_token : 0;
        int h = live ? row - tok * per_token : 0, t = 0;
        if (h >= p.hs) h -= p.hs, t = 1;
        if (t == 1 && h >= p.hs) h -= p.hs, t = 2;
        if (t == 2 && h >= p.hn) h -= p.hn, t = 3;
        const long long token = t0 + tok;
        const T *x = static_cast<const T *>(p.x[t]) + token * p.ld[t] + h * D;
        float a[4], b[4];
        load4(a, x + ln.a);
        load4(b, x + ln.b);
        const float r = rsqrtf(group_sum<LANES>(dot8(a, b, a, b)) * (1.f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] *= r * w[t * D + ln.a + i];
            b[i] *= r * w[t * D + ln.b + i];
        }
        rotate(a, b, ln, table + tok * (p.rot / 2), 1.f);
        if (live) {
            T *y = static_cast<T *>(p.y[t]) + (token * (t < 2 ? p.hs : p.hn) + h) * D;
            store4(y + ln.a, a);
            store4(y + ln.b, b);
        }
    }
}

// Gradients.  A block walks its tokens tensor by tensor, so that the eight
// sums of dw that belong to a lane stay in registers for the whole launch;
// they are joined over the block at the end, in a fixed order, and leave one
// row of partial sums per block and tensor in the workspace.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) gda_qk_norm_rope_bwd_kernel(const NormRopeArgs p, int tokens) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES;
    __shared__ float2 table[kMaxTokens * D / 2];
    __shared__ float part[kWarps][4 * D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Lane ln = lane_of(p, lane % LANES);
    float dwa[4][4] = {}, dwb[4][4] = {};
    for (long long t0 = static_cast<long long>(blockIdx.x) * tokens; t0 < p.T;
         t0 += static_cast<long long>(gridDim.x) * tokens) {
        const int n = static_cast<int>(min(static_cast<long long>(tokens), p.T - t0));
        __syncthreads();                                 // the table's last readers are done
        fill_table(p, table, t0, n);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int heads = t < 2 ? p.hs : p.hn;
            float wa[4], wb[4];
            load4(wa, p.weight + t * D + ln.a);
            load4(wb, p.weight + t * D + ln.b);
            for (int base = warp * ROWS; base < n * heads; base += kWarps * ROWS) {
                const int row = base + lane / LANES;
                const bool live = row < n * heads;
                const int tok = live ? row / heads : 0, h = live ? row - tok * heads : 0;
                const long long token = t0 + tok;
                const T *x = static_cast<const T *>(p.x[t]) + token * p.ld[t] + h * D;
                const float *dy = p.dy[t] + (token * heads + h) * D;
                float a[4], b[4], ga[4], gb[4];
                load4(a, x + ln.a);
                load4(b, x + ln.b);
                load4(ga, dy + ln.a);
                load4(gb, dy + ln.b);
                const float r = rsqrtf(group_sum<LANES>(dot8(a, b, a, b)) * (1.f / D) + p.eps);
                rotate(ga, gb, ln, table + tok * (p.rot / 2), -1.f);
                float ta[4], tb[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (live) {
                        dwa[t][i] = fmaf(ga[i] * r, a[i], dwa[t][i]);
                        dwb[t][i] = fmaf(gb[i] * r, b[i], dwb[t][i]);
                    }
                    ta[i] = ga[i] * wa[i];
                    tb[i] = gb[i] * wb[i];
                }
                const float c = group_sum<LANES>(dot8(ta, tb, a, b)) * (1.f / D) * r * r;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ta[i] = r * (ta[i] - a[i] * c);
                    tb[i] = r * (tb[i] - b[i] * c);
                }
                if (live) {
                    T *dx = static_cast<T *>(p.y[t]) + token * p.ldy[t] + h * D;
                    store4(dx + ln.a, ta);
                    store4(dx + ln.b, tb);
                }
            }
        }
    }
    // rows of a warp, then the warps in order
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = LANES; o < 32; o <<= 1) {
                dwa[t][i] += __shfl_xor_sync(0xffffffffu, dwa[t][i], o);
                dwb[t][i] += __shfl_xor_sync(0xffffffffu, dwb[t][i], o);
            }
            if (lane < LANES) {
                part[warp][t * D + ln.a + i] = dwa[t][i];
                part[warp][t * D + ln.b + i] = dwb[t][i];
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 4 * D; i += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) s += part[k][i];
        p.partial[static_cast<size_t>(blockIdx.x) * 4 * D + i] = s;
    }
}

// dw of 32 columns per block: 32 threads a column, each every 32nd partial row, joined in a fixed order.
__global__ void __launch_bounds__(1024) gda_qk_norm_rope_dw_kernel(const float *partial, float *dw, int blocks, int cols) {
    __shared__ float s[32][33];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    float v = 0.f;
    for (int b = k; b < blocks; b += 32) v += partial[static_cast<size_t>(b) * cols + col];
    s[k][c] = v;
    __syncthreads();
    v = s[c][k];                                  // warp k now holds the 32 sums of column k
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (c == 0) dw[blockIdx.x * 32 + k] = v;
}

// Tokens of a block: one until the SMs are full four times over, then up to eight.
int tokens_of(long long T) {
    const long long want = (T + kNormRopeBlocks - 1) / kNormRopeBlocks;
    return static_cast<int>(std::min<long long>(kMaxTokens, std::max<long long>(1, want)));
}

}  // namespace

int launch_qk_norm_rope(const NormRopeArgs &a, cudaStream_t stream) {
    const int tokens = tokens_of(a.T);
    const unsigned blocks = static_cast<unsigned>((a.T + tokens - 1) / tokens);
    auto kern = a.f32 ? (a.d == 64 ? gda_qk_norm_rope_kernel<float, 64> : gda_qk_norm_rope_kernel<float, 128>)
                      : (a.d == 64 ? gda_qk_norm_rope_kernel<__nv_bfloat16, 64>
                                   : gda_qk_norm_rope_kernel<__nv_bfloat16, 128>);
    kern<<<blocks, kThreads, 0, stream>>>(a, tokens);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

int launch_qk_norm_rope_bwd(const NormRopeArgs &a, cudaStream_t stream) {
    const int tokens = tokens_of(a.T);
    const int blocks = static_cast<int>(std::min<long long>(kNormRopeBlocks, (a.T + tokens - 1) / tokens));
    auto kern = a.f32 ? (a.d == 64 ? gda_qk_norm_rope_bwd_kernel<float, 64> : gda_qk_norm_rope_bwd_kernel<float, 128>)
                      : (a.d == 64 ? gda_qk_norm_rope_bwd_kernel<__nv_bfloat16, 64>
                                   : gda_qk_norm_rope_bwd_kernel<__nv_bfloat16, 128>);
    kern<<<blocks, kThreads, 0, stream>>>(a, tokens);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return record_cuda_error(e);
    gda_qk_norm_rope_dw_kernel<<<4 * a.d / 32, 1024, 0, stream>>>(a.partial, a.dweight, blocks, 4 * a.d);
    e = cudaGetLastError();
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

}  // namespace gda
