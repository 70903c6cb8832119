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
// goes to sincospif.  Those 48 bits leave an angle off by 2^-49 of itself, so
// from 2^22 turns on (and at positions of 2^24 and beyond, which float32 does
// not hold exactly) the same steps are taken in double, with 1 / (2 pi) as two
// doubles.  Either way the angle is off by its one rounding to float32.
//
// Memory-bound: a head row is read and written once (and dy read, for the
// gradients), so the arithmetic is kept below the copy.  d/8 lanes hold a
// row, eight values a lane, in two groups of four that are partners in the
// rotation (a pair is never split over lanes, so only the means need
// shuffles): dims 4l.. and rot/2 + 4l.. when pairs are half a row apart,
// 8l.. and 8l + 4.. otherwise.  A warp keeps its four (two at d = 128) head
// rows for the whole launch, so that their weights, sums of dw and addresses
// stay in registers, and walks over the block's tokens; the warps of a block
// are the rows of a token (and, when those are few, subsets of the tokens),
// and share a table of the tokens' sines in shared memory.  The rows of the
// next tokens are on their way into a ring of the warp's own (cp.async, one
// instruction a token): registers could hold two tokens ahead, which left
// the copy rate half used.  The grid is as many blocks as the SMs hold at a
// time, each with an equal run of tokens.
//
// Measured, of the 6793 GB/s of a copy: 32768 tokens, 24 + 8 heads of 64,
// bf16, 537 MB: 87.5 us (90 %), the kernel alone 81; 12 + 4 heads, float32,
// 537 MB: 81 alone; gradients of 8190 tokens, 16 + 4 heads of 128, float32,
// 503 MB: 84 us (88 %); of 8192 tokens, 12 + 4 heads of 64, bf16, 134 MB: 21.5
// us and 4.4 for the sum of dw (76 % together); 64 tokens: 4 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "gda.h"
#include "gda_device.cuh"
#include "gda_internal.h"

namespace gda {
namespace {

constexpr int kMaxWarps = 8;        // of a block
constexpr int kTokens = 16;         // tokens of a block's sine table
// Blocks of an SM: enough copies in flight, and few fronts in memory (prompt of 32768 tokens, 24 + 8 heads: 87.5 us with
// 3, 95 with 2, 99.5 with 4; gradients, float32: 84 us with 2, 92.5 with 1, 95 with 3).
constexpr int kForwardBlocks = 3, kBackwardBlocks = 2;

// A warp's head rows of one token in its ring: 256 elements, rows of 64 bf16
// with a gap of 64 bytes, which puts the two rows that a load of half a warp
// reads into different banks.
template <typename T, int D>
struct Stage {
    static constexpr int row = D * static_cast<int>(sizeof(T)) + (D * sizeof(T) == 128 ? 64 : 0);
    static constexpr int bytes = 256 / D * row;
};

// Eight elements of global memory (a lane's share of its row) into shared memory, asynchronously.
template <typename T>
__device__ __forceinline__ void copy8(uint32_t dst, const T *src) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * i), "l"(src + 4 * i) : "memory");
}

// Four consecutive values of a row in shared memory.
template <typename T>
__device__ __forceinline__ void fetch4(float (&f)[4], uint32_t a) {
    if constexpr (sizeof(T) == 2) {
        uint32_t x, y;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(a) : "memory");
        f[0] = bf16_lo(x), f[1] = bf16_hi(x), f[2] = bf16_lo(y), f[3] = bf16_hi(y);
    } else {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(a) : "memory");
    }
}

__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&f)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}
__device__ __forceinline__ void store4(float *p, const float (&f)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

// Frequency in turns as hi + lo, and as given.
struct Turns {
    float hi, lo, radians;
};

__device__ __forceinline__ Turns turns_of(float inv_freq) {
    const double t = static_cast<double>(inv_freq) * 0.15915494309189533577;   // 1 / (2 pi)
    const float hi = static_cast<float>(t);
    return {hi, static_cast<float>(t - static_cast<double>(hi)), inv_freq};
}

// (cos, sin) of position * frequency.
__device__ __forceinline__ float2 angle(int pos, Turns f) {
    const float p = static_cast<float>(pos), whole = p * f.hi;
    float turn;
    if (pos > -(1 << 24) && pos < (1 << 24) && fabsf(whole) < 4194304.f) {
        const float rest = fmaf(p, f.hi, -whole);
        turn = (whole - rintf(whole)) + fmaf(p, f.lo, rest);
    } else {
        constexpr double c = 0.15915494309189535, rest_of_c = -9.839338337591243e-18;   // 1 / (2 pi)
        const double q = pos, r = f.radians, t = r * c, low = fma(r, rest_of_c, fma(r, c, -t));   // frequency: t + low
        const double turns = q * t;
        turn = static_cast<float>((turns - rint(turns)) + fma(q, low, fma(q, t, -turns)));
    }
    float s, c;
    sincospif(2.f * turn, &s, &c);
    return make_float2(c, s);
}

// A lane's part of its head row: two groups of four dims, their weights, and
// the place of its four pairs in a token's row of the table.
struct Lane {
    int t, h;            // tensor (-1: no row) and head
    int a, b;            // first dims of the two groups
    int pair, step;      // table index of its first pair, and from token to token (0: pairs that do not turn)
};

template <int D, bool INTER>
__device__ __forceinline__ Lane lane_of(const NormRopeArgs &p, int row, int l) {
    Lane ln;
    ln.t = row < p.hs ? 0 : (row < 2 * p.hs ? 1 : (row < 2 * p.hs + p.hn ? 2 : (row < 2 * (p.hs + p.hn) ? 3 : -1)));
    ln.h = ln.t <= 0 ? row : (ln.t == 1 ? row - p.hs : (ln.t == 2 ? row - 2 * p.hs : row - 2 * p.hs - p.hn));
    if (ln.t < 0) ln.h = 0;
    const bool turns = 8 * l < p.rot;
    ln.a = turns && !INTER ? 4 * l : 8 * l;
    ln.b = turns && !INTER ? p.rot / 2 + 4 * l : 8 * l + 4;
    ln.pair = turns ? 4 * l : kTokens * p.rot;            // behind the table: four pairs of angle 0
    ln.step = turns ? p.rot : 0;
    return ln;
}

// Turns the lane's four pairs by the angles at cs (four cosines; the sines `half` further on),
// by the negative ones with BACK.  The partners are a[i], b[i], or neighbours (INTER).
template <bool INTER, bool BACK>
__device__ __forceinline__ void rotate(float (&a)[4], float (&b)[4], const float *cs, int half) {
    const float4 c = *reinterpret_cast<const float4 *>(cs), s = *reinterpret_cast<const float4 *>(cs + half);
    float x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = INTER ? (i < 2 ? a[2 * i] : b[2 * i - 4]) : a[i];
        y[i] = INTER ? (i < 2 ? a[2 * i + 1] : b[2 * i - 3]) : b[i];
    }
    float u[4] = {x[0], x[1], x[2], x[3]}, v[4] = {y[0], y[1], y[2], y[3]};
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; i += 2) {                      // forward: u = x c - y s, v = y c + x s
        fmul2(x[i], x[i + 1], ss[i], ss[i + 1]);
        fmul2(y[i], y[i + 1], ss[i], ss[i + 1]);
        fmul2(u[i], u[i + 1], cc[i], cc[i + 1]);
        fmul2(v[i], v[i + 1], cc[i], cc[i + 1]);
        if (BACK) {
            fadd2(u[i], u[i + 1], y[i], y[i + 1]);
            fsub2(v[i], v[i + 1], x[i], x[i + 1]);
        } else {
            fsub2(u[i], u[i + 1], y[i], y[i + 1]);
            fadd2(v[i], v[i + 1], x[i], x[i + 1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        (INTER ? (i < 2 ? a[2 * i] : b[2 * i - 4]) : a[i]) = u[i];
        (INTER ? (i < 2 ? a[2 * i + 1] : b[2 * i - 3]) : b[i]) = v[i];
    }
}

__device__ __forceinline__ float dot8(const float (&a)[4], const float (&b)[4], const float (&c)[4],
                                      const float (&d)[4]) {
    float s0 = 0.f, s1 = 0.f;
    ffma2_acc(s0, s1, a[0], a[1], c[0], c[1]);
    ffma2_acc(s0, s1, a[2], a[3], c[2], c[3]);
    ffma2_acc(s0, s1, b[0], b[1], d[0], d[1]);
    ffma2_acc(s0, s1, b[2], b[3], d[2], d[3]);
    return s0 + s1;
}

__device__ __forceinline__ void mul4(float (&a)[4], float b0, float b1, float b2, float b3) {
    fmul2(a[0], a[1], b0, b1);
    fmul2(a[2], a[3], b2, b3);
}

template <int LANES>
__device__ __forceinline__ float group_sum(float s) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// The block's table: for each of n tokens from t0 on, rot/2 cosines and rot/2 sines; behind kTokens of them
// (where only lanes without a turn look) four cosines of 1 and, rot/2 on, sines of 0.  freq: the pairs' turns.
__device__ __forceinline__ void fill_table(const NormRopeArgs &p, float *table, const Turns *freq, long long t0, int n) {
    const int half = p.rot / 2;
    for (int i = threadIdx.x; i < n * half; i += blockDim.x) {
        const int tok = i / half, pair = i - tok * half;
        const float2 cs = angle(p.positions[t0 + tok], freq[pair]);
        table[tok * p.rot + pair] = cs.x;
        table[tok * p.rot + half + pair] = cs.y;
    }
}
__device__ __forceinline__ void fill_rest(const NormRopeArgs &p, float *table, Turns *freq) {
    for (int i = threadIdx.x; i < p.rot / 2; i += blockDim.x) freq[i] = turns_of(p.inv_freq[i]);
    if (threadIdx.x < 4) {
        table[kTokens * p.rot + threadIdx.x] = 1.f;
        table[kTokens * p.rot + p.rot / 2 + threadIdx.x] = 0.f;
    }
}

// Tokens of a block: [first, last) of the launch's, in runs of kTokens.  Warp w has the rows of group w % groups
// of the block's, for every subsets-th token from w / groups on.
struct Shape {
    int groups, subsets, blocks_y;
    long long per;       // tokens of a block
    int blocks_x;
};

template <typename T, int D, bool INTER, int RING>
__global__ void __launch_bounds__(kMaxWarps * 32, kForwardBlocks)
gda_qk_norm_rope_kernel(const NormRopeArgs p, const Shape shape) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES;      // lanes of a row, rows of a warp
    using S = Stage<T, D>;
    extern __shared__ __align__(128) uint8_t rings[];
    __shared__ __align__(16) float table[kTokens * D + D / 2 + 4];
    __shared__ Turns freq[D / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp % shape.groups, subset = warp / shape.groups;
    const int row = (blockIdx.y * shape.groups + group) * ROWS + lane / LANES;
    const Lane ln = lane_of<D, INTER>(p, row, lane % LANES);
    const bool live = ln.t >= 0;
    const int t = live ? ln.t : 0;
    const float4 wa = *reinterpret_cast<const float4 *>(p.weight + t * D + ln.a);
    const float4 wb = *reinterpret_cast<const float4 *>(p.weight + t * D + ln.b);
    const long long ldx = p.ld[t], ldy = static_cast<long long>(t < 2 ? p.hs : p.hn) * D;
    const int half = p.rot / 2, ahead = ln.b - ln.a;
    const long long first = blockIdx.x * shape.per, last = min(p.T, first + shape.per);
    const T *x = static_cast<const T *>(p.x[t]) + min(first + subset, p.T - 1) * ldx + ln.h * D + lane % LANES * 8;
    T *y = static_cast<T *>(p.y[t]) + (first + subset) * ldy + ln.h * D + ln.a;
    int left = static_cast<int>((last - first - subset + shape.subsets - 1) / shape.subsets);   // this warp's tokens
    int loads = left;
    const uint32_t ring = smem_u32(rings) + warp * RING * S::bytes + lane / LANES * S::row;
    auto load = [&](int slot) {
        if (loads > 0) copy8(ring + slot * S::bytes + lane % LANES * 8 * static_cast<int>(sizeof(T)), x);
        asm volatile("cp.async.commit_group;" ::: "memory");
        --loads;
        x += shape.subsets * ldx;
    };
#pragma unroll
    for (int u = 0; u < RING - 1; ++u) load(u);
    int from = 0, to = RING - 1;
    fill_rest(p, table, freq);
    for (long long t0 = first; t0 < last; t0 += kTokens) {
        __syncthreads();                                 // the table's last readers are done
        fill_table(p, table, freq, t0, static_cast<int>(min(static_cast<long long>(kTokens), last - t0)));
        __syncthreads();
        const float *cs = table + ln.pair + subset * ln.step;
        for (int tok = 0; tok < kTokens && left > 0; tok += shape.subsets) {
            --left;
            asm volatile("cp.async.wait_group %0;" ::"n"(RING - 2) : "memory");
            __syncwarp();                                // all lanes' copies have landed; the oldest place is free
            load(to);
            float a[4], b[4];
            fetch4<T>(a, ring + from * S::bytes + ln.a * static_cast<int>(sizeof(T)));
            fetch4<T>(b, ring + from * S::bytes + ln.b * static_cast<int>(sizeof(T)));
            to = to + 1 == RING ? 0 : to + 1;
            from = from + 1 == RING ? 0 : from + 1;
            const float r = rsqrtf(group_sum<LANES>(dot8(a, b, a, b)) * (1.f / D) + p.eps);
            mul4(a, r * wa.x, r * wa.y, r * wa.z, r * wa.w);
            mul4(b, r * wb.x, r * wb.y, r * wb.z, r * wb.w);
            rotate<INTER, false>(a, b, cs, half);
            cs += shape.subsets * ln.step;
            if (live) {
                store4(y, a);
                store4(y + ahead, b);
            }
            y += shape.subsets * ldy;
        }
    }
}

// Gradients.  The eight sums of dw of a lane's row stay in registers for the
// whole launch; they are joined over the block at the end, in a fixed order,
// and leave one row of partial sums per block and tensor in the workspace.
template <typename T, int D, bool INTER, int RING>
__global__ void __launch_bounds__(kMaxWarps * 32, kBackwardBlocks)
gda_qk_norm_rope_bwd_kernel(const NormRopeArgs p, const Shape shape) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES;
    using S = Stage<T, D>;
    using G = Stage<float, D>;
    extern __shared__ __align__(128) uint8_t rings[];
    __shared__ __align__(16) float table[kTokens * D + D / 2 + 4];
    __shared__ Turns freq[D / 2];
    __shared__ float part[kMaxWarps * ROWS][D];
    __shared__ int owner[kMaxWarps * ROWS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp % shape.groups, subset = warp / shape.groups;
    const int row = (blockIdx.y * shape.groups + group) * ROWS + lane / LANES;
    const Lane ln = lane_of<D, INTER>(p, row, lane % LANES);
    const bool live = ln.t >= 0;
    const int t = live ? ln.t : 0;
    const float4 wa = *reinterpret_cast<const float4 *>(p.weight + t * D + ln.a);
    const float4 wb = *reinterpret_cast<const float4 *>(p.weight + t * D + ln.b);
    const long long ldx = p.ld[t], lddx = p.ldy[t], ldg = static_cast<long long>(t < 2 ? p.hs : p.hn) * D;
    const int half = p.rot / 2, ahead = ln.b - ln.a;
    const long long first = blockIdx.x * shape.per, last = min(p.T, first + shape.per);
    float dwa[4] = {}, dwb[4] = {}, suma[4] = {}, sumb[4] = {};   // of a table's tokens; of all before
    fill_rest(p, table, freq);
    const long long at = min(first + subset, p.T - 1);
    const int eighth = lane % LANES * 8;
    const T *x = static_cast<const T *>(p.x[t]) + at * ldx + ln.h * D + eighth;
    const float *g = p.dy[t] + at * ldg + ln.h * D + eighth;
    T *dx = static_cast<T *>(p.y[t]) + (first + subset) * lddx + ln.h * D + ln.a;
    int left = static_cast<int>((last - first - subset + shape.subsets - 1) / shape.subsets);   // this warp's tokens
    int loads = left;
    const uint32_t ring = smem_u32(rings) + warp * RING * (S::bytes + G::bytes) + lane / LANES * S::row;
    const uint32_t gring = ring + RING * S::bytes + lane / LANES * (G::row - S::row);
    auto load = [&](int slot) {
        if (loads > 0) {
            copy8(ring + slot * S::bytes + eighth * static_cast<int>(sizeof(T)), x);
            copy8(gring + slot * G::bytes + eighth * 4, g);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        --loads;
        x += shape.subsets * ldx;
        g += shape.subsets * ldg;
    };
#pragma unroll
    for (int u = 0; u < RING - 1; ++u) load(u);
    int from = 0, to = RING - 1;
    for (long long t0 = first; t0 < last; t0 += kTokens) {
        __syncthreads();
        fill_table(p, table, freq, t0, static_cast<int>(min(static_cast<long long>(kTokens), last - t0)));
        __syncthreads();
        const float *cs = table + ln.pair + subset * ln.step;
        for (int tok = 0; tok < kTokens && left > 0; tok += shape.subsets) {
            --left;
            asm volatile("cp.async.wait_group %0;" ::"n"(RING - 2) : "memory");
            __syncwarp();
            load(to);
            float a[4], b[4], ga[4], gb[4];
            fetch4<T>(a, ring + from * S::bytes + ln.a * static_cast<int>(sizeof(T)));
            fetch4<T>(b, ring + from * S::bytes + ln.b * static_cast<int>(sizeof(T)));
            fetch4<float>(ga, gring + from * G::bytes + ln.a * 4);
            fetch4<float>(gb, gring + from * G::bytes + ln.b * 4);
            to = to + 1 == RING ? 0 : to + 1;
            from = from + 1 == RING ? 0 : from + 1;
            rotate<INTER, true>(ga, gb, cs, half);
            float ta[4] = {ga[0], ga[1], ga[2], ga[3]}, tb[4] = {gb[0], gb[1], gb[2], gb[3]};
            mul4(ta, wa.x, wa.y, wa.z, wa.w);
            mul4(tb, wb.x, wb.y, wb.z, wb.w);
            const float xx = group_sum<LANES>(dot8(a, b, a, b)), tx = group_sum<LANES>(dot8(ta, tb, a, b));
            const float r = rsqrtf(xx * (1.f / D) + p.eps);
            const float c = -(tx * (1.f / D) * r * r);
            // t + c x, then x r for dw
            ffma2_acc(ta[0], ta[1], c, c, a[0], a[1]);
            ffma2_acc(ta[2], ta[3], c, c, a[2], a[3]);
            ffma2_acc(tb[0], tb[1], c, c, b[0], b[1]);
            ffma2_acc(tb[2], tb[3], c, c, b[2], b[3]);
            mul4(ta, r, r, r, r);
            mul4(tb, r, r, r, r);
            mul4(a, r, r, r, r);
            mul4(b, r, r, r, r);
            ffma2_acc(dwa[0], dwa[1], ga[0], ga[1], a[0], a[1]);
            ffma2_acc(dwa[2], dwa[3], ga[2], ga[3], a[2], a[3]);
            ffma2_acc(dwb[0], dwb[1], gb[0], gb[1], b[0], b[1]);
            ffma2_acc(dwb[2], dwb[3], gb[2], gb[3], b[2], b[3]);
            if (live) {
                store4(dx, ta);
                store4(dx + ahead, tb);
            }
            dx += shape.subsets * lddx;
            cs += shape.subsets * ln.step;
        }
        // sums of sums: the error of one long float32 sum grows with its length (dw of 8190 tokens was off by 2.0e-7 of
        // its size, this way by 1.5e-7; at no cost)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            suma[i] += dwa[i], sumb[i] += dwb[i];
            dwa[i] = dwb[i] = 0.f;
        }
    }
    const int mine = warp * ROWS + lane / LANES;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        part[mine][ln.a + i] = suma[i];
        part[mine][ln.b + i] = sumb[i];
    }
    if (lane % LANES == 0) owner[mine] = ln.t;
    __syncthreads();
    const int rows = (blockDim.x >> 5) * ROWS;
    float *out = p.partial + static_cast<size_t>(blockIdx.y * gridDim.x + blockIdx.x) * 4 * D;
    for (int i = threadIdx.x; i < 4 * D; i += blockDim.x) {
        float s[4] = {};
        for (int k = 0; k < rows; ++k)
            if (owner[k] == i / D) s[k & 3] += part[k][i % D];
        out[i] = (s[0] + s[1]) + (s[2] + s[3]);
    }
}

// dw of 8 columns per block: 128 threads a column, each every 128th partial row, joined in a fixed order.
__global__ void __launch_bounds__(1024) gda_qk_norm_rope_dw_kernel(const float *partial, float *dw, int blocks, int cols) {
    __shared__ float s[128][9];
    // a programmatic dependent of the gradient kernel: returns once that grid has completed and its writes are visible
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = threadIdx.x & 7, k = threadIdx.x >> 3;
    float v = 0.f;
#pragma unroll 4
    for (int b = k; b < blocks; b += 128) v += partial[static_cast<size_t>(b) * cols + blockIdx.x * 8 + c];
    s[k][c] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31, col = threadIdx.x >> 5;
    if (col >= 8) return;                         // a warp for each column
    v = (s[lane][col] + s[lane + 32][col]) + (s[lane + 64][col] + s[lane + 96][col]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) dw[blockIdx.x * 8 + col] = v;
}

// As many blocks as fit `sms` * `each` at a time, over the head rows and equal runs of tokens.
Shape shape_of(const NormRopeArgs &a, int most) {
    const int rows = a.d == 64 ? 4 : 2, groups = (2 * (a.hs + a.hn) + rows - 1) / rows;
    Shape s;
    s.blocks_y = (groups + kMaxWarps - 1) / kMaxWarps;
    s.groups = (groups + s.blocks_y - 1) / s.blocks_y;
    s.subsets = kMaxWarps / s.groups;
    const long long want = std::max(1, most / s.blocks_y);
    s.per = (a.T + want - 1) / want;
    if (s.per < s.subsets) s.per = s.subsets;    // a token for each warp
    s.blocks_x = static_cast<int>((a.T + s.per - 1) / s.per);
    return s;
}

template <typename T, int D, bool INTER>
cudaError_t forward(const NormRopeArgs &a, const Shape &s, cudaStream_t stream) {
    constexpr int RING = 5;                       // prompt of 32768 tokens: 87.5 us; 88.5 with 4, 94 with 6, 98.5 with 7
    auto kern = gda_qk_norm_rope_kernel<T, D, INTER, RING>;
    const int warps = s.groups * s.subsets, one = RING * Stage<T, D>::bytes;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxWarps * one);
    if (e != cudaSuccess) return e;
    kern<<<dim3(s.blocks_x, s.blocks_y), warps * 32, warps * one, stream>>>(a, s);
    return cudaGetLastError();
}

template <typename T, int D, bool INTER>
cudaError_t backward(const NormRopeArgs &a, const Shape &s, cudaStream_t stream) {
    constexpr int RING = 4;
    auto kern = gda_qk_norm_rope_bwd_kernel<T, D, INTER, RING>;
    const int warps = s.groups * s.subsets, one = RING * (Stage<T, D>::bytes + Stage<float, D>::bytes);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxWarps * one);
    if (e != cudaSuccess) return e;
    kern<<<dim3(s.blocks_x, s.blocks_y), warps * 32, warps * one, stream>>>(a, s);
    return cudaGetLastError();
}

template <bool INTER>
cudaError_t forward(const NormRopeArgs &a, const Shape &s, cudaStream_t stream) {
    if (a.f32) return a.d == 64 ? forward<float, 64, INTER>(a, s, stream) : forward<float, 128, INTER>(a, s, stream);
    return a.d == 64 ? forward<__nv_bfloat16, 64, INTER>(a, s, stream) : forward<__nv_bfloat16, 128, INTER>(a, s, stream);
}

template <bool INTER>
cudaError_t backward(const NormRopeArgs &a, const Shape &s, cudaStream_t stream) {
    if (a.f32) return a.d == 64 ? backward<float, 64, INTER>(a, s, stream) : backward<float, 128, INTER>(a, s, stream);
    return a.d == 64 ? backward<__nv_bfloat16, 64, INTER>(a, s, stream) : backward<__nv_bfloat16, 128, INTER>(a, s, stream);
}

}  // namespace

int launch_qk_norm_rope(const NormRopeArgs &a, cudaStream_t stream) {
    const Shape s = shape_of(a, kNormRopeSms * kForwardBlocks);
    const cudaError_t e = a.interleaved ? forward<true>(a, s, stream) : forward<false>(a, s, stream);
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

int launch_qk_norm_rope_bwd(const NormRopeArgs &a, cudaStream_t stream) {
    const Shape s = shape_of(a, kNormRopeSms * kBackwardBlocks);
    cudaError_t e = a.interleaved ? backward<true>(a, s, stream) : backward<false>(a, s, stream);
    if (e != cudaSuccess) return record_cuda_error(e);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(4 * a.d / 8);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gda_qk_norm_rope_dw_kernel, static_cast<const float *>(a.partial), a.dweight,
                           s.blocks_x * s.blocks_y, 4 * a.d);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

size_t qk_norm_rope_bwd_workspace_bytes(int T, int hs, int hn, int d) {
    NormRopeArgs a{};
    a.T = T, a.hs = hs, a.hn = hn, a.d = d;
    const Shape s = shape_of(a, kNormRopeSms * kBackwardBlocks);
    return static_cast<size_t>(s.blocks_x) * s.blocks_y * 4 * d * sizeof(float);
}

}  // namespace gda
