// Grouped differential attention decode over an 8-bit KV cache with a scale
// for each block of tokens and head (one new query token per sequence; format
// in gda_fp8_block.cuh), contiguous or paged, over all positions of a sequence
// or over the blocks that a list names.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "gda.h"
#include "gda_device.cuh"
#include "gda_fp8_block.cuh"
#include "gda_internal.h"

namespace gda {
namespace {

constexpr int kWarps = 8;

// Length of sequence b; one outside [0, Lcap] is clamped and reported.
__device__ __forceinline__ int length_of(const DecodeFp8BlockArgs &p, int b) {
    const int len = p.lens[b];
    if (len >= 0 && len <= p.Lcap) return len;
    atomicOr(p.dev_err, GDA_DEVERR_BAD_LENGTH);
    return len < 0 ? 0 : p.Lcap;
}

// Cache row of position pos of sequence b.  A page outside the pool is read as page 0 and reported.
__device__ __forceinline__ uint32_t row_of(const DecodeFp8BlockArgs &p, int b, int pos) {
    const int pg = pos / p.page_size;
    int phys = b;
    if (p.block_table != nullptr) {
        phys = p.block_table[static_cast<size_t>(b) * p.max_pages + pg];
        if (phys < 0 || phys >= p.num_pages) {
            atomicOr(p.dev_err, GDA_DEVERR_BAD_PAGE);
            phys = 0;
        }
    }
    return static_cast<uint32_t>(phys) * p.page_size + (pos - pg * p.page_size);
}

template <int N>
__device__ __forceinline__ void load_codes(float (&v)[N], const uint8_t *src, float scale) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 f = half2_bits_to_float2(e4m3x2_to_half2(*reinterpret_cast<const uint16_t *>(src + i)));
        v[i] = f.x * scale, v[i + 1] = f.y * scale;
    }
}

// One map's running softmax over the positions of a warp.
template <int N>
struct State {
    float m = -INFINITY, l = 0.f, o[N] = {};
    __device__ void add(float x, const float (&v)[N]) {
        const float top = fmaxf(m, x), f = fast_exp2(m - top), w = fast_exp2(x - top);
        m = top;
        l = fmaf(l, f, w);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(o[i], f, w * v[i]);
    }
};

// grid (hs, B): one signal head of one sequence; a warp takes every kWarps-th position, a lane D / 32 and DV / 32 dims.
template <int D, int DV>
__global__ void __launch_bounds__(kWarps * 32) gda_decode_fp8_block_kernel(const DecodeFp8BlockArgs p, float scale_log2) {
    constexpr int ND = D / 32, NV = DV / 32;
    __shared__ float2 stats[2][kWarps];
    __shared__ float sums[2][kWarps][DV];
    __shared__ float squares[kWarps];
    const int h = blockIdx.x, b = blockIdx.y, g = h / (p.hs / p.hn);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + (static_cast<size_t>(b) * p.hs + h) * DV;
    const int len = length_of(p, b);
    long long n = len;
    if (p.list != nullptr) {
        int count = p.count[b];
        if (count < 0 || count > p.keep) {
            if (threadIdx.x == 0) atomicOr(p.dev_err, GDA_DEVERR_BAD_LENGTH);
            count = count < 0 ? 0 : p.keep;
        }
        n = static_cast<long long>(count) * p.block;
    }
    float q1[ND], q2[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) {
        q1[i] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.q1)[(static_cast<size_t>(b) * p.hs + h) * D + lane * ND + i]);
        q2[i] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.q2)[(static_cast<size_t>(b) * p.hn + g) * D + lane * ND + i]);
    }
    State<NV> s1, s2;
    for (long long i = warp; i < n; i += kWarps) {
        long long pos = i;
        if (p.list != nullptr) {
            const int id = p.list[(static_cast<size_t>(b) * p.hn + g) * p.keep + i / p.block];
            if (id < 0) continue;
            pos = static_cast<long long>(id) * p.block + i % p.block;
            if (pos >= len) continue;
        }
        const size_t row = row_of(p, b, static_cast<int>(pos)), blk = row / p.block;
        float k[ND], v[NV], x1 = 0.f, x2 = 0.f;
        load_codes<ND>(k, p.k1c + (row * p.hs + h) * D + lane * ND, p.k1s[blk * p.hs + h]);
#pragma unroll
        for (int j = 0; j < ND; ++j) x1 = fmaf(q1[j], k[j], x1);
        load_codes<ND>(k, p.k2c + (row * p.hn + g) * D + lane * ND, p.k2s[blk * p.hn + g]);
#pragma unroll
        for (int j = 0; j < ND; ++j) x2 = fmaf(q2[j], k[j], x2);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            x1 += __shfl_xor_sync(0xffffffffu, x1, o);
            x2 += __shfl_xor_sync(0xffffffffu, x2, o);
        }
        load_codes<NV>(v, p.vc + (row * p.hs + h) * DV + lane * NV, p.vs[blk * p.hs + h]);
        s1.add(x1 * scale_log2, v);
        s2.add(x2 * scale_log2, v);
    }
    if (lane == 0) stats[0][warp] = make_float2(s1.m, s1.l), stats[1][warp] = make_float2(s2.m, s2.l);
#pragma unroll
    for (int j = 0; j < NV; ++j) sums[0][warp][lane * NV + j] = s1.o[j], sums[1][warp][lane * NV + j] = s2.o[j];
    __syncthreads();
    float M[2], L[2] = {0.f, 0.f}, o = 0.f;
    for (int i = 0; i < 2; ++i) {
        M[i] = -INFINITY;
        for (int w = 0; w < kWarps; ++w) M[i] = fmaxf(M[i], stats[i][w].x);
        for (int w = 0; w < kWarps; ++w)
            if (stats[i][w].y != 0.f) L[i] += stats[i][w].y * fast_exp2(stats[i][w].x - M[i]);
    }
    const bool none = L[0] == 0.f;                           // no position: the row is zero
    if (threadIdx.x < DV && !none) {
        for (int i = 0; i < 2; ++i) {
            float a = 0.f;
            for (int w = 0; w < kWarps; ++w)
                if (stats[i][w].y != 0.f) a += sums[i][w][threadIdx.x] * fast_exp2(stats[i][w].x - M[i]);
            o += (i == 0 ? 1.f : -p.lambda[h]) * a / L[i];
        }
    }
    float ss = o * o;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if (lane == 0) squares[warp] = ss;
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < kWarps; ++w) ss += squares[w];
    if (threadIdx.x < DV)
        out[threadIdx.x] = __float2bfloat16((1.f - p.lambda_init) * o * rsqrtf(ss * (1.f / DV) + p.eps));
}

template <int D, int DV>
cudaError_t launch(const DecodeFp8BlockArgs &a, cudaStream_t stream) {
    const float scale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
    gda_decode_fp8_block_kernel<D, DV><<<dim3(a.hs, a.B), kWarps * 32, 0, stream>>>(a, scale);
    return cudaGetLastError();
}

}  // namespace

size_t decode_fp8_block_workspace_bytes(int B, int hs, int hn, int d, int dv) { return 16; }

int launch_decode_fp8_block(const DecodeFp8BlockArgs &a, cudaStream_t stream) {
    cudaError_t e = cudaErrorInvalidValue;
    switch (a.d * 1000 + a.dv) {
        case 64064: e = launch<64, 64>(a, stream); break;
        case 64128: e = launch<64, 128>(a, stream); break;
        case 64256: e = launch<64, 256>(a, stream); break;
        case 128064: e = launch<128, 64>(a, stream); break;
        case 128128: e = launch<128, 128>(a, stream); break;
        case 128256: e = launch<128, 256>(a, stream); break;
        default: return GDA_ERR_UNSUPPORTED;
    }
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

}  // namespace gda
