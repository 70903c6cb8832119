// Rows of K and V written into a 4-bit paged cache, and read back as bf16.
//
// Format (gda_fp4.cuh): for each block of 16 elements x of a head row, with
// the head's float32 scale g,
//   s = e4m3(max |x| / (6 g))            6 is the largest e2m1 magnitude
//   code_i = e2m1(x_i * (1 / (s g)))     0 where s rounds to 0
// in float32, each conversion to the nearest with ties to even and
// saturating; a NaN in the block makes s NaN, so that reading gives NaN for
// the whole block.  Reading gives bf16(code * s * g): the product code * s
// has at most six significant bits and is exact.
//
// One thread handles one block: 32 bytes of bf16 on one side, 8 bytes of
// codes and one scale byte on the other, so a warp touches 1 KB of
// consecutive bf16 whatever the head layout.  Memory-bound: 2.5625 bytes an
// element in each direction.  8192 tokens of 12 + 4 heads of 64/128, 53.7 MB:
// 12.5 us to write the cache, 13.3 to read it (kernels alone, cold; 7.9 at
// the copy rate of 6793 GB/s, the rest is the launch and the ramp at both
// ends); 64 tokens 3.6 and 3.4.  Two or four blocks to a thread, or threads in
// blocks of 128 or 512, are no faster (12.5 to 15.7, and 4 to 5.5 for 64).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "gda.h"
#include "gda_device.cuh"
#include "gda_fp4.cuh"
#include "gda_internal.h"

namespace gda {
namespace {

constexpr int kThreads = 256;

// Which tensor a block of 16 elements belongs to, and its place in the token's row there.
struct Place {
    int t;            // tensor: 0 K_sig, 1 K_noise, 2 V
    int in_row;       // block within the token's row of that tensor
};

__device__ __forceinline__ Place place_of(const CacheFp4Args &a, int blk) {
    if (blk < a.nb[0]) return {0, blk};
    blk -= a.nb[0];
    if (blk < a.nb[1]) return {1, blk};
    return {2, blk - a.nb[1]};
}

// Slot of token t: negative for a token to leave out.  A slot outside the pool is reported.
__device__ __forceinline__ int slot_of(const CacheFp4Args &a, long long t) {
    const int slot = a.slot_map[t];
    if (slot >= a.slots) {
        atomicOr(a.dev_err, GDA_DEVERR_BAD_PAGE);
        return -1;
    }
    return slot;
}

// A thread's token and block within it: `tokens` tokens to a thread block (32-bit division, a 64-bit one costs as much
// as the conversion).  False past the end.
__device__ __forceinline__ bool place(const CacheFp4Args &a, unsigned tokens, unsigned i, long long *tok, Place *pl) {
    const unsigned per_token = a.nb[0] + a.nb[1] + a.nb[2], t = i / per_token;
    *tok = static_cast<long long>(blockIdx.x) * tokens + t;
    *pl = place_of(a, static_cast<int>(i - t * per_token));
    return t < tokens && *tok < a.T;
}

__global__ void __launch_bounds__(kThreads) gda_cache_append_fp4_kernel(const CacheFp4Args a, unsigned tokens) {
    long long tok;
    Place pl;
    if (!place(a, tokens, blockIdx.y * kThreads + threadIdx.x, &tok, &pl)) return;
    const int slot = slot_of(a, tok);
    if (slot < 0) return;
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.rows[pl.t]) +
                                                       tok * a.ld[pl.t] + pl.in_row * kFp4Block);
    const uint4 lo = src[0], hi = src[1];
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    // magnitudes of bf16 order like their bits, and a NaN's are above infinity's
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) most = __vmaxu2(most, w[j] & 0x7fff7fffu);
    most = max(most & 0xffffu, most >> 16);
    const float g = a.scale[pl.t][pl.in_row >> a.shift[pl.t]];
    uint8_t s8 = 0x7f;
    float r = 0.f;
    if (most <= 0x7f80u) {
        s8 = float_to_e4m3(fminf(__fdiv_rn(__uint_as_float(most << 16), __fmul_rn(6.f, g)), 448.f));
        const float s = e4m3_to_float(s8);
        if (s > 0.f) r = __frcp_rn(__fmul_rn(s, g));
    }
    uint2 codes = {0u, 0u};
    if (r > 0.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = float2_to_e2m1x2(__fmul_rn(bf16_lo(w[j]), r), __fmul_rn(bf16_hi(w[j]), r));
            (j < 4 ? codes.x : codes.y) |= b << (8 * (j & 3));
        }
    }
    const size_t at = static_cast<size_t>(slot) * a.nb[pl.t] + pl.in_row;
    reinterpret_cast<uint2 *>(a.codes[pl.t])[at] = codes;
    a.blocks[pl.t][at] = s8;
}

__global__ void __launch_bounds__(kThreads) gda_cache_read_fp4_kernel(const CacheFp4Args a, unsigned tokens) {
    long long tok;
    Place pl;
    if (!place(a, tokens, blockIdx.y * kThreads + threadIdx.x, &tok, &pl)) return;
    const int slot = slot_of(a, tok);
    uint32_t o[8] = {};
    if (slot >= 0) {
        const size_t at = static_cast<size_t>(slot) * a.nb[pl.t] + pl.in_row;
        const uint2 codes = reinterpret_cast<const uint2 *>(a.codes[pl.t])[at];
        const float s = e4m3_to_float(a.blocks[pl.t][at]);
        const float g = a.scale[pl.t][pl.in_row >> a.shift[pl.t]];
        uint32_t h[2][4];
        e2m1x8_to_half2x4(h[0], codes.x);
        e2m1x8_to_half2x4(h[1], codes.y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 v = half2_bits_to_float2(h[j / 4][j % 4]);
            o[j] = pack_bf16x2(__fmul_rn(__fmul_rn(v.x, s), g), __fmul_rn(__fmul_rn(v.y, s), g));
        }
    }
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(const_cast<void *>(a.rows[pl.t])) +
                                           tok * a.ld[pl.t] + pl.in_row * kFp4Block);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// Thread blocks of kThreads blocks of 16 elements each: over groups of as many tokens as fill them best (x), and the
// pieces of a group (y).  With groups of one token 12 + 4 heads of 64/128 leave 96 of 256 threads idle; with 8, none.
dim3 grid_of(const CacheFp4Args &a, unsigned *tokens) {
    const unsigned per_token = a.nb[0] + a.nb[1] + a.nb[2];
    *tokens = 1;
    unsigned waste = kThreads;                       // idle threads, relative to the group's work
    for (unsigned t = 1; t <= 8; ++t) {
        const unsigned idle = (kThreads - t * per_token % kThreads) % kThreads;
        if (idle * *tokens < waste * t) *tokens = t, waste = idle;
    }
    return dim3(static_cast<unsigned>((a.T + *tokens - 1) / *tokens), (*tokens * per_token + kThreads - 1) / kThreads);
}

}  // namespace

int launch_cache_append_fp4(const CacheFp4Args &a, cudaStream_t stream) {
    unsigned tokens = 0;
    const dim3 grid = grid_of(a, &tokens);
    gda_cache_append_fp4_kernel<<<grid, kThreads, 0, stream>>>(a, tokens);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

int launch_cache_read_fp4(const CacheFp4Args &a, cudaStream_t stream) {
    unsigned tokens = 0;
    const dim3 grid = grid_of(a, &tokens);
    gda_cache_read_fp4_kernel<<<grid, kThreads, 0, stream>>>(a, tokens);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

}  // namespace gda
