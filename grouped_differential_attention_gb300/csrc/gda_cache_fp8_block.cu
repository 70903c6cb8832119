// Rows of K and V written into an 8-bit paged cache with a scale for each
// block of tokens and head, and read back as bf16.
//
// A block of tokens (consecutive slots of a page) and a head have one float32
// scale.  Writing rows x into it:
//   s     = the least power of two with max |x| <= 448 s   (448: e4m3's largest)
//   scale = max(scale before, s); the rows that are there already are brought
//           to it, code' = e4m3(code * (before / scale)).  A call that writes
//           the first row of the block starts it anew: nothing is there.
//   code  = e4m3(x * (1 / scale)), to the nearest, ties to even; above 1.875 *
//           2^127, where that would stand for 2^128, the code below.
// NaN and infinities are NaN codes and do not count for s.  A power of two
// loses nothing: e4m3 is a floating type, so all codes keep their four digits
// down to its subnormals, 2^-15 of the block's largest, and a growing scale
// leaves the digits of the rows before as they are.
// Bounds of a block's keys, for gda_block_select, in fours of the scale:
//   max over rows of ceil(code / 4), min of floor(code / 4), one int8 each for
// every channel (|code| <= 448, so at most 112), -128 and 127 if there is none.
// ceil(ceil(x / 4) / 2^k) = ceil(x / 4 / 2^k), so a growing scale keeps them exact.
//
// Two launches.  The rows of a block may be anywhere in the call, so the first
// one writes into index[slot] which row has that slot.  An entry counts only
// if that row's slot is this slot, so what else the workspace holds does no
// harm.  In the second one the block of the row with the lowest slot of a
// block does all of it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "gda.h"
#include "gda_device.cuh"
#include "gda_fp8_block.cuh"
#include "gda_internal.h"

namespace gda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlock = 128;

__global__ void __launch_bounds__(kThreads) gda_cache_index_kernel(const CacheFp8BlockArgs a) {
    const long long t = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    if (t >= a.T) return;
    const int slot = a.slot_map[t];
    if (slot >= a.slots) atomicOr(a.dev_err, GDA_DEVERR_BAD_PAGE);
    else if (slot >= 0) a.index[slot] = static_cast<int>(t);
}

// The row of this call that has this slot, or -1.
__device__ __forceinline__ int row_of_slot(const CacheFp8BlockArgs &a, int slot) {
    const int t = a.index[slot];
    return t >= 0 && t < a.T && a.slot_map[t] == slot ? t : -1;
}

__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
    const __half2 r = __hmax2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {
    const __half2 r = __hmin2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Bits of |x| where x is finite, 0 where not.
__device__ __forceinline__ uint32_t finite_abs(uint32_t bits) {
    bits &= 0x7fffffffu;
    return bits < 0x7f800000u ? bits : 0u;
}

// One warp, one (block, head): N / 8 lanes to a row.  row[]: the call's row of each slot of the block, or -1.
template <int N>
__device__ void write_head(const CacheFp8BlockArgs &a, int tensor, int head, int blk, const int *row, bool fresh) {
    constexpr int LANES = N / 8, STEP = 32 / LANES;
    const int lane = threadIdx.x & 31, sub = lane / LANES, ch = lane % LANES * 8;
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.rows[tensor]) + head * N + ch;
    const long long ld = a.ld[tensor];
    const size_t pitch = static_cast<size_t>(a.heads[tensor]) * N;
    uint8_t *codes = a.codes[tensor] + static_cast<size_t>(blk) * a.block * pitch + head * N + ch;

    uint32_t most = 0;
    for (int i = sub; i < a.block; i += STEP) {
        const int t = row[i];
        if (t < 0) continue;
        const uint4 w = *reinterpret_cast<const uint4 *>(x + t * ld);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) most = max(most, max(finite_abs(v[k] << 16), finite_abs(v[k] & 0xffff0000u)));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    float *const where = a.scale[tensor] + static_cast<size_t>(blk) * a.heads[tensor] + head;
    const float old = fresh ? 0.f : *where, scale = fmaxf(old, fp8_scale_of(most));
    const float r = __frcp_rn(scale), shift = fresh ? 1.f : __fdiv_rn(old, scale);
    const float most_code = fminf(448.f, __fdiv_rn(0x1.ep127f, scale));
    __syncwarp();
    if (lane == 0) *where = scale;

    const uint32_t none_max = 0xfc00fc00u, none_min = 0x7c007c00u;   // -inf, inf
    uint32_t top[4] = {none_max, none_max, none_max, none_max}, low[4] = {none_min, none_min, none_min, none_min};
    for (int i = sub; i < a.block; i += STEP) {
        const int t = row[i];
        uint2 *const dst = reinterpret_cast<uint2 *>(codes + i * pitch);
        if (t < 0) {
            if (shift == 1.f) continue;
            const uint2 c = *dst;                            // a row that is there already
            const uint32_t w[2] = {c.x, c.y};
            uint32_t o[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint2 h = e4m3x4_to_half2x2(w[k]);
                const float2 p = half2_bits_to_float2(h.x), q = half2_bits_to_float2(h.y);
                o[k] = float2_to_e4m3x2(p.x * shift, p.y * shift) | float2_to_e4m3x2(q.x * shift, q.y * shift) << 16;
            }
            *dst = make_uint2(o[0], o[1]);
            continue;
        }
        const uint4 w = *reinterpret_cast<const uint4 *>(x + t * ld);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
        uint32_t c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float lo = bf16_lo(v[k]), hi = bf16_hi(v[k]);
            c[k] = float2_to_e4m3x2(fmaxf(-most_code, fminf(most_code, __fmul_rn(lo, r))),
                                    fmaxf(-most_code, fminf(most_code, __fmul_rn(hi, r))));
            // the limits have made a number of what is none
            if ((v[k] & 0x7fffu) >= 0x7f80u) c[k] |= 0x7fu;
            if ((v[k] & 0x7fff0000u) >= 0x7f800000u) c[k] |= 0x7f00u;
            if (tensor < 2) {
                const uint32_t h = e4m3x2_to_half2(c[k]);    // a NaN is passed over by max and min
                top[k] = hmax2(top[k], h);
                low[k] = hmin2(low[k], h);
            }
        }
        *dst = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    }
    if (tensor == 2 || a.bounds[0] == nullptr) return;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
            top[k] = hmax2(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
            low[k] = hmin2(low[k], __shfl_xor_sync(0xffffffffu, low[k], o));
        }
    if (sub != 0) return;
    int8_t *const bounds = a.bounds[tensor] + (static_cast<size_t>(blk) * a.heads[tensor] + head) * 2 * N + ch;
    uint2 *const at_top = reinterpret_cast<uint2 *>(bounds), *const at_low = reinterpret_cast<uint2 *>(bounds + N);
    const uint2 old_top = *at_top, old_low = *at_low;
    uint32_t nt[2] = {0u, 0u}, nl[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 t2 = half2_bits_to_float2(top[k / 2]), l2 = half2_bits_to_float2(low[k / 2]);
        float t = ceilf((k & 1 ? t2.y : t2.x) * 0.25f), l = floorf((k & 1 ? l2.y : l2.x) * 0.25f);
        t = fmaxf(t, -128.f), l = fminf(l, 127.f);           // no finite value: -128 and 127
        if (!fresh) {
            const uint32_t ot = (k < 4 ? old_top.x : old_top.y) >> 8 * (k & 3);
            const uint32_t ol = (k < 4 ? old_low.x : old_low.y) >> 8 * (k & 3);
            t = fmaxf(t, ceilf(static_cast<float>(static_cast<int8_t>(ot)) * shift));
            l = fminf(l, floorf(static_cast<float>(static_cast<int8_t>(ol)) * shift));
        }
        nt[k / 4] |= (static_cast<uint32_t>(static_cast<int>(t)) & 0xffu) << 8 * (k & 3);
        nl[k / 4] |= (static_cast<uint32_t>(static_cast<int>(l)) & 0xffu) << 8 * (k & 3);
    }
    *at_top = make_uint2(nt[0], nt[1]);
    *at_low = make_uint2(nl[0], nl[1]);
}

// grid: a thread block for each row of the call; the row with the lowest slot of a block of tokens writes that block.
__global__ void __launch_bounds__(kThreads) gda_cache_append_fp8_block_kernel(const CacheFp8BlockArgs a) {
    __shared__ int row[kMaxBlock];
    const int t = blockIdx.x, slot = a.slot_map[t];
    if (slot < 0 || slot >= a.slots) return;
    const int blk = slot / a.block, first = blk * a.block;
    bool earlier = a.index[slot] != t;                       // two rows with one slot: one of them is written
    for (int i = threadIdx.x; i < a.block; i += kThreads) {
        row[i] = row_of_slot(a, first + i);
        earlier |= row[i] >= 0 && first + i < slot;
    }
    if (__syncthreads_or(earlier)) return;
    const bool fresh = row[0] >= 0;
    const int total = a.heads[0] + a.heads[1] + a.heads[2];
    for (int i = threadIdx.x >> 5; i < total; i += kThreads / 32) {
        const int tensor = i < a.heads[0] ? 0 : (i < a.heads[0] + a.heads[1] ? 1 : 2);
        const int head = i - (tensor > 0 ? a.heads[0] : 0) - (tensor > 1 ? a.heads[1] : 0);
        const int n = a.dims[tensor];
        if (n == 64) write_head<64>(a, tensor, head, blk, row, fresh);
        else if (n == 128) write_head<128>(a, tensor, head, blk, row, fresh);
        else write_head<256>(a, tensor, head, blk, row, fresh);
    }
}

// One thread: 16 elements of one row.
__global__ void __launch_bounds__(kThreads) gda_cache_read_fp8_block_kernel(const CacheFp8BlockArgs a) {
    const int n0 = a.heads[0] * a.dims[0] / 16, n1 = a.heads[1] * a.dims[1] / 16, n2 = a.heads[2] * a.dims[2] / 16;
    const long long tok = blockIdx.x;
    const int slot = a.slot_map[tok];
    if (slot >= a.slots && threadIdx.x == 0) atomicOr(a.dev_err, GDA_DEVERR_BAD_PAGE);
    for (int i = threadIdx.x; i < n0 + n1 + n2; i += kThreads) {
        const int tensor = i < n0 ? 0 : (i < n0 + n1 ? 1 : 2), in_row = i - (tensor > 0 ? n0 : 0) - (tensor > 1 ? n1 : 0);
        uint32_t o[8] = {};
        if (slot >= 0 && slot < a.slots) {
            const size_t pitch = static_cast<size_t>(a.heads[tensor]) * a.dims[tensor];
            const uint4 c = *reinterpret_cast<const uint4 *>(a.codes[tensor] + slot * pitch + in_row * 16);
            const float s = a.scale[tensor][static_cast<size_t>(slot / a.block) * a.heads[tensor] +
                                            in_row * 16 / a.dims[tensor]];
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint2 h = e4m3x4_to_half2x2(w[k]);
                const float2 p = half2_bits_to_float2(h.x), q = half2_bits_to_float2(h.y);
                o[2 * k] = pack_bf16x2(__fmul_rn(p.x, s), __fmul_rn(p.y, s));
                o[2 * k + 1] = pack_bf16x2(__fmul_rn(q.x, s), __fmul_rn(q.y, s));
            }
        }
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(const_cast<void *>(a.rows[tensor])) +
                                               tok * a.ld[tensor] + in_row * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

}  // namespace

int launch_cache_append_fp8_block(const CacheFp8BlockArgs &a, cudaStream_t stream) {
    gda_cache_index_kernel<<<static_cast<unsigned>((a.T + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return record_cuda_error(e);
    gda_cache_append_fp8_block_kernel<<<static_cast<unsigned>(a.T), kThreads, 0, stream>>>(a);
    e = cudaGetLastError();
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

int launch_cache_read_fp8_block(const CacheFp8BlockArgs &a, cudaStream_t stream) {
    gda_cache_read_fp8_block_kernel<<<static_cast<unsigned>(a.T), kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

}  // namespace gda
