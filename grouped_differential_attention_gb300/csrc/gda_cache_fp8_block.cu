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
// The rows of a block may be anywhere in the call.  The row with the lowest slot
// of a block writes all of it; to find the others, a call of few rows looks
// through the slot map, one of many takes a launch before that notes in
// index[slot] which row has that slot.  An entry counts only if that row's slot
// is this slot, so what else the workspace holds does no harm.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "gda.h"
#include "gda_device.cuh"
#include "gda_fp8_block.cuh"
#include "gda_internal.h"

namespace gda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlock = 128;
constexpr int kScanRows = 1024;        // a call of at most so many rows needs no index
constexpr int kHeadsPerBlock = 8;      // heads that a thread block writes: one for each warp
constexpr int kMaxRows = 32;           // rows of the call that a thread block looks at

__global__ void __launch_bounds__(kThreads) gda_cache_index_kernel(const CacheFp8BlockArgs a) {
    const long long t = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    if (t >= a.T) return;
    const int slot = a.slot_map[t];
    if (slot >= 0 && slot < a.slots) a.index[slot] = static_cast<int>(t);
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

// The rows of a call that go into one block of tokens: what[k] = the row's place in the block, rows[k] = the row.
struct Members {
    int rows[kMaxBlock];
    short what[kMaxBlock];
    int place[kMaxBlock];              // the row of each place, or -1
    int count;
};

// One warp, one (block, head): N / 8 lanes to a row, KEEP rows of a lane held between the two passes over them.
template <int N>
__device__ void write_head(const CacheFp8BlockArgs &a, int tensor, int head, int blk, const Members &in, bool fresh) {
    constexpr int LANES = N / 8, STEP = 32 / LANES, KEEP = 8;
    const int lane = threadIdx.x & 31, sub = lane / LANES, ch = lane % LANES * 8, count = in.count;
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.rows[tensor]) + head * N + ch;
    const long long ld = a.ld[tensor];
    const size_t pitch = static_cast<size_t>(a.heads[tensor]) * N;
    uint8_t *codes = a.codes[tensor] + static_cast<size_t>(blk) * a.block * pitch + head * N + ch;
    float *const where = a.scale[tensor] + static_cast<size_t>(blk) * a.heads[tensor] + head;
    const float old = fresh ? 0.f : *where;

    uint4 w[KEEP];
    auto load = [&](int base) {                              // rows base + sub + STEP * 0 .. KEEP - 1
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int k = base + sub + i * STEP;
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (k < count) w[i] = *reinterpret_cast<const uint4 *>(x + in.rows[k] * ld);
        }
    };
    constexpr int BATCH = KEEP * STEP;
    uint32_t most = 0;
    int base = 0;
    for (;; base += BATCH) {
        load(base);
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) most = max(most, max(finite_abs(v[k] << 16), finite_abs(v[k] & 0xffff0000u)));
        }
        if (base + BATCH >= count) break;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    const float scale = fmaxf(old, fp8_scale_of(most));
    const float r = __frcp_rn(scale), shift = fresh ? 1.f : __fdiv_rn(old, scale);
    const float most_code = fminf(448.f, __fdiv_rn(0x1.ep127f, scale));
    __syncwarp();
    if (lane == 0) *where = scale;

    const bool bounds_too = tensor < 2 && a.bounds[0] != nullptr;
    const uint32_t none_max = 0xfc00fc00u, none_min = 0x7c007c00u;   // -inf, inf
    uint32_t top[4] = {none_max, none_max, none_max, none_max}, low[4] = {none_min, none_min, none_min, none_min};
    for (;; base -= BATCH) {                                 // the batch that is still here first
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int row = base + sub + i * STEP;
            if (row >= count) continue;
            const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float lo = bf16_lo(v[k]), hi = bf16_hi(v[k]);
                c[k] = float2_to_e4m3x2(fmaxf(-most_code, fminf(most_code, __fmul_rn(lo, r))),
                                        fmaxf(-most_code, fminf(most_code, __fmul_rn(hi, r))));
                // the limits have made a number of what is none
                if ((v[k] & 0x7fffu) >= 0x7f80u) c[k] |= 0x7fu;
                if ((v[k] & 0x7fff0000u) >= 0x7f800000u) c[k] |= 0x7f00u;
                if (bounds_too) {
                    const uint32_t h = e4m3x2_to_half2(c[k]);    // a NaN is passed over by max and min
                    top[k] = hmax2(top[k], h);
                    low[k] = hmin2(low[k], h);
                }
            }
            *reinterpret_cast<uint2 *>(codes + in.what[row] * pitch) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
        }
        if (base == 0) break;
        load(base - BATCH);
    }
    if (shift != 1.f) {                                      // the rows that are there already
        for (int i = sub; i < a.block; i += STEP) {
            if (in.place[i] >= 0) continue;
            uint2 *const dst = reinterpret_cast<uint2 *>(codes + i * pitch);
            const uint2 c = *dst;
            const uint32_t v[2] = {c.x, c.y};
            uint32_t o[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint2 h = e4m3x4_to_half2x2(v[k]);
                const float2 p = half2_bits_to_float2(h.x), q = half2_bits_to_float2(h.y);
                o[k] = float2_to_e4m3x2(p.x * shift, p.y * shift) | float2_to_e4m3x2(q.x * shift, q.y * shift) << 16;
            }
            *dst = make_uint2(o[0], o[1]);
        }
    }
    if (!bounds_too) return;
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

// grid (groups of `per` rows of the call, groups of kHeadsPerBlock heads).  SCAN: members are looked for in the slot map.
template <bool SCAN>
__global__ void __launch_bounds__(kThreads) gda_cache_append_fp8_block_kernel(const CacheFp8BlockArgs a, int per) {
    __shared__ Members in;
    __shared__ int slots[kMaxRows];
    __shared__ unsigned some;
    const long long t0 = static_cast<long long>(blockIdx.x) * per;
    const int warp = threadIdx.x >> 5, heads = a.heads[0] + a.heads[1] + a.heads[2];
    if (warp == 0) {                                         // the rows that may have the lowest slot of a block
        const long long t = t0 + threadIdx.x;
        const bool mine = static_cast<int>(threadIdx.x) < per && t < a.T;
        const int slot = mine ? a.slot_map[t] : -1;
        bool may = slot >= 0 && slot < a.slots;
        if (slot >= a.slots && blockIdx.y == 0) atomicOr(a.dev_err, GDA_DEVERR_BAD_PAGE);
        // most rows of a prompt have the slot after that of the row before
        if (may && (slot & (a.block - 1)) != 0 && t > 0 && a.slot_map[t - 1] == slot - 1) may = false;
        slots[threadIdx.x] = slot;
        const unsigned mask = __ballot_sync(0xffffffffu, may);
        if (threadIdx.x == 0) some = mask;
    }
    __syncthreads();
    for (unsigned rest = some; rest != 0; rest &= rest - 1) {    // a step is the same for the whole thread block
        const int step = __ffs(rest) - 1, slot = slots[step];
        const long long t = t0 + step;
        const int in_block = slot & (a.block - 1), first = slot - in_block, blk = slot / a.block;
        if (rest != some) __syncthreads();                   // the readers of `in` are done
        if (threadIdx.x < kMaxBlock) in.place[threadIdx.x] = -1;
        if (threadIdx.x == 0) in.count = 0;
        __syncthreads();
        if constexpr (SCAN) {
            for (int i = threadIdx.x; i < a.T; i += kThreads) {
                const unsigned other = static_cast<unsigned>(a.slot_map[i]) - static_cast<unsigned>(first);
                if (other < static_cast<unsigned>(a.block)) atomicMax(&in.place[other], i);
            }
        } else if (threadIdx.x < a.block) {
            const int i = a.index[first + threadIdx.x];
            if (i >= 0 && i < a.T && a.slot_map[i] == first + static_cast<int>(threadIdx.x)) in.place[threadIdx.x] = i;
        }
        __syncthreads();
        bool lower = false;
        if (threadIdx.x < a.block) {
            const int i = in.place[threadIdx.x];
            lower = threadIdx.x < in_block ? i >= 0 : threadIdx.x == in_block && i != t;   // two rows, one slot: one is written
            if (i >= 0) {
                const int k = atomicAdd(&in.count, 1);
                in.rows[k] = i, in.what[k] = static_cast<short>(threadIdx.x);
            }
        }
        if (__syncthreads_or(lower)) continue;
        const bool fresh = in.place[0] >= 0;
        const int i = blockIdx.y * kHeadsPerBlock + warp;
        if (i >= heads) continue;
        const int tensor = i < a.heads[0] ? 0 : (i < a.heads[0] + a.heads[1] ? 1 : 2);
        const int head = i - (tensor > 0 ? a.heads[0] : 0) - (tensor > 1 ? a.heads[1] : 0);
        const int n = a.dims[tensor];
        if (n == 64) write_head<64>(a, tensor, head, blk, in, fresh);
        else if (n == 128) write_head<128>(a, tensor, head, blk, in, fresh);
        else write_head<256>(a, tensor, head, blk, in, fresh);
    }
}

// A thread's token and its 16 elements of the token's row: `tokens` tokens to a thread block (32-bit division).
__global__ void __launch_bounds__(kThreads) gda_cache_read_fp8_block_kernel(const CacheFp8BlockArgs a, unsigned tokens) {
    const unsigned n0 = a.heads[0] * a.dims[0] / 16, n1 = a.heads[1] * a.dims[1] / 16, n2 = a.heads[2] * a.dims[2] / 16;
    const unsigned per_token = n0 + n1 + n2, i = blockIdx.y * kThreads + threadIdx.x, of = i / per_token;
    const long long tok = static_cast<long long>(blockIdx.x) * tokens + of;
    if (of >= tokens || tok >= a.T) return;
    unsigned in_row = i - of * per_token;
    int tensor = 0;
    if (in_row >= n0) tensor = 1, in_row -= n0;
    if (tensor == 1 && in_row >= n1) tensor = 2, in_row -= n1;
    const int slot = a.slot_map[tok];
    uint32_t o[8] = {};
    if (slot >= a.slots) {
        atomicOr(a.dev_err, GDA_DEVERR_BAD_PAGE);
    } else if (slot >= 0) {
        const unsigned dim = a.dims[tensor], shift = dim == 64 ? 2 : (dim == 128 ? 3 : 4);   // pieces of a head row
        const size_t pitch = static_cast<size_t>(a.heads[tensor]) * dim;
        const uint4 c = *reinterpret_cast<const uint4 *>(a.codes[tensor] + slot * pitch + in_row * 16);
        const float s = a.scale[tensor][static_cast<size_t>(static_cast<unsigned>(slot) / static_cast<unsigned>(a.block)) *
                                        a.heads[tensor] + (in_row >> shift)];
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

// Thread blocks of kThreads pieces of 16 elements: over groups of as many tokens as fill them best (x), and the pieces
// of a group (y).
dim3 read_grid(const CacheFp8BlockArgs &a, unsigned *tokens) {
    unsigned per_token = 0;
    for (int t = 0; t < 3; ++t) per_token += a.heads[t] * a.dims[t] / 16;
    *tokens = 1;
    unsigned waste = kThreads;                       // idle threads, relative to the group's work
    for (unsigned t = 1; t <= 8; ++t) {
        const unsigned idle = (kThreads - t * per_token % kThreads) % kThreads;
        if (idle * *tokens < waste * t) *tokens = t, waste = idle;
    }
    return dim3(static_cast<unsigned>((a.T + *tokens - 1) / *tokens), (*tokens * per_token + kThreads - 1) / kThreads);
}

}  // namespace

int launch_cache_append_fp8_block(const CacheFp8BlockArgs &a, cudaStream_t stream) {
    const unsigned heads = (a.heads[0] + a.heads[1] + a.heads[2] + kHeadsPerBlock - 1) / kHeadsPerBlock;
    const bool scan = a.T <= kScanRows;
    // rows of a thread block: the rows of a prompt but one in a block are passed over at once
    const int per = static_cast<int>(std::min<long long>(kMaxRows, std::max<long long>(1, a.T / 256)));
    const dim3 grid(static_cast<unsigned>((a.T + per - 1) / per), heads);
    if (scan) {
        gda_cache_append_fp8_block_kernel<true><<<grid, kThreads, 0, stream>>>(a, per);
    } else {
        gda_cache_index_kernel<<<static_cast<unsigned>((a.T + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return record_cuda_error(e);
        gda_cache_append_fp8_block_kernel<false><<<grid, kThreads, 0, stream>>>(a, per);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

int launch_cache_read_fp8_block(const CacheFp8BlockArgs &a, cudaStream_t stream) {
    unsigned tokens = 0;
    const dim3 grid = read_grid(a, &tokens);
    gda_cache_read_fp8_block_kernel<<<grid, kThreads, 0, stream>>>(a, tokens);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

}  // namespace gda
