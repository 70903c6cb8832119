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
// ceil(ceil(x / 4) / 2^k) = ceil(x / 4 / 2^k), so a growing scale keeps them exact.  A scale of the caller's own need be no
// power of two: codes brought from it are rounded up as well as down, and the bounds follow to where 4 bound would be.
//
// The rows of a block may be anywhere in the call.  The row with the lowest slot
// of a block writes all of it; to find the others, a call of few rows looks
// through the slot map, one of many takes a launch before that notes in
// index[slot] which row has that slot.  An entry counts only if that row's slot
// is this slot, so what else the workspace holds does no harm.  A row that is
// alone in its block (a decode step) is 256 elements to a warp; several are
// held by a thread block in shared memory between the two passes over them.
//
// Measured (graph replay; 12 + 4 heads of 64/128, blocks of 64): 64 rows of as
// many sequences 6.3 us, 256 10.3, 1024 22; 8192 rows of a prompt 20.5 (63 MB,
// 9.3 at the copy rate of 6793 GB/s: noting the slots 2.5, then a wave and a half
// of thread blocks, each a chain of looking up, loading and writing); reading
// 8192 rows 12.4 (63 MB).  Rows prefetched into L2 while the slots are noted:
// 22.6 with the rows there already, 25.7 for 28.8 with them in HBM, not kept.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "gda.h"
#include "gda_device.cuh"
#include "gda_fp8_block.cuh"
#include "gda_internal.h"

namespace gda {
namespace {

constexpr int kThreads = 256;          // of reading, and of noting slots
constexpr int kMaxBlock = 128;         // (a thread block has as many threads at least)
constexpr int kMaxRows = 64;           // rows of the call that a thread block looks at
constexpr int kKeep = 16;              // pieces of 8 elements that a lane holds

__global__ void __launch_bounds__(kThreads) gda_cache_index_kernel(const CacheFp8BlockArgs a) {
    const long long t = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    if (t >= a.T) return;
    const int slot = a.slot_map[t];
    if (slot >= 0 && slot < a.slots) a.index[slot] = static_cast<int>(t);
}

// The greater and the lesser of two pairs of bf16; a NaN is passed over.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 0xffff in the halves of a pair of bf16 that are infinite or NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    return ((w & 0x7fffu) >= 0x7f80u ? 0xffffu : 0u) | ((w & 0x7fff0000u) >= 0x7f800000u ? 0xffff0000u : 0u);
}

// The code of x: at most `most` in magnitude.
__device__ __forceinline__ uint32_t codes_of(float lo, float hi, float r, float most) {
    return float2_to_e4m3x2(fmaxf(-most, fminf(most, __fmul_rn(lo, r))), fmaxf(-most, fminf(most, __fmul_rn(hi, r))));
}

// Warps that share a head row of n elements: a lane's kKeep pieces of 8 then hold the whole block of tokens.
__host__ __device__ constexpr int warps_of(int block, int n) {
    return block * n <= kKeep * 8 * 32 ? 1 : block * n / (kKeep * 8 * 32);
}
__host__ __device__ constexpr int groups_of(int heads, int block, int n, int warps) {   // thread blocks for a tensor's heads
    return (heads * warps_of(block, n) + warps - 1) / warps;
}

template <int WARPS>
struct Shared {
    int place[kMaxBlock];              // the call's row of each place of the block of tokens, or -1
    int slots[kMaxRows];
    unsigned some[kMaxRows / 32];
    int one[kMaxRows], more[kMaxRows], ones, mores;   // the rows that write a block: alone, and with others
    uint32_t most[WARPS];
    uint32_t top[WARPS][64], low[WARPS][64];   // pairs of a key's channels
};
constexpr int kPieces = kKeep * 512;   // bytes of a warp's pieces

__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Eight channels' bounds of codes that are brought to a scale 1 / shift as large, where shift is no power of two: rounded
// outwards, and at least as far as the code 4 bound would come, since codes are rounded to the nearest (their order stays).
__device__ __forceinline__ void bring_bounds(uint2 &top, uint2 &low, float shift) {
    uint2 nt = {}, nl = {};
#pragma unroll 1
    for (int at = 0; at < 32; at += 8) {
        auto bring = [&](uint32_t word_t, uint32_t word_l, uint32_t &to_t, uint32_t &to_l) {
            const float t = static_cast<float>(static_cast<int8_t>(word_t >> at)), l = static_cast<float>(static_cast<int8_t>(word_l >> at));
            const uint32_t codes = float2_to_e4m3x2(__fmul_rn(4.f * t, shift), __fmul_rn(4.f * l, shift));
            const float2 far = half2_bits_to_float2(e4m3x2_to_half2(codes));
            to_t |= (static_cast<uint32_t>(static_cast<int>(fmaxf(ceilf(t * shift), ceilf(far.x * 0.25f)))) & 0xffu) << at;
            to_l |= (static_cast<uint32_t>(static_cast<int>(fminf(floorf(l * shift), floorf(far.y * 0.25f)))) & 0xffu) << at;
        };
        bring(top.x, low.x, nt.x, nl.x);
        bring(top.y, low.y, nt.y, nl.y);
    }
    top = nt, low = nl;
}
__device__ __forceinline__ bool power_of_two(float x) { return (__float_as_uint(x) & 0x7fffffu) == 0; }

// One block of tokens, the heads of this thread block: `share` warps to a head, n / 8 lanes to a row.  A lane's pieces
// go through shared memory, where no other thread reads them: that many loads are in flight without as many registers,
// in loops that need not be unrolled (a call of few rows runs once through cold instructions: unrolled over registers 64
// rows took 18 us and 8192 rows 50).
template <int WARPS>
__device__ __forceinline__ void write_heads(const CacheFp8BlockArgs &a, int tensor, int group, int blk, Shared<WARPS> &sh,
                                            uint8_t *pieces, bool fresh) {
    const int n = a.dims[tensor], log = n == 64 ? 3 : (n == 128 ? 4 : 5), lanes = 1 << log, step = 32 >> log;
    const int share = warps_of(a.block, n), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = (group * WARPS + warp) / share, member = warp % share;
    const bool here = head < a.heads[tensor];
    const int ch = (lane & (lanes - 1)) * 8, row0 = member * step + (lane >> log), stride = share * step;   // this lane's places
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.rows[tensor]) + head * n + ch;
    const size_t pitch = static_cast<size_t>(a.heads[tensor]) * n, place = static_cast<size_t>(blk) * a.heads[tensor] + head;
    uint8_t *codes = a.codes[tensor] + static_cast<size_t>(blk) * a.block * pitch + head * n + ch;
    const bool bounds_too = tensor < 2 && a.bounds[0] != nullptr;
    int8_t *const bounds = bounds_too ? a.bounds[tensor] + place * 2 * n + ch : nullptr;

    uint8_t *const mine = pieces + warp * kPieces + lane * 16;
    const uint32_t at_mine = smem_u32(mine);
    const int count = here ? (a.block - row0 + stride - 1) / stride : 0;
    unsigned have = 0;                                       // the pieces that are rows of this call
    for (int i = 0; i < count; ++i) {
        const int t = sh.place[row0 + i * stride];
        if (t < 0) continue;
        have |= 1u << i;
        copy_async16(at_mine + i * 512, x + t * a.ld[tensor]);
    }
    const float old = fresh || !here ? 0.f : a.scale[tensor][place];
    uint2 old_top = {}, old_low = {};
    if (bounds_too && here && !fresh && member == 0 && lane < lanes) {
        old_top = *reinterpret_cast<const uint2 *>(bounds);
        old_low = *reinterpret_cast<const uint2 *>(bounds + n);
    }
    copies_landed();
    // magnitudes of bf16 order like their bits; what is not finite is above all others, and then looked at once more
    const uint32_t lowest = 0xff80ff80u, highest = 0x7f807f80u;             // -inf, inf
    uint32_t top[4] = {lowest, lowest, lowest, lowest}, low[4] = {highest, highest, highest, highest};
    uint32_t both = 0;
    for (unsigned rest = have; rest != 0; rest &= rest - 1) {
        const uint4 w = *reinterpret_cast<const uint4 *>(mine + (__ffs(rest) - 1) * 512);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) both = __vmaxu2(both, v[k] & 0x7fff7fffu);
        if (bounds_too) {
#pragma unroll
            for (int k = 0; k < 4; ++k) top[k] = max_bf16x2(top[k], v[k]), low[k] = min_bf16x2(low[k], v[k]);
        }
    }
    uint32_t most = __reduce_max_sync(0xffffffffu, max(both & 0xffffu, both >> 16));
    bool odd = most >= 0x7f80u;                              // some of the warp's elements are not finite
    if (odd) {
        both = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) top[k] = lowest, low[k] = highest;
        for (unsigned rest = have; rest != 0; rest &= rest - 1) {
            const uint4 w = *reinterpret_cast<const uint4 *>(mine + (__ffs(rest) - 1) * 512);
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t no = not_finite(v[k]);
                both = __vmaxu2(both, v[k] & 0x7fff7fffu & ~no);
                top[k] = max_bf16x2(top[k], (v[k] & ~no) | (lowest & no));
                low[k] = min_bf16x2(low[k], (v[k] & ~no) | (highest & no));
            }
        }
        most = __reduce_max_sync(0xffffffffu, max(both & 0xffffu, both >> 16));
    }
    if (share > 1) {
        if (lane == 0) sh.most[warp] = most | (odd ? 0x80000000u : 0u);
        __syncthreads();
        for (int i = 0; i < share; ++i) {
            const uint32_t other = sh.most[warp - member + i];
            most = max(most, other & 0xffffu), odd |= other >> 31;
        }
    }
    const float scale = fmaxf(old, fp8_scale_of(most << 16));
    const float r = __frcp_rn(scale), shift = fresh ? 1.f : __fdiv_rn(old, scale);
    const float most_code = fminf(448.f, __fdiv_rn(0x1.ep127f, scale));
    if (here && member == 0 && lane == 0) a.scale[tensor][place] = scale;   // all have read it: they share `most`

    odd |= most_code < 448.f;
    for (unsigned rest = have; rest != 0; rest &= rest - 1) {
        const int i = __ffs(rest) - 1;
        const uint4 w = *reinterpret_cast<const uint4 *>(mine + i * 512);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
        uint32_t c[4];
        if (odd) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t no = not_finite(v[k]);        // the limits make numbers of those
                c[k] = codes_of(bf16_lo(v[k]), bf16_hi(v[k]), r, most_code) | (no & 0x7fu) | (no >> 16 & 0x7f00u);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = float2_to_e4m3x2(__fmul_rn(bf16_lo(v[k]), r), __fmul_rn(bf16_hi(v[k]), r));
        }
        *reinterpret_cast<uint2 *>(codes + (row0 + i * stride) * pitch) =
            make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
    }
    if (shift != 1.f) {                                      // the rows that are there already
        const unsigned others = ~have & (count < 32 ? (1u << count) - 1 : ~0u);
        for (unsigned rest = others; rest != 0; rest &= rest - 1) {
            const int i = __ffs(rest) - 1;
            copy_async8(at_mine + i * 512, codes + (row0 + i * stride) * pitch);
        }
        copies_landed();
        for (unsigned rest = others; rest != 0; rest &= rest - 1) {
            const int i = __ffs(rest) - 1;
            const uint2 w = *reinterpret_cast<const uint2 *>(mine + i * 512);
            const uint32_t v[2] = {w.x, w.y};
            uint32_t o[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint2 h = e4m3x4_to_half2x2(v[k]);
                const float2 p = half2_bits_to_float2(h.x), q = half2_bits_to_float2(h.y);
                o[k] = float2_to_e4m3x2(p.x * shift, p.y * shift) | float2_to_e4m3x2(q.x * shift, q.y * shift) << 16;
            }
            *reinterpret_cast<uint2 *>(codes + (row0 + i * stride) * pitch) = make_uint2(o[0], o[1]);
        }
    }
    if (!bounds_too) return;
    for (int o = lanes; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            top[k] = max_bf16x2(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
            low[k] = min_bf16x2(low[k], __shfl_xor_sync(0xffffffffu, low[k], o));
        }
    if (share > 1) {
        if (lane < lanes)
#pragma unroll
            for (int k = 0; k < 4; ++k) sh.top[warp][4 * lane + k] = top[k], sh.low[warp][4 * lane + k] = low[k];
        __syncthreads();
        if (member == 0 && lane < lanes)
            for (int i = 1; i < share; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    top[k] = max_bf16x2(top[k], sh.top[warp + i][4 * lane + k]);
                    low[k] = min_bf16x2(low[k], sh.low[warp + i][4 * lane + k]);
                }
    }
    if (!here || member != 0 || lane >= lanes) return;
    const bool odd_shift = !fresh && !power_of_two(shift);
    if (odd_shift) bring_bounds(old_top, old_low, shift);
    const float by = odd_shift ? 1.f : shift;
    uint32_t nt[2] = {0u, 0u}, nl[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        // the code of the greatest is the greatest code
        const float tx = k & 1 ? bf16_hi(top[k / 2]) : bf16_lo(top[k / 2]), lx = k & 1 ? bf16_hi(low[k / 2]) : bf16_lo(low[k / 2]);
        const float2 tl = half2_bits_to_float2(e4m3x2_to_half2(codes_of(tx, lx, r, most_code)));
        const bool none = tx < lx;                           // no finite value
        float t = none ? -128.f : ceilf(tl.x * 0.25f), l = none ? 127.f : floorf(tl.y * 0.25f);
        if (!fresh) {
            const uint32_t ot = (k < 4 ? old_top.x : old_top.y) >> 8 * (k & 3);
            const uint32_t ol = (k < 4 ? old_low.x : old_low.y) >> 8 * (k & 3);
            t = fmaxf(t, ceilf(static_cast<float>(static_cast<int8_t>(ot)) * by));
            l = fminf(l, floorf(static_cast<float>(static_cast<int8_t>(ol)) * by));
        }
        nt[k / 4] |= (static_cast<uint32_t>(static_cast<int>(t)) & 0xffu) << 8 * (k & 3);
        nl[k / 4] |= (static_cast<uint32_t>(static_cast<int>(l)) & 0xffu) << 8 * (k & 3);
    }
    *reinterpret_cast<uint2 *>(bounds) = make_uint2(nt[0], nt[1]);
    *reinterpret_cast<uint2 *>(bounds + n) = make_uint2(nl[0], nl[1]);
}

// 256 elements of a row that is the only one of its block, 8 to a lane (a head is n / 8 lanes): what is read of them.
struct Piece {
    uint4 w;
    uint2 old_top, old_low;
    float old;
    int tensor, slot, head, ch;
    bool here;
};

__device__ __forceinline__ Piece fetch_piece(const CacheFp8BlockArgs &a, long long t, int slot, int piece) {
    Piece p{};
    for (; p.tensor < 2; ++p.tensor) {
        const int of = (a.heads[p.tensor] * a.dims[p.tensor] + 255) / 256;
        if (piece < of) break;
        piece -= of;
    }
    const int n = a.dims[p.tensor], e = piece * 256 + (threadIdx.x & 31) * 8;
    p.slot = slot;
    p.head = e / n, p.ch = e & (n - 1);
    p.here = p.head < a.heads[p.tensor];
    if (!p.here) return p;
    p.w = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.rows[p.tensor]) + t * a.ld[p.tensor] + e);
    if ((slot & (a.block - 1)) == 0) return p;               // the block begins: nothing of it is read
    const size_t place = static_cast<size_t>(slot / a.block) * a.heads[p.tensor] + p.head;
    p.old = a.scale[p.tensor][place];
    if (p.tensor == 2 || a.bounds[0] == nullptr) return p;
    const int8_t *bounds = a.bounds[p.tensor] + place * 2 * n + p.ch;
    p.old_top = *reinterpret_cast<const uint2 *>(bounds);
    p.old_low = *reinterpret_cast<const uint2 *>(bounds + n);
    return p;
}

// The greatest and the least of bounds, for 8 channels: those before, brought to the scale, and codes of one row.
__device__ __forceinline__ void join_bounds(uint2 &top, uint2 &low, const uint32_t (&c)[4], float shift, bool fresh) {
    if (!fresh && !power_of_two(shift)) bring_bounds(top, low, shift), shift = 1.f;
    uint32_t nt[2] = {0u, 0u}, nl[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 pair = half2_bits_to_float2(e4m3x2_to_half2(c[k / 2]));
        const float v = k & 1 ? pair.y : pair.x;
        float t = v == v ? ceilf(v * 0.25f) : -128.f, l = v == v ? floorf(v * 0.25f) : 127.f;
        if (!fresh) {
            const uint32_t ot = (k < 4 ? top.x : top.y) >> 8 * (k & 3), ol = (k < 4 ? low.x : low.y) >> 8 * (k & 3);
            t = fmaxf(t, ceilf(static_cast<float>(static_cast<int8_t>(ot)) * shift));
            l = fminf(l, floorf(static_cast<float>(static_cast<int8_t>(ol)) * shift));
        }
        nt[k / 4] |= (static_cast<uint32_t>(static_cast<int>(t)) & 0xffu) << 8 * (k & 3);
        nl[k / 4] |= (static_cast<uint32_t>(static_cast<int>(l)) & 0xffu) << 8 * (k & 3);
    }
    top = make_uint2(nt[0], nt[1]), low = make_uint2(nl[0], nl[1]);
}

__device__ __forceinline__ void write_piece(const CacheFp8BlockArgs &a, Piece &p) {
    const int n = a.dims[p.tensor], in_block = p.slot & (a.block - 1);
    const bool fresh = in_block == 0;
    const uint32_t v[4] = {p.w.x, p.w.y, p.w.z, p.w.w};
    uint32_t no[4], both = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) no[k] = not_finite(v[k]), both = __vmaxu2(both, v[k] & 0x7fff7fffu & ~no[k]);
    uint32_t most = max(both & 0xffffu, both >> 16);
    for (int o = 1; o < n / 8; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    const float scale = fmaxf(p.old, fp8_scale_of(most << 16)), r = __frcp_rn(scale);
    const float shift = fresh ? 1.f : __fdiv_rn(p.old, scale), most_code = fminf(448.f, __fdiv_rn(0x1.ep127f, scale));
    if (!p.here) return;
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)                              // the limits make numbers of what is none
        c[k] = codes_of(bf16_lo(v[k]), bf16_hi(v[k]), r, most_code) | (no[k] & 0x7fu) | (no[k] >> 16 & 0x7f00u);
    const size_t pitch = static_cast<size_t>(a.heads[p.tensor]) * n, blk = p.slot / a.block;
    uint8_t *const codes = a.codes[p.tensor] + blk * a.block * pitch + p.head * n + p.ch;
    *reinterpret_cast<uint2 *>(codes + in_block * pitch) =
        make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
    if (p.ch == 0) a.scale[p.tensor][blk * a.heads[p.tensor] + p.head] = scale;
    if (shift != 1.f) {                                      // the rows that are there already
        for (int base = 0; base < a.block; base += 8) {
            uint2 was[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) was[i] = *reinterpret_cast<const uint2 *>(codes + (base + i) * pitch);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t x[2] = {was[i].x, was[i].y};
                uint32_t o[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint2 h = e4m3x4_to_half2x2(x[k]);
                    const float2 y = half2_bits_to_float2(h.x), z = half2_bits_to_float2(h.y);
                    o[k] = float2_to_e4m3x2(y.x * shift, y.y * shift) | float2_to_e4m3x2(z.x * shift, z.y * shift) << 16;
                }
                if (base + i != in_block) *reinterpret_cast<uint2 *>(codes + (base + i) * pitch) = make_uint2(o[0], o[1]);
            }
        }
    }
    if (p.tensor == 2 || a.bounds[0] == nullptr) return;
    join_bounds(p.old_top, p.old_low, c, shift, fresh);
    int8_t *const bounds = a.bounds[p.tensor] + (blk * a.heads[p.tensor] + p.head) * 2 * n + p.ch;
    *reinterpret_cast<uint2 *>(bounds) = p.old_top;
    *reinterpret_cast<uint2 *>(bounds + n) = p.old_low;
}

// The rows of a call in the block of tokens from slot `first` on, a bit for each place; a whole warp.  `wins`: row t is
// the one that is written to its place.  SCAN: they are looked for in the slot map.
template <bool SCAN>
__device__ __forceinline__ void members_of(const CacheFp8BlockArgs &a, int first, int in_block, long long t, uint32_t (&m)[4],
                                           int (&rows)[4], bool &wins) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 0; w < 4; ++w) m[w] = 0;
    wins = false;
    if constexpr (SCAN) {
        int last = -1;                                       // of two rows with one slot the later one is written
#pragma unroll 4
        for (int i = lane; i < a.T; i += 32) {
            const unsigned at = static_cast<unsigned>(a.slot_map[i]) - static_cast<unsigned>(first);
            if (at < static_cast<unsigned>(a.block)) {
#pragma unroll
                for (int w = 0; w < 4; ++w) m[w] |= static_cast<int>(at >> 5) == w ? 1u << (at & 31) : 0u;
                if (static_cast<int>(at) == in_block) last = i;
            }
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) m[w] = __reduce_or_sync(0xffffffffu, m[w]);
        wins = __reduce_max_sync(0xffffffffu, last) == t;
    } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int at = 32 * w + lane;
            const int i = at < a.block ? a.index[first + at] : -1;
            const bool there = i >= 0 && i < a.T && a.slot_map[i] == first + at;
            rows[w] = there ? i : -1;                        // of this lane's places
            m[w] = __ballot_sync(0xffffffffu, there);
            wins |= __any_sync(0xffffffffu, there && at == in_block && i == t);
        }
    }
}

// grid (groups of `per` rows of the call, groups of heads).
template <bool SCAN, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) gda_cache_append_fp8_block_kernel(const CacheFp8BlockArgs a, int per) {
    __shared__ Shared<WARPS> sh;
    extern __shared__ __align__(16) uint8_t pieces[];        // [WARPS][kKeep][32][16]
    const long long t0 = static_cast<long long>(blockIdx.x) * per;
    const int warp = threadIdx.x >> 5;
    if constexpr (!SCAN) asm volatile("griddepcontrol.wait;" ::: "memory");   // the index is written
    if (threadIdx.x < kMaxRows) {                            // the rows that may have the lowest slot of a block
        const long long t = t0 + threadIdx.x;
        const bool mine = static_cast<int>(threadIdx.x) < per && t < a.T;
        const int slot = mine ? a.slot_map[t] : -1;
        bool may = slot >= 0 && slot < a.slots;
        if (slot >= a.slots && blockIdx.y == 0) atomicOr(a.dev_err, GDA_DEVERR_BAD_PAGE);
        // most rows of a prompt have the slot after that of the row before
        if (may && (slot & (a.block - 1)) != 0 && t > 0 && a.slot_map[t - 1] == slot - 1) may = false;
        if constexpr (!SCAN) {
            // and some other row has it where the rows come in any order
            if (may && (slot & (a.block - 1)) != 0) {
                const int i = a.index[slot - 1];
                if (i >= 0 && i < a.T && a.slot_map[i] == slot - 1) may = false;
            }
        }
        sh.slots[threadIdx.x] = slot;
        const unsigned mask = __ballot_sync(0xffffffffu, may);
        if (threadIdx.x % 32 == 0) sh.some[threadIdx.x / 32] = mask;
        if (threadIdx.x == 0) sh.ones = sh.mores = 0;
    }
    __syncthreads();
    int nth = 0;                                             // which of them have it, a warp to a row
    for (uint64_t rest = sh.some[0] | static_cast<uint64_t>(sh.some[1]) << 32; rest != 0; rest &= rest - 1) {
        if (nth++ % WARPS != warp) continue;
        const int step = __ffsll(static_cast<long long>(rest)) - 1, slot = sh.slots[step], in_block = slot & (a.block - 1);
        uint32_t m[4];
        int rows[4];
        bool wins;
        members_of<SCAN>(a, slot - in_block, in_block, t0 + step, m, rows, wins);
        const int w = in_block >> 5;
        const uint32_t below = (w > 0 ? m[0] : 0u) | (w > 1 ? m[1] : 0u) | (w > 2 ? m[2] : 0u) |
                               ((w == 0 ? m[0] : (w == 1 ? m[1] : (w == 2 ? m[2] : m[3]))) & ((1u << (in_block & 31)) - 1));
        if (!wins || below != 0) continue;
        const bool alone = __popc(m[0]) + __popc(m[1]) + __popc(m[2]) + __popc(m[3]) == 1;
        int k = 0;
        if ((threadIdx.x & 31) == 0) {
            k = atomicAdd(alone ? &sh.ones : &sh.mores, 1);
            (alone ? sh.one : sh.more)[k] = step;
        }
        k = __shfl_sync(0xffffffffu, k, 0);
        if (!SCAN && !alone && k == 0) {                     // the first one's rows are known already
#pragma unroll
            for (int i = 0; i < 4; ++i) sh.place[32 * i + (threadIdx.x & 31)] = rows[i];
        }
    }
    __syncthreads();

    // rows that are alone in their blocks, as in a decode step: a warp to 256 elements, the next ones on their way
    int total = 0;
    for (int t = 0; t < 3; ++t) total += (a.heads[t] * a.dims[t] + 255) / 256;
    const int lo = total * static_cast<int>(blockIdx.y) / static_cast<int>(gridDim.y);
    const int own = total * (static_cast<int>(blockIdx.y) + 1) / static_cast<int>(gridDim.y) - lo, tasks = sh.ones * own;
    auto fetch = [&](int i) {
        const int step = sh.one[i / own];
        return fetch_piece(a, t0 + step, sh.slots[step], lo + i % own);
    };
    if (warp < tasks) {
        Piece now = fetch(warp);
        for (int i = warp; i < tasks; i += WARPS) {
            Piece next{};
            if (i + WARPS < tasks) next = fetch(i + WARPS);
            write_piece(a, now);
            now = next;
        }
    }

    for (int k = 0; k < sh.mores; ++k) {                     // the same for the whole thread block
        const int slot = sh.slots[sh.more[k]], in_block = slot & (a.block - 1), first = slot - in_block, blk = slot / a.block;
        if (SCAN || k > 0) {
            if (k > 0) __syncthreads();                      // the readers of `place` are done
            if constexpr (SCAN) {
                if (threadIdx.x < kMaxBlock) sh.place[threadIdx.x] = -1;
                __syncthreads();
                for (int i = threadIdx.x; i < a.T; i += WARPS * 32) {
                    const unsigned other = static_cast<unsigned>(a.slot_map[i]) - static_cast<unsigned>(first);
                    if (other < static_cast<unsigned>(a.block)) atomicMax(&sh.place[other], i);
                }
            } else if (threadIdx.x < a.block) {
                const int i = a.index[first + threadIdx.x];
                sh.place[threadIdx.x] = i >= 0 && i < a.T && a.slot_map[i] == first + static_cast<int>(threadIdx.x) ? i : -1;
            }
            __syncthreads();
        }
        const bool fresh = sh.place[0] >= 0;
        int group = blockIdx.y, tensor = 0;
        for (; tensor < 2; ++tensor) {
            const int of = groups_of(a.heads[tensor], a.block, a.dims[tensor], WARPS);
            if (group < of) break;
            group -= of;
        }
        write_heads(a, tensor, group, blk, sh, pieces, fresh);
    }
}

// c * s towards zero, the last digit set where digits are lost: rounded to bf16 after that, the product is rounded once.
// (A code's 4 digits and a scale's 24 are more than float32 has; with scales that are powers of two nothing is lost.  8192
// rows in a row of graph nodes 10.3 us without it, 10.4 with a branch around the loop, 10.6 with one inside.)
__device__ __forceinline__ float product_to_odd(float c, float s) {
    const float p = __fmul_rz(c, s), rest = __fmaf_ru(fabsf(c), s, -fabsf(p));
    return rest > 0.f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
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
        if (__builtin_expect(power_of_two(s), 1)) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint2 h = e4m3x4_to_half2x2(w[k]);
                const float2 p = half2_bits_to_float2(h.x), q = half2_bits_to_float2(h.y);
                o[2 * k] = pack_bf16x2(__fmul_rn(p.x, s), __fmul_rn(p.y, s));
                o[2 * k + 1] = pack_bf16x2(__fmul_rn(q.x, s), __fmul_rn(q.y, s));
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint2 h = e4m3x4_to_half2x2(w[k]);
                const float2 p = half2_bits_to_float2(h.x), q = half2_bits_to_float2(h.y);
                o[2 * k] = pack_bf16x2(product_to_odd(p.x, s), product_to_odd(p.y, s));
                o[2 * k + 1] = pack_bf16x2(product_to_odd(q.x, s), product_to_odd(q.y, s));
            }
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

template <bool SCAN, int WARPS>
cudaError_t launch_append(const CacheFp8BlockArgs &a, cudaStream_t stream) {
    unsigned groups = 0;
    for (int t = 0; t < 3; ++t) groups += groups_of(a.heads[t], a.block, a.dims[t], WARPS);
    // Rows of a thread block: the rows of a prompt but one in a block are passed over at once, so there are more where
    // blocks are longer.  us of the call with T block / 8192, / 16384: 8192 rows of a prompt, blocks of 64 20.5 / 22.6, in
    // any order 36.6 / 31.1; 256 rows of 256 blocks 10.4 / 12.4.  Nine pieces of 227 rows, blocks of 16, with the rows read
    // back: 33 with the first (three rows) and 29 with T / 256.
    const int per = static_cast<int>(
        std::min<long long>(kMaxRows, std::max<long long>(1, std::max<long long>(a.T / 256, a.T * a.block / 8192))));
    constexpr auto kern = gda_cache_append_fp8_block_kernel<SCAN, WARPS>;
    const cudaError_t e = allow_shared_memory<kern>(WARPS * kPieces);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((a.T + per - 1) / per), groups);
    cfg.blockDim = dim3(WARPS * 32);
    cfg.dynamicSmemBytes = WARPS * kPieces;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SCAN ? 0 : 1;                             // after the index kernel only: others may write what is read here
    return cudaLaunchKernelEx(&cfg, kern, a, per);
}

}  // namespace

int launch_cache_append_fp8_block(const CacheFp8BlockArgs &a, cudaStream_t stream) {
    const bool scan = a.T <= kCacheScanRows;
    if (!scan) {
        gda_cache_index_kernel<<<static_cast<unsigned>((a.T + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return record_cuda_error(e);
    }
    // Warps of a thread block: four, unless more share a head (blocks of 128 at dim 256).  us of the call with four / eight:
    // 8192 rows of a prompt, blocks of 64 20.5 / 22.6, of 16 25.0 / 31.0; nine pieces of 227 rows of 128/256 18.9 / 20.8;
    // 8192 rows of as many blocks 102 / 97.
    const bool four = warps_of(a.block, std::max(a.dims[0], a.dims[2])) <= 4;
    const cudaError_t e = four ? (scan ? launch_append<true, 4>(a, stream) : launch_append<false, 4>(a, stream))
                               : (scan ? launch_append<true, 8>(a, stream) : launch_append<false, 8>(a, stream));
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
