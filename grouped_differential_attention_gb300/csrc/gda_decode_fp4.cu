// Grouped differential attention decode over a 4-bit KV cache (one new query
// token per sequence; format in gda_fp4.cuh), contiguous or paged, split over
// the cache length, plus a combine pass.
//
// The batch's cache positions, concatenated sequence after sequence, are cut
// into equal contiguous ranges.  A warp takes one range for one signal head
// and the noise head it shares: online softmax of both maps (exp2 units) and
// the two accumulators O1, O2.  Each part of a range that lies in one
// sequence leaves (m, l) of both maps and (O1, O2) in workspace slot
// (range + sequence), which is unique because along the position axis
// neither index falls and one grows from part to part.  The combine kernel
// joins the parts of a sequence and applies the difference and the
// (1 - lambda_init) RMSNorm.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gda.h"
#include "gda_device.cuh"
#include "gda_fp4.cuh"
#include "gda_internal.h"

namespace gda {
namespace {

constexpr int kWarpsPerBlock = 4;
constexpr int kMaxWarps = 2048;        // warps of the split kernel at most
constexpr int kMinRange = 32;          // fewest positions of a range

struct Fp4Plan {
    int splits;        // ranges at most
    size_t ml_at, seg_at, bytes;
};

Fp4Plan plan_of(int B, int hs, int dv) {
    Fp4Plan p;
    p.splits = std::max(1, kMaxWarps / hs);
    const size_t slots = static_cast<size_t>(p.splits) + B;
    p.ml_at = (slots * hs * 2 * dv * sizeof(float) + 255) / 256 * 256;
    p.seg_at = p.ml_at + (slots * hs * 4 * sizeof(float) + 255) / 256 * 256;
    p.bytes = p.seg_at + static_cast<size_t>(B) * 2 * sizeof(int);
    return p;
}

struct Params {
    const __nv_bfloat16 *q1, *q2;
    const uint8_t *k1c, *k2c, *vc, *k1b, *k2b, *vb;
    const float *k1_scale, *k2_scale, *v_scale;
    const int *lens;
    const float *lambda;
    __nv_bfloat16 *out;
    float *ws_o;       // [slots][hs][2][dv]
    float *ws_ml;      // [slots][hs][4]: m1, l1, m2, l2
    int *ws_seg;       // [B][2]: first and last range of a sequence
    unsigned *err;
    float lambda_init, eps, scale_log2;
    int B, Lcap, hs, hn;
    int splits;
    const int *block_table;
    int page_size, max_pages, num_pages;
};

// Length of sequence b; one outside [0, Lcap] is clamped and reported.
__device__ __forceinline__ int length_of(const Params &p, int b) {
    const int len = p.lens[b];
    if (len >= 0 && len <= p.Lcap) return len;
    atomicOr(p.err, GDA_DEVERR_BAD_LENGTH);
    return len < 0 ? 0 : p.Lcap;
}

// Cache row of position pos of sequence b.  A page outside the pool is read as page 0 and reported.
__device__ __forceinline__ size_t row_of(const Params &p, int b, int pos) {
    if (p.block_table == nullptr) return static_cast<size_t>(b) * p.Lcap + pos;
    const int pg = pos / p.page_size;
    int phys = p.block_table[static_cast<size_t>(b) * p.max_pages + pg];
    if (phys < 0 || phys >= p.num_pages) {
        atomicOr(p.err, GDA_DEVERR_BAD_PAGE);
        phys = 0;
    }
    return static_cast<size_t>(phys) * p.page_size + (pos - pg * p.page_size);
}

// The range [start, end) of a split in the concatenated positions, and where it begins.
struct Range {
    long long start, end, per, before;   // before: positions of the sequences ahead of b
    int b;
};

// Computed by a whole warp; false if the split has nothing to do.
__device__ __forceinline__ bool range_of(const Params &p, int split, Range &r) {
    const int lane = threadIdx.x & 31;
    long long total = 0;
    for (int b = lane; b < p.B; b += 32) total += length_of(p, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    r.per = max(static_cast<long long>(kMinRange), (total + p.splits - 1) / p.splits);
    r.per = (r.per + 15) / 16 * 16;
    r.start = split * r.per;
    r.end = min(total, r.start + r.per);
    if (r.start >= total) return false;
    long long carry = 0;
    for (int base = 0; base < p.B; base += 32) {
        const int b = base + lane;
        const long long len = b < p.B ? length_of(p, b) : 0;
        long long incl = len;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const long long before = carry + incl - len;
        const unsigned hit = __ballot_sync(0xffffffffu, before <= r.start && r.start < before + len);
        if (hit) {
            const int src = __ffs(hit) - 1;
            r.b = base + src;
            r.before = __shfl_sync(0xffffffffu, before, src);
            return true;
        }
        carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;                         // not reached: start < total
}

// The N = D / 32 consecutive elements of a head row that belong to this lane.
template <int N>
__device__ __forceinline__ void load_lane(float (&x)[N], const uint8_t *codes, const uint8_t *blocks, int lane) {
    const float s = e4m3_to_float(blocks[lane * N / kFp4Block]);
    uint32_t w = 0;
    if constexpr (N == 2) w = codes[lane];
    if constexpr (N == 4) w = reinterpret_cast<const uint16_t *>(codes)[lane];
    if constexpr (N == 8) w = reinterpret_cast<const uint32_t *>(codes)[lane];
    uint32_t h[4];
    e2m1x8_to_half2x4(h, w);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 v = half2_bits_to_float2(h[i / 2]);
        x[i] = v.x * s;
        x[i + 1] = v.y * s;
    }
}

template <int D, int DV>
__global__ void __launch_bounds__(kWarpsPerBlock * 32) gda_decode_fp4_split_kernel(const Params p) {
    constexpr int NK = D / 32, NV = DV / 32;
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
    const int split = unit / p.hs, h = unit % p.hs, g = h / (p.hs / p.hn);
    if (split >= p.splits) return;
    Range r;
    if (!range_of(p, split, r)) return;
    long long at = r.start;
    while (at < r.end) {
        const int len = length_of(p, r.b);
        const int pos0 = static_cast<int>(at - r.before);
        const int pos1 = static_cast<int>(min(static_cast<long long>(len), r.end - r.before));
        float q1[NK], q2[NK], o1[NV] = {}, o2[NV] = {};
        const float f1 = p.scale_log2 * p.k1_scale[h], f2 = p.scale_log2 * p.k2_scale[g];
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            q1[i] = f1 * __bfloat162float(p.q1[(static_cast<size_t>(r.b) * p.hs + h) * D + lane * NK + i]);
            q2[i] = f2 * __bfloat162float(p.q2[(static_cast<size_t>(r.b) * p.hn + g) * D + lane * NK + i]);
        }
        float m1 = -INFINITY, m2 = -INFINITY, l1 = 0.f, l2 = 0.f;
        for (int pos = pos0; pos < pos1; ++pos) {
            const size_t row = row_of(p, r.b, pos);
            float k1[NK], k2[NK], v[NV];
            load_lane<NK>(k1, p.k1c + (row * p.hs + h) * (D / 2), p.k1b + (row * p.hs + h) * (D / 16), lane);
            load_lane<NK>(k2, p.k2c + (row * p.hn + g) * (D / 2), p.k2b + (row * p.hn + g) * (D / 16), lane);
            load_lane<NV>(v, p.vc + (row * p.hs + h) * (DV / 2), p.vb + (row * p.hs + h) * (DV / 16), lane);
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                s1 = fmaf(q1[i], k1[i], s1);
                s2 = fmaf(q2[i], k2[i], s2);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                s1 += __shfl_xor_sync(0xffffffffu, s1, o);
                s2 += __shfl_xor_sync(0xffffffffu, s2, o);
            }
            const float n1 = fmaxf(m1, s1), n2 = fmaxf(m2, s2);
            const float a1 = exp2f(m1 - n1), a2 = exp2f(m2 - n2), w1 = exp2f(s1 - n1), w2 = exp2f(s2 - n2);
            m1 = n1, m2 = n2;
            l1 = l1 * a1 + w1, l2 = l2 * a2 + w2;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                o1[i] = fmaf(w1, v[i], o1[i] * a1);
                o2[i] = fmaf(w2, v[i], o2[i] * a2);
            }
        }
        const size_t slot = static_cast<size_t>(split) + r.b;
        float *o = p.ws_o + (slot * p.hs + h) * 2 * DV;
        const float vs = p.v_scale[h];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            o[lane * NV + i] = o1[i] * vs;
            o[DV + lane * NV + i] = o2[i] * vs;
        }
        if (lane == 0) {
            reinterpret_cast<float4 *>(p.ws_ml)[slot * p.hs + h] = make_float4(m1, l1, m2, l2);
            if (pos0 == 0 && h == 0) {
                p.ws_seg[2 * r.b] = split;
                p.ws_seg[2 * r.b + 1] = static_cast<int>((r.before + len - 1) / r.per);
            }
        }
        at = r.before + pos1;
        r.before += len;
        ++r.b;
        while (at < r.end && length_of(p, r.b) == 0) ++r.b;
    }
}

// grid (h_s, B), block dv threads: joins the parts of one (sequence, head).
__global__ void __launch_bounds__(256) gda_decode_fp4_combine_kernel(const Params p) {
    __shared__ float red[8];
    const int h = blockIdx.x, b = blockIdx.y, col = threadIdx.x, dv = blockDim.x;
    __nv_bfloat16 *out = p.out + (static_cast<size_t>(b) * p.hs + h) * dv + col;
    if (length_of(p, b) == 0) {          // no position: the row is zero
        *out = __float2bfloat16_rn(0.f);
        return;
    }
    const int c0 = min(max(p.ws_seg[2 * b], 0), p.splits - 1);
    const int c1 = min(max(p.ws_seg[2 * b + 1], c0), p.splits - 1);
    const float4 *ml = reinterpret_cast<const float4 *>(p.ws_ml);
    float M1 = -INFINITY, M2 = -INFINITY;
    for (int c = c0; c <= c1; ++c) {
        const float4 s = ml[(static_cast<size_t>(c) + b) * p.hs + h];
        M1 = fmaxf(M1, s.x);
        M2 = fmaxf(M2, s.z);
    }
    float L1 = 0.f, L2 = 0.f, O1 = 0.f, O2 = 0.f;
    for (int c = c0; c <= c1; ++c) {
        const size_t at = (static_cast<size_t>(c) + b) * p.hs + h;
        const float4 s = ml[at];
        const float f1 = exp2f(s.x - M1), f2 = exp2f(s.z - M2);
        L1 = fmaf(s.y, f1, L1);
        L2 = fmaf(s.w, f2, L2);
        O1 = fmaf(p.ws_o[at * 2 * dv + col], f1, O1);
        O2 = fmaf(p.ws_o[(at * 2 + 1) * dv + col], f2, O2);
    }
    const float o = O1 / L1 - p.lambda[h] * (O2 / L2);
    float ss = o * o;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if ((col & 31) == 0) red[col >> 5] = ss;
    __syncthreads();
    float tot = 0.f;
    for (int w = 0; w < dv / 32; ++w) tot += red[w];
    *out = __float2bfloat16_rn((1.f - p.lambda_init) * o * rsqrtf(tot / static_cast<float>(dv) + p.eps));
}

}  // namespace

size_t decode_fp4_workspace_bytes(int B, int hs, int hn, int d, int dv) {
    (void)hn;
    (void)d;
    return plan_of(B, hs, dv).bytes;
}

int launch_decode_fp4(const DecodeFp4Args &a, cudaStream_t stream) {
    const Fp4Plan pl = plan_of(a.B, a.hs, a.dv);
    char *ws = static_cast<char *>(a.workspace);
    const Params p{static_cast<const __nv_bfloat16 *>(a.q1),
                   static_cast<const __nv_bfloat16 *>(a.q2),
                   a.k1c, a.k2c, a.vc, a.k1b, a.k2b, a.vb, a.k1_scale, a.k2_scale, a.v_scale, a.lens, a.lambda,
                   static_cast<__nv_bfloat16 *>(a.out),
                   reinterpret_cast<float *>(ws),
                   reinterpret_cast<float *>(ws + pl.ml_at),
                   reinterpret_cast<int *>(ws + pl.seg_at),
                   a.dev_err, a.lambda_init, a.eps,
                   static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a.d))),
                   a.B, a.Lcap, a.hs, a.hn, pl.splits, a.block_table, a.page_size, a.max_pages, a.num_pages};
    const int units = pl.splits * a.hs;
    const int grid = (units + kWarpsPerBlock - 1) / kWarpsPerBlock;
    void (*kern)(Params) = nullptr;
    switch (a.d * 1000 + a.dv) {
        case 64064: kern = gda_decode_fp4_split_kernel<64, 64>; break;
        case 64128: kern = gda_decode_fp4_split_kernel<64, 128>; break;
        case 64256: kern = gda_decode_fp4_split_kernel<64, 256>; break;
        case 128064: kern = gda_decode_fp4_split_kernel<128, 64>; break;
        case 128128: kern = gda_decode_fp4_split_kernel<128, 128>; break;
        case 128256: kern = gda_decode_fp4_split_kernel<128, 256>; break;
        default: return GDA_ERR_UNSUPPORTED;
    }
    kern<<<grid, kWarpsPerBlock * 32, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return record_cuda_error(e);
    gda_decode_fp4_combine_kernel<<<dim3(a.hs, a.B), a.dv, 0, stream>>>(p);
    e = cudaGetLastError();
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

}  // namespace gda
