// C ABI of libgda.so (declared in include/gda.h): argument validation,
// device checks, TMA descriptor encoding and dispatch to the kernels.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>

#include "gda.h"
#include "gda_internal.h"

// Device error word (one per device that loads the library).  Kernels set
// GDA_DEVERR_* bits here instead of trapping.
__device__ unsigned g_gda_device_error;

namespace gda {
namespace {

constexpr int kMaxDevices = 64;

struct DeviceState {
    std::once_flag once;
    int status = GDA_ERR_CUDA;     // GDA_OK once the device checked out
    unsigned *err_word = nullptr;  // device address of g_gda_device_error
};
DeviceState g_dev[kMaxDevices];

// Checks the current device once: compute capability 10.3 (GB300) and the
// address of the error word.  Returns a gda_status and the word's address.
int current_device(unsigned **err_word) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return GDA_ERR_CUDA;
    }
    DeviceState &s = g_dev[dev];
    std::call_once(s.once, [&s, dev]() {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
            cudaGetLastError();
            s.status = GDA_ERR_CUDA;
            return;
        }
        if (major != 10 || minor != 3) {
            s.status = GDA_ERR_UNSUPPORTED;
            return;
        }
        void *addr = nullptr;
        if (cudaGetSymbolAddress(&addr, g_gda_device_error) != cudaSuccess) {
            cudaGetLastError();
            s.status = GDA_ERR_CUDA;
            return;
        }
        s.err_word = static_cast<unsigned *>(addr);
        s.status = GDA_OK;
    });
    *err_word = s.err_word;
    return s.status;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_prefill_common(const void *q1, const void *k1, const void *q2, const void *k2,
                         const void *v, const float *lam, float lambda_init, const void *out, int B,
                         int L, int hs, int hn, int d, int dv, int causal, float eps,
                         unsigned flags, unsigned allowed_flags = GDA_FLAG_NO_NORM) {
    if (!q1 || !k1 || !q2 || !k2 || !v || !lam || !out) return GDA_ERR_INVALID_ARG;
    if (B < 1 || L < 1 || hs < 1 || hn < 1 || d < 1 || dv < 1) return GDA_ERR_INVALID_ARG;
    if (hs % hn != 0) return GDA_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return GDA_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(lambda_init)) return GDA_ERR_INVALID_ARG;
    if (flags & ~allowed_flags) return GDA_ERR_INVALID_ARG;
    // element counts must fit the 64-bit index arithmetic with room to spare
    const double elems = static_cast<double>(B) * L * (hs > hn ? hs : hn) * (d > dv ? d : dv);
    if (elems > 9.0e15) return GDA_ERR_INVALID_ARG;
    if (!aligned16(q1) || !aligned16(k1) || !aligned16(q2) || !aligned16(k2) || !aligned16(v) ||
        !aligned16(lam) || !aligned16(out))
        return GDA_ERR_MISALIGNED;
    return GDA_OK;
}

thread_local int g_last_cuda_error = 0;

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

}  // namespace

int device_state(unsigned **err_word) { return current_device(err_word); }

int record_cuda_error(cudaError_t e) {
    g_last_cuda_error = static_cast<int>(e);
    cudaGetLastError();   // do not leak a launch error into the caller's next check
    return GDA_ERR_CUDA;
}

namespace {

// The driver's tensor map encoder, or nullptr.
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    std::call_once(g_encode_once, []() {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
        else
            cudaGetLastError();
    });
    return g_encode;
}

}  // namespace

bool encode_tmap_4d_bf16(CUtensorMap *map, const void *base, const uint64_t dims[4],
                         const uint64_t strides_bytes[3], const uint32_t box[4]) {
    const auto encode = encoder();
    if (!encode) return false;
    cuuint64_t gdim[4] = {dims[0], dims[1], dims[2], dims[3]};
    cuuint64_t gstr[3] = {strides_bytes[0], strides_bytes[1], strides_bytes[2]};
    cuuint32_t bdim[4] = {box[0], box[1], box[2], box[3]};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), gdim,
                              gstr, bdim, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

bool encode_tmap_3d_u8(CUtensorMap *map, const void *base, const uint64_t dims[3], const uint64_t strides_bytes[2],
                       const uint32_t box[3], int swizzle, bool narrow) {
    const auto encode = encoder();
    if (!encode) return false;
    const cuuint64_t gdim[3] = {dims[0], dims[1], dims[2]}, gstr[2] = {strides_bytes[0], strides_bytes[1]};
    const cuuint32_t bdim[3] = {box[0], box[1], box[2]}, estr[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), gdim, gstr, bdim, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE,
                              swizzle == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                              : swizzle == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                              : CU_TENSOR_MAP_SWIZZLE_NONE,
                              narrow ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

namespace {

const uint8_t *bytes_of(const void *p) { return static_cast<const uint8_t *>(p); }

// Whether hs + hn (both positive) is above `most`; the sum itself may not fit an int.
bool heads_above(int hs, int hn, int most) { return hs > most || hn > most - hs; }

// Arguments that both decodes over a 4-bit cache check; `rows`: rows of the caches.
int check_decode_fp4(const void *const (&ptrs)[9], const float *k1_scale, const float *k2_scale,
                     const float *v_scale, const int *lens, const float *lambda, float lambda_init, int B, int Lcap,
                     int hs, int hn, int d, int dv, float eps, double rows, const void *workspace,
                     size_t workspace_bytes) {
    for (const void *p : ptrs)
        if (!p) return GDA_ERR_INVALID_ARG;
    if (!k1_scale || !k2_scale || !v_scale || !lens || !lambda) return GDA_ERR_INVALID_ARG;
    if (B < 1 || Lcap < 1 || hs < 1 || hn < 1 || d < 1 || dv < 1 || hs % hn != 0) return GDA_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(lambda_init)) return GDA_ERR_INVALID_ARG;
    if (rows * hs * (d > dv ? d : dv) > 9.0e15) return GDA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128) || !(dv == 64 || dv == 128 || dv == 256)) return GDA_ERR_UNSUPPORTED;
    if (heads_above(hs, hn, 128) || B > 65535) return GDA_ERR_UNSUPPORTED;
    if (rows > 4294967296.0) return GDA_ERR_UNSUPPORTED;   // rows of the caches are counted in 32 bits
    // positions are 32 bits wide and stepped by 16; a range (a 19th of the batch's at most) is counted in 32 bits too
    if (Lcap > 0x7ffffff0 || static_cast<long long>(B) * Lcap > 1LL << 35) return GDA_ERR_UNSUPPORTED;
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDA_ERR_MISALIGNED;
    if (!aligned16(lens) || !aligned16(lambda)) return GDA_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(k1_scale) | reinterpret_cast<uintptr_t>(k2_scale) |
         reinterpret_cast<uintptr_t>(v_scale)) & 3u)
        return GDA_ERR_MISALIGNED;
    if (!workspace || !aligned16(workspace) || workspace_bytes < decode_fp4_workspace_bytes(B, hs, hn, d, dv))
        return GDA_ERR_WORKSPACE;
    return GDA_OK;
}

// Checks the arguments of gda_cache_append_fp4 and gda_cache_read_fp4 and fills what follows from them.
int fill_cache_fp4(CacheFp4Args &a, int num_pages, int page_size, int hs, int hn, int d, int dv) {
    const int heads[3] = {hs, hn, hs}, dims[3] = {d, d, dv};
    if (!a.slot_map) return GDA_ERR_INVALID_ARG;
    for (int t = 0; t < 3; ++t)
        if (!a.rows[t] || !a.codes[t] || !a.blocks[t] || !a.scale[t]) return GDA_ERR_INVALID_ARG;
    if (a.T < 1 || num_pages < 1 || page_size < 1 || hs < 1 || hn < 1 || d < 1 || dv < 1 || hs % hn != 0)
        return GDA_ERR_INVALID_ARG;
    if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL) return GDA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128) || !(dv == 64 || dv == 128 || dv == 256)) return GDA_ERR_UNSUPPORTED;
    if (heads_above(hs, hn, 128)) return GDA_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(a.slot_map) & 3u) return GDA_ERR_MISALIGNED;
    for (int t = 0; t < 3; ++t) {
        const long long row = static_cast<long long>(heads[t]) * dims[t];
        if (a.ld[t] < row || a.ld[t] > (1LL << 40)) return GDA_ERR_INVALID_ARG;
        if (a.ld[t] % 8 != 0 || !aligned16(a.rows[t]) || !aligned16(a.codes[t]) || !aligned16(a.blocks[t]) ||
            (reinterpret_cast<uintptr_t>(a.scale[t]) & 3u))
            return GDA_ERR_MISALIGNED;
        a.shift[t] = dims[t] == 64 ? 2 : (dims[t] == 128 ? 3 : 4);
        a.nb[t] = static_cast<int>(row / 16);
    }
    a.slots = num_pages * page_size;
    return current_device(&a.dev_err);
}

// What the calls over an 8-bit cache with a scale for each block of tokens ask of its geometry.
bool block_fits(int block) { return block == 16 || block == 32 || block == 64 || block == 128; }

int check_pages(int num_pages, int page_size, int block) {
    if (num_pages < 1 || page_size < 1 || block < 1 || page_size % block != 0) return GDA_ERR_INVALID_ARG;
    return block_fits(block) ? GDA_OK : GDA_ERR_UNSUPPORTED;
}

bool aligned4(std::initializer_list<const void *> ptrs) {
    uintptr_t any = 0;
    for (const void *p : ptrs) any |= reinterpret_cast<uintptr_t>(p);
    return (any & 3u) == 0;
}

// Checks the arguments of gda_cache_append_fp8_block and gda_cache_read_fp8_block and fills what follows from them.
int fill_cache_fp8_block(CacheFp8BlockArgs &a, int num_pages, int page_size, int hs, int hn, int d, int dv) {
    if (!a.slot_map) return GDA_ERR_INVALID_ARG;
    for (int t = 0; t < 3; ++t)
        if (!a.rows[t] || !a.codes[t] || !a.scale[t]) return GDA_ERR_INVALID_ARG;
    if (!a.bounds[0] != !a.bounds[1]) return GDA_ERR_INVALID_ARG;
    if (a.T < 1 || hs < 1 || hn < 1 || d < 1 || dv < 1 || hs % hn != 0) return GDA_ERR_INVALID_ARG;
    const int st = check_pages(num_pages, page_size, a.block);
    if (st != GDA_OK) return st;
    if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL) return GDA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128) || !(dv == 64 || dv == 128 || dv == 256)) return GDA_ERR_UNSUPPORTED;
    if (heads_above(hs, hn, 128)) return GDA_ERR_UNSUPPORTED;
    if (!aligned4({a.slot_map, a.scale[0], a.scale[1], a.scale[2]})) return GDA_ERR_MISALIGNED;
    a.heads[0] = a.heads[2] = hs, a.heads[1] = hn, a.dims[0] = a.dims[1] = d, a.dims[2] = dv;
    for (int t = 0; t < 3; ++t) {
        if (a.ld[t] < static_cast<long long>(a.heads[t]) * a.dims[t] || a.ld[t] > (1LL << 40)) return GDA_ERR_INVALID_ARG;
        if (a.ld[t] % 8 != 0 || !aligned16(a.rows[t]) || !aligned16(a.codes[t])) return GDA_ERR_MISALIGNED;
    }
    if (!aligned16(a.bounds[0]) || !aligned16(a.bounds[1])) return GDA_ERR_MISALIGNED;
    a.slots = num_pages * page_size;
    return GDA_OK;
}

// Checks what the three decodes over that cache have in common, and launches.
int decode_fp8_block(DecodeFp8BlockArgs &a, size_t workspace_bytes, gda_stream_t stream) {
    const void *ptrs[] = {a.q1, a.q2, a.k1c, a.k2c, a.vc, a.out};
    for (const void *p : ptrs)
        if (!p) return GDA_ERR_INVALID_ARG;
    if (!a.k1s || !a.k2s || !a.vs || !a.lens || !a.lambda) return GDA_ERR_INVALID_ARG;
    if (a.B < 1 || a.max_pages < 1 || a.hs < 1 || a.hn < 1 || a.d < 1 || a.dv < 1 || a.hs % a.hn != 0)
        return GDA_ERR_INVALID_ARG;
    int st = check_pages(a.num_pages, a.page_size, a.block);
    if (st == GDA_ERR_INVALID_ARG) return st;
    if (!std::isfinite(a.eps) || a.eps < 0.f || !std::isfinite(a.lambda_init)) return GDA_ERR_INVALID_ARG;
    const long long Lcap = static_cast<long long>(a.max_pages) * a.page_size;
    const double rows = static_cast<double>(a.num_pages) * a.page_size;
    if (Lcap > 0x7fffffffLL || rows * a.hs * (a.d > a.dv ? a.d : a.dv) > 9.0e15) return GDA_ERR_INVALID_ARG;
    if (a.list && a.keep < 1) return GDA_ERR_INVALID_ARG;
    if (st != GDA_OK) return st;
    if (!(a.d == 64 || a.d == 128) || !(a.dv == 64 || a.dv == 128 || a.dv == 256)) return GDA_ERR_UNSUPPORTED;
    if (heads_above(a.hs, a.hn, 128) || a.B > 65535) return GDA_ERR_UNSUPPORTED;
    if (rows > 2147483647.0) return GDA_ERR_UNSUPPORTED;   // a row is a coordinate of the copies
    // positions of a sequence, and tiles of 16 of all sequences, are counted in 32 bits
    const long long reach = a.list ? static_cast<long long>(a.keep) * a.block : Lcap;
    if (Lcap > 0x7ffffff0 || reach > 0x7ffffff0 || a.B * reach > 1LL << 34) return GDA_ERR_UNSUPPORTED;
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDA_ERR_MISALIGNED;
    if (!aligned4({a.k1s, a.k2s, a.vs, a.lens, a.lambda, a.block_table, a.list, a.count})) return GDA_ERR_MISALIGNED;
    if (!a.workspace || !aligned16(a.workspace) ||
        workspace_bytes < decode_fp8_block_workspace_bytes(a.B, a.hs, a.hn, a.d, a.dv))
        return GDA_ERR_WORKSPACE;
    a.Lcap = static_cast<int>(Lcap);
    if ((st = device_state(&a.dev_err)) != GDA_OK) return st;
    return launch_decode_fp8_block(a, reinterpret_cast<cudaStream_t>(stream));
}

struct Four {
    const void *p[4];
};
struct FourOut {
    void *p[4];
};
struct FourStrides {
    long long s[4];
};

int check_norm_rope(const Four &x, const FourOut &y, const float *weight, const int *positions, const float *inv_freq,
                    int T, int hs, int hn, int d, int rot, float eps, unsigned flags) {
    for (int t = 0; t < 4; ++t)
        if (!x.p[t] || !y.p[t]) return GDA_ERR_INVALID_ARG;
    if (!weight || !positions || !inv_freq) return GDA_ERR_INVALID_ARG;
    if (T < 1 || hs < 1 || hn < 1 || d < 1 || rot < 1 || hs % hn != 0) return GDA_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f) return GDA_ERR_INVALID_ARG;
    if (flags & ~GDA_FLAG_ROPE_INTERLEAVED) return GDA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128) || rot > d || rot % 16 != 0 || heads_above(hs, hn, 1024)) return GDA_ERR_UNSUPPORTED;
    for (int t = 0; t < 4; ++t)
        if (!aligned16(x.p[t]) || !aligned16(y.p[t])) return GDA_ERR_MISALIGNED;
    if (!aligned16(weight) || ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(inv_freq)) & 3u))
        return GDA_ERR_MISALIGNED;
    return GDA_OK;
}

// Strides between tokens: a whole row at least, and a multiple of 16 bytes.
int check_stride(long long s, int heads, int d, bool f32) {
    if (s < static_cast<long long>(heads) * d || s > (1LL << 40)) return GDA_ERR_INVALID_ARG;
    return s % (f32 ? 4 : 8) == 0 ? GDA_OK : GDA_ERR_MISALIGNED;
}

int norm_rope(const Four &x, const FourStrides &ld, const float *weight, const int *positions, const float *inv_freq,
              const FourOut &y, int T, int hs, int hn, int d, int rot, float eps, unsigned flags, bool f32,
              gda_stream_t stream) {
    int st = check_norm_rope(x, y, weight, positions, inv_freq, T, hs, hn, d, rot, eps, flags);
    if (st != GDA_OK) return st;
    NormRopeArgs a{};
    for (int t = 0; t < 4; ++t) {
        const int heads = t < 2 ? hs : hn;
        if ((st = check_stride(ld.s[t], heads, d, f32)) != GDA_OK) return st;
        a.x[t] = x.p[t];
        a.ld[t] = ld.s[t];
        a.y[t] = y.p[t];
        a.ldy[t] = static_cast<long long>(heads) * d;
    }
    a.weight = weight, a.positions = positions, a.inv_freq = inv_freq;
    a.T = T, a.hs = hs, a.hn = hn, a.d = d, a.rot = rot;
    a.interleaved = (flags & GDA_FLAG_ROPE_INTERLEAVED) != 0, a.f32 = f32, a.eps = eps;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDA_OK) return st;
    return launch_qk_norm_rope(a, reinterpret_cast<cudaStream_t>(stream));
}

int norm_rope_bwd(const Four &x, const long long *strides, const float *weight, const int *positions,
                  const float *inv_freq, const Four &dy, const FourOut &dx, float *dweight, int T, int hs, int hn,
                  int d, int rot, float eps, unsigned flags, bool f32, void *workspace, size_t workspace_bytes,
                  gda_stream_t stream) {
    int st = check_norm_rope(x, dx, weight, positions, inv_freq, T, hs, hn, d, rot, eps, flags);
    if (st != GDA_OK) return st;
    if (!strides || !dweight) return GDA_ERR_INVALID_ARG;
    NormRopeArgs a{};
    for (int t = 0; t < 4; ++t) {
        const int heads = t < 2 ? hs : hn;
        if (!dy.p[t]) return GDA_ERR_INVALID_ARG;
        if (!aligned16(dy.p[t])) return GDA_ERR_MISALIGNED;
        if ((st = check_stride(strides[t], heads, d, f32)) != GDA_OK) return st;
        if ((st = check_stride(strides[4 + t], heads, d, f32)) != GDA_OK) return st;
        a.x[t] = x.p[t];
        a.ld[t] = strides[t];
        a.y[t] = dx.p[t];
        a.ldy[t] = strides[4 + t];
        a.dy[t] = static_cast<const float *>(dy.p[t]);
    }
    if (reinterpret_cast<uintptr_t>(dweight) & 3u) return GDA_ERR_MISALIGNED;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < qk_norm_rope_bwd_workspace_bytes(T, hs, hn, d))
        return GDA_ERR_WORKSPACE;
    a.weight = weight, a.positions = positions, a.inv_freq = inv_freq;
    a.partial = static_cast<float *>(workspace), a.dweight = dweight;
    a.T = T, a.hs = hs, a.hn = hn, a.d = d, a.rot = rot;
    a.interleaved = (flags & GDA_FLAG_ROPE_INTERLEAVED) != 0, a.f32 = f32, a.eps = eps;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDA_OK) return st;
    return launch_qk_norm_rope_bwd(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

}  // namespace gda

using namespace gda;

extern "C" {

int gda_attn_fwd_ex(const void *q_sig, const void *k_sig, const void *q_noise, const void *k_noise,
                    const void *v, const float *lambda, float lambda_init, void *out, int B, int L,
                    int h_s, int h_n, int d, int dv, int causal, float eps, unsigned flags,
                    gda_stream_t stream) {
    int st = check_prefill_common(q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, out, B, L,
                                  h_s, h_n, d, dv, causal, eps, flags,
                                  GDA_FLAG_NO_NORM | GDA_FLAG_SINGLE_PASS);
    if (st != GDA_OK) return st;
    if (!(d == 64 || d == 128) || !(dv == 128 || dv == 256)) return GDA_ERR_UNSUPPORTED;
    unsigned *err = nullptr;
    st = current_device(&err);
    if (st != GDA_OK) return st;
    PrefillArgs a{q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, out, B, L, h_s, h_n,
                  d, dv, causal, eps, flags & GDA_FLAG_NO_NORM, err};
    if (!(flags & GDA_FLAG_SINGLE_PASS) && prefill_group_supported(a))
        return launch_prefill_group(a, reinterpret_cast<cudaStream_t>(stream));
    return launch_prefill_tc(a, reinterpret_cast<cudaStream_t>(stream));
}

int gda_attn_fwd_chunk(const void *q_sig, const void *k_sig, const void *q_noise, const void *k_noise,
                       const void *v, const float *lambda, float lambda_init, void *out, int B, int L,
                       int Lk, int h_s, int h_n, int d, int dv, int causal, float eps, unsigned flags,
                       gda_stream_t stream) {
    int st = check_prefill_common(q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, out, B, L,
                                  h_s, h_n, d, dv, causal, eps, flags,
                                  GDA_FLAG_NO_NORM | GDA_FLAG_SINGLE_PASS);
    if (st != GDA_OK) return st;
    if (Lk < 1 || (causal && Lk < L)) return GDA_ERR_INVALID_ARG;
    if (static_cast<double>(B) * Lk * (h_s > h_n ? h_s : h_n) * (d > dv ? d : dv) > 9.0e15)
        return GDA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128) || !(dv == 128 || dv == 256)) return GDA_ERR_UNSUPPORTED;
    unsigned *err = nullptr;
    st = current_device(&err);
    if (st != GDA_OK) return st;
    PrefillArgs a{q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, out, B, L, h_s, h_n,
                  d, dv, causal, eps, flags & GDA_FLAG_NO_NORM, err};
    a.Lk = Lk;
    if (!(flags & GDA_FLAG_SINGLE_PASS) && prefill_group_supported(a))
        return launch_prefill_group(a, reinterpret_cast<cudaStream_t>(stream));
    return launch_prefill_tc(a, reinterpret_cast<cudaStream_t>(stream));
}

int gda_attn_fwd_chunk_2pass(const void *q_sig, const void *k_sig, const void *q_noise, const void *k_noise,
                             const void *v, const float *lambda, float lambda_init, void *out, int B, int L,
                             int Lk, int h_s, int h_n, int d, int dv, int causal, float eps, unsigned flags,
                             void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    int st = check_prefill_common(q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, out, B, L,
                                  h_s, h_n, d, dv, causal, eps, flags);
    if (st != GDA_OK) return st;
    if (Lk < 1 || (causal && Lk < L)) return GDA_ERR_INVALID_ARG;
    if (static_cast<double>(B) * Lk * (h_s > h_n ? h_s : h_n) * (d > dv ? d : dv) > 9.0e15)
        return GDA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128) || !(dv == 128 || dv == 256)) return GDA_ERR_UNSUPPORTED;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < prefill_2pass_workspace_bytes(B, L, h_s, h_n))
        return GDA_ERR_WORKSPACE;
    unsigned *err = nullptr;
    st = current_device(&err);
    if (st != GDA_OK) return st;
    PrefillArgs a{q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, out, B, L, h_s, h_n,
                  d, dv, causal, eps, flags, err};
    a.Lk = Lk;
    return launch_prefill_2pass(a, workspace, reinterpret_cast<cudaStream_t>(stream));
}

int gda_attn_fwd(const void *q_sig, const void *k_sig, const void *q_noise, const void *k_noise,
                 const void *v, const float *lambda, float lambda_init, void *out, int B, int L,
                 int h_s, int h_n, int d, int dv, int causal, float eps, gda_stream_t stream) {
    return gda_attn_fwd_ex(q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, out, B, L, h_s,
                           h_n, d, dv, causal, eps, 0u, stream);
}

int gda_attn_fwd_f32_ex(const float *q_sig, const float *k_sig, const float *q_noise,
                        const float *k_noise, const float *v, const float *lambda,
                        float lambda_init, float *out, int B, int L, int h_s, int h_n, int d,
                        int dv, int causal, float eps, unsigned flags, gda_stream_t stream) {
    int st = check_prefill_common(q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, out, B, L,
                                  h_s, h_n, d, dv, causal, eps, flags);
    if (st != GDA_OK) return st;
    if (d > 256 || dv % 32 != 0 || dv > 256) return GDA_ERR_UNSUPPORTED;
    if (h_s > 65535 || B > 65535) return GDA_ERR_UNSUPPORTED;
    unsigned *err = nullptr;
    st = current_device(&err);
    if (st != GDA_OK) return st;
    PrefillArgs a{q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, out, B, L, h_s, h_n,
                  d, dv, causal, eps, flags, err};
    return launch_prefill_f32(a, reinterpret_cast<cudaStream_t>(stream));
}

int gda_attn_fwd_f32(const float *q_sig, const float *k_sig, const float *q_noise,
                     const float *k_noise, const float *v, const float *lambda, float lambda_init,
                     float *out, int B, int L, int h_s, int h_n, int d, int dv, int causal,
                     float eps, gda_stream_t stream) {
    return gda_attn_fwd_f32_ex(q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, out, B, L,
                               h_s, h_n, d, dv, causal, eps, 0u, stream);
}

size_t gda_attn_bwd_bf16_workspace_size(int B, int L, int h_s, int h_n, int dv) {
    if (B < 1 || L < 1 || h_s < 1 || h_n < 1 || dv < 1) return 0;
    if (static_cast<double>(B) * L * (h_s + h_n) * (dv > 1 ? dv : 1) > 9.0e15) return 0;
    return backward_tc_workspace_bytes(B, L, h_s, h_n, dv);
}

int gda_attn_bwd_bf16(const void *q_sig, const void *k_sig, const void *q_noise, const void *k_noise,
                      const void *v, const float *lambda, float lambda_init, const void *dy, float *dq_sig,
                      float *dk_sig, float *dq_noise, float *dk_noise, float *dv_out, float *dlambda, int B,
                      int L, int h_s, int h_n, int d, int dv, int causal, float eps, unsigned flags,
                      void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    int st = check_prefill_common(q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, dy, B, L, h_s,
                                  h_n, d, dv, causal, eps, flags);
    if (st != GDA_OK) return st;
    if (!dq_sig || !dk_sig || !dq_noise || !dk_noise || !dv_out || !dlambda) return GDA_ERR_INVALID_ARG;
    if (d != 64 || dv != 128) return GDA_ERR_UNSUPPORTED;
    if (!aligned16(dq_sig) || !aligned16(dk_sig) || !aligned16(dq_noise) || !aligned16(dk_noise) ||
        !aligned16(dv_out) || !aligned16(dlambda))
        return GDA_ERR_MISALIGNED;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < gda_attn_bwd_bf16_workspace_size(B, L, h_s, h_n, dv))
        return GDA_ERR_WORKSPACE;
    unsigned *err = nullptr;
    st = current_device(&err);
    if (st != GDA_OK) return st;
    BackwardTcArgs a{q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, dy, dq_sig, dk_sig, dq_noise,
                     dk_noise, dv_out, dlambda, B, L, h_s, h_n, d, dv, causal, eps, flags, workspace, err};
    return launch_backward_tc(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t gda_attn_fwd_2pass_workspace_size(int B, int L, int h_s, int h_n) {
    if (B < 1 || L < 1 || h_s < 1 || h_n < 1) return 0;
    if (static_cast<double>(B) * L * (h_s + h_n) > 9.0e15) return 0;
    return prefill_2pass_workspace_bytes(B, L, h_s, h_n);
}

int gda_attn_fwd_2pass(const void *q_sig, const void *k_sig, const void *q_noise, const void *k_noise,
                       const void *v, const float *lambda, float lambda_init, void *out, int B, int L,
                       int h_s, int h_n, int d, int dv, int causal, float eps, unsigned flags,
                       void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    int st = check_prefill_common(q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, out, B, L,
                                  h_s, h_n, d, dv, causal, eps, flags);
    if (st != GDA_OK) return st;
    if (!(d == 64 || d == 128) || !(dv == 128 || dv == 256)) return GDA_ERR_UNSUPPORTED;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < gda_attn_fwd_2pass_workspace_size(B, L, h_s, h_n))
        return GDA_ERR_WORKSPACE;
    unsigned *err = nullptr;
    st = current_device(&err);
    if (st != GDA_OK) return st;
    PrefillArgs a{q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, out, B, L, h_s, h_n,
                  d, dv, causal, eps, flags, err};
    return launch_prefill_2pass(a, workspace, reinterpret_cast<cudaStream_t>(stream));
}

size_t gda_attn_bwd_workspace_size(int B, int L, int h_s, int d, int dv) {
    if (B < 1 || L < 1 || h_s < 1 || d < 1 || dv < 1) return 0;
    if (static_cast<double>(B) * L * h_s * (d > dv ? d : dv) > 9.0e15) return 0;
    return backward_f32_workspace_bytes(B, L, h_s, d, dv);
}

int gda_attn_bwd(const float *q_sig, const float *k_sig, const float *q_noise, const float *k_noise,
                 const float *v, const float *lambda, float lambda_init, const float *dy, float *dq_sig,
                 float *dk_sig, float *dq_noise, float *dk_noise, float *dv_out, float *dlambda, int B,
                 int L, int h_s, int h_n, int d, int dv, int causal, float eps, unsigned flags,
                 void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    int st = check_prefill_common(q_sig, k_sig, q_noise, k_noise, v, lambda, lambda_init, dy, B, L, h_s,
                                  h_n, d, dv, causal, eps, flags);
    if (st != GDA_OK) return st;
    if (!dq_sig || !dk_sig || !dq_noise || !dk_noise || !dv_out || !dlambda) return GDA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128) || !(dv == 64 || dv == 128 || dv == 256)) return GDA_ERR_UNSUPPORTED;
    if (h_s > 65535 || B > 65535) return GDA_ERR_UNSUPPORTED;
    if (!aligned16(dq_sig) || !aligned16(dk_sig) || !aligned16(dq_noise) || !aligned16(dk_noise) ||
        !aligned16(dv_out) || !aligned16(dlambda))
        return GDA_ERR_MISALIGNED;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < gda_attn_bwd_workspace_size(B, L, h_s, d, dv))
        return GDA_ERR_WORKSPACE;
    unsigned *err = nullptr;
    st = current_device(&err);
    if (st != GDA_OK) return st;
    BackwardArgs a{q_sig, k_sig, q_noise, k_noise, v, lambda, dy, lambda_init, dq_sig, dk_sig, dq_noise,
                   dk_noise, dv_out, dlambda, B, L, h_s, h_n, d, dv, causal, eps, flags, workspace};
    return launch_backward_f32(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t gda_attn_decode_workspace_size(int B, int Lcap, int h_s, int h_n, int dv) {
    if (B < 1 || Lcap < 1 || h_s < 1 || h_n < 1 || dv < 1 || h_s % h_n != 0) return 0;
    return decode_plan(B, Lcap, h_s, h_n, dv).bytes;
}

int gda_attn_decode(const void *q_sig, const void *q_noise, const void *k_sig_cache,
                    const void *k_noise_cache, const void *v_cache, const int *cache_lens,
                    const float *lambda, float lambda_init, void *out, int B, int Lcap, int h_s,
                    int h_n, int d, int dv, float eps, void *workspace, size_t workspace_bytes,
                    gda_stream_t stream) {
    if (!q_sig || !q_noise || !k_sig_cache || !k_noise_cache || !v_cache || !cache_lens || !lambda ||
        !out)
        return GDA_ERR_INVALID_ARG;
    if (B < 1 || Lcap < 1 || h_s < 1 || h_n < 1 || d < 1 || dv < 1 || h_s % h_n != 0)
        return GDA_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(lambda_init)) return GDA_ERR_INVALID_ARG;
    if (static_cast<double>(B) * Lcap * h_s * (d > dv ? d : dv) > 9.0e15) return GDA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128) || !(dv == 64 || dv == 128 || dv == 256)) return GDA_ERR_UNSUPPORTED;
    if ((h_s * d + h_n * d + h_s * dv) / 8 > 1024 || h_s + h_n > 128 || B > 65535)
        return GDA_ERR_UNSUPPORTED;
    if (!aligned16(q_sig) || !aligned16(q_noise) || !aligned16(k_sig_cache) ||
        !aligned16(k_noise_cache) || !aligned16(v_cache) || !aligned16(cache_lens) ||
        !aligned16(lambda) || !aligned16(out))
        return GDA_ERR_MISALIGNED;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < gda_attn_decode_workspace_size(B, Lcap, h_s, h_n, dv))
        return GDA_ERR_WORKSPACE;
    unsigned *err = nullptr;
    const int st = current_device(&err);
    if (st != GDA_OK) return st;
    DecodeArgs a{q_sig, q_noise, k_sig_cache, k_noise_cache, v_cache, cache_lens, lambda, lambda_init,
                 out, B, Lcap, h_s, h_n, d, dv, eps, workspace, workspace_bytes, err};
    return launch_decode(a, reinterpret_cast<cudaStream_t>(stream));
}

int gda_attn_decode_fp8(const void *q_sig, const void *q_noise, const void *k_sig_cache,
                        const void *k_noise_cache, const void *v_cache, const float *k_sig_scale,
                        const float *k_noise_scale, const float *v_scale, const int *cache_lens,
                        const float *lambda, float lambda_init, void *out, int B, int Lcap, int h_s,
                        int h_n, int d, int dv, float eps, void *workspace, size_t workspace_bytes,
                        gda_stream_t stream) {
    if (!q_sig || !q_noise || !k_sig_cache || !k_noise_cache || !v_cache || !k_sig_scale || !k_noise_scale ||
        !v_scale || !cache_lens || !lambda || !out)
        return GDA_ERR_INVALID_ARG;
    if (B < 1 || Lcap < 1 || h_s < 1 || h_n < 1 || d < 1 || dv < 1 || h_s % h_n != 0)
        return GDA_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(lambda_init)) return GDA_ERR_INVALID_ARG;
    if (static_cast<double>(B) * Lcap * h_s * (d > dv ? d : dv) > 9.0e15) return GDA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128) || !(dv == 64 || dv == 128 || dv == 256)) return GDA_ERR_UNSUPPORTED;
    if (h_s + h_n > 128 || B > 65535) return GDA_ERR_UNSUPPORTED;
    if (!aligned16(q_sig) || !aligned16(q_noise) || !aligned16(k_sig_cache) || !aligned16(k_noise_cache) ||
        !aligned16(v_cache) || !aligned16(cache_lens) || !aligned16(lambda) || !aligned16(out))
        return GDA_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(k_sig_scale) | reinterpret_cast<uintptr_t>(k_noise_scale) |
         reinterpret_cast<uintptr_t>(v_scale)) & 3u)
        return GDA_ERR_MISALIGNED;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < gda_attn_decode_workspace_size(B, Lcap, h_s, h_n, dv))
        return GDA_ERR_WORKSPACE;
    unsigned *err = nullptr;
    const int st = current_device(&err);
    if (st != GDA_OK) return st;
    DecodeArgs a{q_sig, q_noise, k_sig_cache, k_noise_cache, v_cache, cache_lens, lambda, lambda_init,
                 out, B, Lcap, h_s, h_n, d, dv, eps, workspace, workspace_bytes, err};
    a.fp8 = 1;
    a.k1_scale = k_sig_scale;
    a.k2_scale = k_noise_scale;
    a.v_scale = v_scale;
    return launch_decode(a, reinterpret_cast<cudaStream_t>(stream));
}

int gda_attn_decode_paged(const void *q_sig, const void *q_noise, const void *k_sig_pool,
                          const void *k_noise_pool, const void *v_pool, const int *block_table,
                          const int *cache_lens, const float *lambda, float lambda_init, void *out, int B,
                          int max_pages, int page_size, int num_pages, int h_s, int h_n, int d, int dv,
                          float eps, void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    if (!q_sig || !q_noise || !k_sig_pool || !k_noise_pool || !v_pool || !block_table || !cache_lens ||
        !lambda || !out)
        return GDA_ERR_INVALID_ARG;
    if (B < 1 || max_pages < 1 || page_size < 1 || num_pages < 1 || h_s < 1 || h_n < 1 || d < 1 || dv < 1 ||
        h_s % h_n != 0)
        return GDA_ERR_INVALID_ARG;
    const long long Lcap = static_cast<long long>(max_pages) * page_size;
    if (Lcap > 0x7fffffffLL) return GDA_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(lambda_init)) return GDA_ERR_INVALID_ARG;
    if (static_cast<double>(num_pages) * page_size * h_s * (d > dv ? d : dv) > 9.0e15) return GDA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128) || !(dv == 64 || dv == 128 || dv == 256)) return GDA_ERR_UNSUPPORTED;
    if ((h_s * d + h_n * d + h_s * dv) / 8 > 1024 || h_s + h_n > 128 || B > 65535) return GDA_ERR_UNSUPPORTED;
    if (!aligned16(q_sig) || !aligned16(q_noise) || !aligned16(k_sig_pool) || !aligned16(k_noise_pool) ||
        !aligned16(v_pool) || !aligned16(cache_lens) || !aligned16(lambda) || !aligned16(out) ||
        (reinterpret_cast<uintptr_t>(block_table) & 3u))
        return GDA_ERR_MISALIGNED;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < gda_attn_decode_workspace_size(B, static_cast<int>(Lcap), h_s, h_n, dv))
        return GDA_ERR_WORKSPACE;
    unsigned *err = nullptr;
    const int st = current_device(&err);
    if (st != GDA_OK) return st;
    DecodeArgs a{q_sig, q_noise, k_sig_pool, k_noise_pool, v_pool, cache_lens, lambda, lambda_init,
                 out, B, static_cast<int>(Lcap), h_s, h_n, d, dv, eps, workspace, workspace_bytes, err};
    a.block_table = block_table;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    return launch_decode(a, reinterpret_cast<cudaStream_t>(stream));
}

int gda_attn_decode_paged_fp8(const void *q_sig, const void *q_noise, const void *k_sig_pool,
                              const void *k_noise_pool, const void *v_pool, const float *k_sig_scale,
                              const float *k_noise_scale, const float *v_scale, const int *block_table,
                              const int *cache_lens, const float *lambda, float lambda_init, void *out, int B,
                              int max_pages, int page_size, int num_pages, int h_s, int h_n, int d, int dv,
                              float eps, void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    if (!q_sig || !q_noise || !k_sig_pool || !k_noise_pool || !v_pool || !k_sig_scale || !k_noise_scale ||
        !v_scale || !block_table || !cache_lens || !lambda || !out)
        return GDA_ERR_INVALID_ARG;
    if (B < 1 || max_pages < 1 || page_size < 1 || num_pages < 1 || h_s < 1 || h_n < 1 || d < 1 || dv < 1 ||
        h_s % h_n != 0)
        return GDA_ERR_INVALID_ARG;
    const long long Lcap = static_cast<long long>(max_pages) * page_size;
    if (Lcap > 0x7fffffffLL) return GDA_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(lambda_init)) return GDA_ERR_INVALID_ARG;
    if (static_cast<double>(num_pages) * page_size * h_s * (d > dv ? d : dv) > 9.0e15) return GDA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128) || !(dv == 64 || dv == 128 || dv == 256)) return GDA_ERR_UNSUPPORTED;
    if (h_s + h_n > 128 || B > 65535) return GDA_ERR_UNSUPPORTED;
    if (!aligned16(q_sig) || !aligned16(q_noise) || !aligned16(k_sig_pool) || !aligned16(k_noise_pool) ||
        !aligned16(v_pool) || !aligned16(cache_lens) || !aligned16(lambda) || !aligned16(out) ||
        (reinterpret_cast<uintptr_t>(block_table) & 3u))
        return GDA_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(k_sig_scale) | reinterpret_cast<uintptr_t>(k_noise_scale) |
         reinterpret_cast<uintptr_t>(v_scale)) & 3u)
        return GDA_ERR_MISALIGNED;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < gda_attn_decode_workspace_size(B, static_cast<int>(Lcap), h_s, h_n, dv))
        return GDA_ERR_WORKSPACE;
    unsigned *err = nullptr;
    const int st = current_device(&err);
    if (st != GDA_OK) return st;
    DecodeArgs a{q_sig, q_noise, k_sig_pool, k_noise_pool, v_pool, cache_lens, lambda, lambda_init,
                 out, B, static_cast<int>(Lcap), h_s, h_n, d, dv, eps, workspace, workspace_bytes, err};
    a.fp8 = 1;
    a.k1_scale = k_sig_scale;
    a.k2_scale = k_noise_scale;
    a.v_scale = v_scale;
    a.block_table = block_table;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    return launch_decode(a, reinterpret_cast<cudaStream_t>(stream));
}

int gda_lambda_reparam(const float *lambda_q1, const float *lambda_k1, const float *lambda_q2,
                       const float *lambda_k2, float lambda_init, float *lambda_out, int h_s, int d,
                       gda_stream_t stream) {
    if (!lambda_q1 || !lambda_k1 || !lambda_q2 || !lambda_k2 || !lambda_out) return GDA_ERR_INVALID_ARG;
    if (h_s < 1 || d < 1 || !std::isfinite(lambda_init)) return GDA_ERR_INVALID_ARG;
    if (static_cast<long long>(h_s) * d > 0x7fffffffLL) return GDA_ERR_INVALID_ARG;
    const uintptr_t any = reinterpret_cast<uintptr_t>(lambda_q1) | reinterpret_cast<uintptr_t>(lambda_k1) |
                          reinterpret_cast<uintptr_t>(lambda_q2) | reinterpret_cast<uintptr_t>(lambda_k2) |
                          reinterpret_cast<uintptr_t>(lambda_out);
    if (any & 3u) return GDA_ERR_MISALIGNED;
    unsigned *err = nullptr;
    const int st = current_device(&err);
    if (st != GDA_OK) return st;
    return launch_lambda_reparam(lambda_q1, lambda_k1, lambda_q2, lambda_k2, lambda_init, lambda_out, h_s, d,
                                 reinterpret_cast<cudaStream_t>(stream));
}

size_t gda_attn_decode_fp4_workspace_size(int B, int h_s, int h_n, int d, int dv) {
    if (B < 1 || h_s < 1 || h_n < 1 || d < 1 || dv < 1 || h_s % h_n != 0) return 0;
    if (B > 65535 || heads_above(h_s, h_n, 128)) return 0;
    if (!(d == 64 || d == 128) || !(dv == 64 || dv == 128 || dv == 256)) return 0;   // the plan divides by a tile's bytes
    return decode_fp4_workspace_bytes(B, h_s, h_n, d, dv);
}

int gda_attn_decode_fp4(const void *q_sig, const void *q_noise, const void *k_sig_cache,
                        const void *k_noise_cache, const void *v_cache, const void *k_sig_block_scale,
                        const void *k_noise_block_scale, const void *v_block_scale, const float *k_sig_scale,
                        const float *k_noise_scale, const float *v_scale, const int *cache_lens,
                        const float *lambda, float lambda_init, void *out, int B, int Lcap, int h_s, int h_n,
                        int d, int dv, float eps, void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    const void *ptrs[] = {q_sig, q_noise, k_sig_cache, k_noise_cache, v_cache, k_sig_block_scale,
                          k_noise_block_scale, v_block_scale, out};
    int st = check_decode_fp4(ptrs, k_sig_scale, k_noise_scale, v_scale, cache_lens, lambda, lambda_init, B, Lcap,
                              h_s, h_n, d, dv, eps, static_cast<double>(B) * Lcap, workspace, workspace_bytes);
    if (st != GDA_OK) return st;
    DecodeFp4Args a{q_sig, q_noise, bytes_of(k_sig_cache), bytes_of(k_noise_cache), bytes_of(v_cache),
                    bytes_of(k_sig_block_scale), bytes_of(k_noise_block_scale), bytes_of(v_block_scale),
                    k_sig_scale, k_noise_scale, v_scale, cache_lens, lambda, lambda_init, out, B, Lcap, h_s, h_n,
                    d, dv, eps, workspace, nullptr};
    st = current_device(&a.dev_err);
    if (st != GDA_OK) return st;
    return launch_decode_fp4(a, reinterpret_cast<cudaStream_t>(stream));
}

int gda_attn_decode_paged_fp4(const void *q_sig, const void *q_noise, const void *k_sig_pool,
                              const void *k_noise_pool, const void *v_pool, const void *k_sig_block_scale,
                              const void *k_noise_block_scale, const void *v_block_scale, const float *k_sig_scale,
                              const float *k_noise_scale, const float *v_scale, const int *block_table,
                              const int *cache_lens, const float *lambda, float lambda_init, void *out, int B,
                              int max_pages, int page_size, int num_pages, int h_s, int h_n, int d, int dv,
                              float eps, void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    if (!block_table) return GDA_ERR_INVALID_ARG;
    if (max_pages < 1 || page_size < 1 || num_pages < 1) return GDA_ERR_INVALID_ARG;
    const long long Lcap = static_cast<long long>(max_pages) * page_size;
    if (Lcap > 0x7fffffffLL) return GDA_ERR_INVALID_ARG;
    const void *ptrs[] = {q_sig, q_noise, k_sig_pool, k_noise_pool, v_pool, k_sig_block_scale,
                          k_noise_block_scale, v_block_scale, out};
    int st = check_decode_fp4(ptrs, k_sig_scale, k_noise_scale, v_scale, cache_lens, lambda, lambda_init, B,
                              static_cast<int>(Lcap), h_s, h_n, d, dv, eps,
                              static_cast<double>(num_pages) * page_size, workspace, workspace_bytes);
    if (st != GDA_OK) return st;
    if (reinterpret_cast<uintptr_t>(block_table) & 3u) return GDA_ERR_MISALIGNED;
    DecodeFp4Args a{q_sig, q_noise, bytes_of(k_sig_pool), bytes_of(k_noise_pool), bytes_of(v_pool),
                    bytes_of(k_sig_block_scale), bytes_of(k_noise_block_scale), bytes_of(v_block_scale),
                    k_sig_scale, k_noise_scale, v_scale, cache_lens, lambda, lambda_init, out, B,
                    static_cast<int>(Lcap), h_s, h_n, d, dv, eps, workspace, nullptr};
    a.block_table = block_table;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    st = current_device(&a.dev_err);
    if (st != GDA_OK) return st;
    return launch_decode_fp4(a, reinterpret_cast<cudaStream_t>(stream));
}

int gda_cache_append_fp4(const void *k_sig, const void *k_noise, const void *v, const int *slot_map,
                         void *k_sig_pool, void *k_noise_pool, void *v_pool, void *k_sig_block_scale,
                         void *k_noise_block_scale, void *v_block_scale, const float *k_sig_scale,
                         const float *k_noise_scale, const float *v_scale, int T, int num_pages, int page_size,
                         int h_s, int h_n, int d, int dv, long long k_sig_stride, long long k_noise_stride,
                         long long v_stride, gda_stream_t stream) {
    CacheFp4Args a{{k_sig, k_noise, v}, {k_sig_stride, k_noise_stride, v_stride}, slot_map,
                   {static_cast<uint8_t *>(k_sig_pool), static_cast<uint8_t *>(k_noise_pool),
                    static_cast<uint8_t *>(v_pool)},
                   {static_cast<uint8_t *>(k_sig_block_scale), static_cast<uint8_t *>(k_noise_block_scale),
                    static_cast<uint8_t *>(v_block_scale)},
                   {k_sig_scale, k_noise_scale, v_scale}, {}, {}, T, 0, nullptr};
    const int st = fill_cache_fp4(a, num_pages, page_size, h_s, h_n, d, dv);
    if (st != GDA_OK) return st;
    return launch_cache_append_fp4(a, reinterpret_cast<cudaStream_t>(stream));
}

int gda_cache_read_fp4(const int *slot_map, const void *k_sig_pool, const void *k_noise_pool, const void *v_pool,
                       const void *k_sig_block_scale, const void *k_noise_block_scale, const void *v_block_scale,
                       const float *k_sig_scale, const float *k_noise_scale, const float *v_scale, void *k_sig_out,
                       void *k_noise_out, void *v_out, int T, int num_pages, int page_size, int h_s, int h_n, int d,
                       int dv, gda_stream_t stream) {
    auto pool = [](const void *x) { return const_cast<uint8_t *>(bytes_of(x)); };
    CacheFp4Args a{{k_sig_out, k_noise_out, v_out},
                   {static_cast<long long>(h_s) * d, static_cast<long long>(h_n) * d, static_cast<long long>(h_s) * dv},
                   slot_map,
                   {pool(k_sig_pool), pool(k_noise_pool), pool(v_pool)},
                   {pool(k_sig_block_scale), pool(k_noise_block_scale), pool(v_block_scale)},
                   {k_sig_scale, k_noise_scale, v_scale}, {}, {}, T, 0, nullptr};
    const int st = fill_cache_fp4(a, num_pages, page_size, h_s, h_n, d, dv);
    if (st != GDA_OK) return st;
    return launch_cache_read_fp4(a, reinterpret_cast<cudaStream_t>(stream));
}

int gda_qk_norm_rope(const void *q_sig, const void *k_sig, const void *q_noise, const void *k_noise,
                     const float *weight, const int *positions, const float *inv_freq, void *q_sig_out,
                     void *k_sig_out, void *q_noise_out, void *k_noise_out, int T, int h_s, int h_n, int d, int rot,
                     long long q_sig_stride, long long k_sig_stride, long long q_noise_stride,
                     long long k_noise_stride, float eps, unsigned flags, gda_stream_t stream) {
    return norm_rope({q_sig, k_sig, q_noise, k_noise}, {q_sig_stride, k_sig_stride, q_noise_stride, k_noise_stride},
                     weight, positions, inv_freq, {q_sig_out, k_sig_out, q_noise_out, k_noise_out}, T, h_s, h_n, d,
                     rot, eps, flags, false, stream);
}

int gda_qk_norm_rope_f32(const float *q_sig, const float *k_sig, const float *q_noise, const float *k_noise,
                         const float *weight, const int *positions, const float *inv_freq, float *q_sig_out,
                         float *k_sig_out, float *q_noise_out, float *k_noise_out, int T, int h_s, int h_n, int d,
                         int rot, long long q_sig_stride, long long k_sig_stride, long long q_noise_stride,
                         long long k_noise_stride, float eps, unsigned flags, gda_stream_t stream) {
    return norm_rope({q_sig, k_sig, q_noise, k_noise}, {q_sig_stride, k_sig_stride, q_noise_stride, k_noise_stride},
                     weight, positions, inv_freq, {q_sig_out, k_sig_out, q_noise_out, k_noise_out}, T, h_s, h_n, d,
                     rot, eps, flags, true, stream);
}

size_t gda_qk_norm_rope_bwd_workspace_size(int T, int h_s, int h_n, int d) {
    if (T < 1 || h_s < 1 || h_n < 1 || h_s % h_n != 0 || heads_above(h_s, h_n, 1024) || !(d == 64 || d == 128)) return 0;
    return qk_norm_rope_bwd_workspace_bytes(T, h_s, h_n, d);
}

int gda_qk_norm_rope_bwd(const void *q_sig, const void *k_sig, const void *q_noise, const void *k_noise,
                         const float *weight, const int *positions, const float *inv_freq, const float *dq_sig,
                         const float *dk_sig, const float *dq_noise, const float *dk_noise, void *dq_sig_out,
                         void *dk_sig_out, void *dq_noise_out, void *dk_noise_out, float *dweight, int T, int h_s,
                         int h_n, int d, int rot, const long long *strides, float eps, unsigned flags,
                         void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    return norm_rope_bwd({q_sig, k_sig, q_noise, k_noise}, strides, weight, positions, inv_freq,
                         {dq_sig, dk_sig, dq_noise, dk_noise}, {dq_sig_out, dk_sig_out, dq_noise_out, dk_noise_out},
                         dweight, T, h_s, h_n, d, rot, eps, flags, false, workspace, workspace_bytes, stream);
}

int gda_qk_norm_rope_bwd_f32(const float *q_sig, const float *k_sig, const float *q_noise, const float *k_noise,
                             const float *weight, const int *positions, const float *inv_freq, const float *dq_sig,
                             const float *dk_sig, const float *dq_noise, const float *dk_noise, float *dq_sig_out,
                             float *dk_sig_out, float *dq_noise_out, float *dk_noise_out, float *dweight, int T,
                             int h_s, int h_n, int d, int rot, const long long *strides, float eps, unsigned flags,
                             void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    return norm_rope_bwd({q_sig, k_sig, q_noise, k_noise}, strides, weight, positions, inv_freq,
                         {dq_sig, dk_sig, dq_noise, dk_noise}, {dq_sig_out, dk_sig_out, dq_noise_out, dk_noise_out},
                         dweight, T, h_s, h_n, d, rot, eps, flags, true, workspace, workspace_bytes, stream);
}

int gda_block_tables(const int *cache_lens, const int *new_lens, int *block_table, const int *free_pages,
                     const int *free_count, int *slot_map, int *positions, int *row_starts, int *lens_out,
                     int *free_count_out, int B, int max_pages, int page_size, int num_pages, int free_capacity,
                     int max_rows, gda_stream_t stream) {
    const void *ptrs[] = {cache_lens, new_lens, block_table, free_pages, free_count, slot_map, positions, row_starts,
                          lens_out, free_count_out};
    uintptr_t any = 0;
    for (const void *x : ptrs) {
        if (!x) return GDA_ERR_INVALID_ARG;
        any |= reinterpret_cast<uintptr_t>(x);
    }
    if (B < 1 || max_pages < 1 || page_size < 1 || num_pages < 1 || free_capacity < 1 || max_rows < 1)
        return GDA_ERR_INVALID_ARG;
    if (static_cast<long long>(max_pages) * page_size > 0x7fffffffLL ||
        static_cast<long long>(num_pages) * page_size > 0x7fffffffLL)
        return GDA_ERR_INVALID_ARG;
    if (B > kBlockTablesMaxB) return GDA_ERR_UNSUPPORTED;
    if (any & 3u) return GDA_ERR_MISALIGNED;
    BlockTablesArgs a{cache_lens, new_lens, block_table, free_pages, free_count, slot_map, positions, row_starts,
                      lens_out, free_count_out, B, max_pages, page_size, num_pages, free_capacity, max_rows, nullptr};
    const int st = current_device(&a.dev_err);
    if (st != GDA_OK) return st;
    return launch_block_tables(a, reinterpret_cast<cudaStream_t>(stream));
}

int gda_cache_append_fp8_block(const void *k_sig, const void *k_noise, const void *v, const int *slot_map,
                               void *k_sig_pool, void *k_noise_pool, void *v_pool, float *k_sig_scale,
                               float *k_noise_scale, float *v_scale, int8_t *k_sig_bounds, int8_t *k_noise_bounds, int T,
                               int num_pages, int page_size, int block, int h_s, int h_n, int d, int dv,
                               long long k_sig_stride, long long k_noise_stride, long long v_stride, void *workspace,
                               size_t workspace_bytes, gda_stream_t stream) {
    CacheFp8BlockArgs a{{k_sig, k_noise, v}, {k_sig_stride, k_noise_stride, v_stride}, slot_map,
                        {static_cast<uint8_t *>(k_sig_pool), static_cast<uint8_t *>(k_noise_pool),
                         static_cast<uint8_t *>(v_pool)},
                        {k_sig_scale, k_noise_scale, v_scale}, {k_sig_bounds, k_noise_bounds}, {}, {}, T, 0, block,
                        static_cast<int *>(workspace), nullptr};
    int st = fill_cache_fp8_block(a, num_pages, page_size, h_s, h_n, d, dv);
    if (st != GDA_OK) return st;
    const size_t need = gda_cache_append_fp8_block_workspace_size(T, num_pages, page_size);
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return GDA_ERR_WORKSPACE;
    if ((st = current_device(&a.dev_err)) != GDA_OK) return st;
    return launch_cache_append_fp8_block(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t gda_cache_append_fp8_block_workspace_size(int T, int num_pages, int page_size) {
    if (num_pages < 1 || page_size < 1 || static_cast<long long>(num_pages) * page_size > 0x7fffffffLL) return 0;
    if (T <= kCacheScanRows) return 0;
    return static_cast<size_t>(num_pages) * page_size * sizeof(int);
}

int gda_cache_read_fp8_block(const int *slot_map, const void *k_sig_pool, const void *k_noise_pool, const void *v_pool,
                             const float *k_sig_scale, const float *k_noise_scale, const float *v_scale,
                             void *k_sig_out, void *k_noise_out, void *v_out, int T, int num_pages, int page_size,
                             int block, int h_s, int h_n, int d, int dv, gda_stream_t stream) {
    auto pool = [](const void *x) { return const_cast<uint8_t *>(bytes_of(x)); };
    auto scale = [](const float *x) { return const_cast<float *>(x); };
    CacheFp8BlockArgs a{{k_sig_out, k_noise_out, v_out},
                        {static_cast<long long>(h_s) * d, static_cast<long long>(h_n) * d, static_cast<long long>(h_s) * dv},
                        slot_map, {pool(k_sig_pool), pool(k_noise_pool), pool(v_pool)},
                        {scale(k_sig_scale), scale(k_noise_scale), scale(v_scale)}, {}, {}, {}, T, 0, block, nullptr, nullptr};
    int st = fill_cache_fp8_block(a, num_pages, page_size, h_s, h_n, d, dv);
    if (st != GDA_OK) return st;
    if ((st = current_device(&a.dev_err)) != GDA_OK) return st;
    return launch_cache_read_fp8_block(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t gda_block_select_workspace_size(int B, int max_blocks, int h_s, int h_n) {
    if (B < 1 || max_blocks < 1 || h_s < 1 || h_n < 1 || h_s % h_n != 0) return 0;
    if (B > 65535 || max_blocks > kBlockSelectMaxBlocks || heads_above(h_s, h_n, 128)) return 0;
    return block_select_workspace_bytes(B, max_blocks, h_s, h_n);
}

int gda_block_select(const void *q_sig, const void *q_noise, const int8_t *k_sig_bounds, const int8_t *k_noise_bounds,
                     const float *k_sig_scale, const float *k_noise_scale, const int *block_table, const int *cache_lens,
                     int *block_list, int *block_count, int B, int max_pages, int page_size, int num_pages, int block,
                     int keep, int first, int last, int h_s, int h_n, int d, void *workspace, size_t workspace_bytes,
                     gda_stream_t stream) {
    if (!q_sig || !q_noise || !k_sig_bounds || !k_noise_bounds || !k_sig_scale || !k_noise_scale || !cache_lens ||
        !block_list || !block_count)
        return GDA_ERR_INVALID_ARG;
    if (B < 1 || max_pages < 1 || h_s < 1 || h_n < 1 || d < 1 || h_s % h_n != 0) return GDA_ERR_INVALID_ARG;
    if (keep < 1 || first < 0 || last < 0 || first > keep || last > keep - first) return GDA_ERR_INVALID_ARG;
    if (!block_table && (max_pages != 1 || num_pages != B)) return GDA_ERR_INVALID_ARG;
    int st = check_pages(num_pages, page_size, block);
    if (st != GDA_OK) return st;
    if (static_cast<long long>(max_pages) * page_size > 0x7fffffffLL) return GDA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128) || heads_above(h_s, h_n, 128) || B > 65535) return GDA_ERR_UNSUPPORTED;
    const long long most = static_cast<long long>(max_pages) * (page_size / block);
    if (most > kBlockSelectMaxBlocks || static_cast<double>(num_pages) * page_size > 4294967296.0)
        return GDA_ERR_UNSUPPORTED;
    if (!aligned16(q_sig) || !aligned16(q_noise) || !aligned16(k_sig_bounds) || !aligned16(k_noise_bounds))
        return GDA_ERR_MISALIGNED;
    if (!aligned4({k_sig_scale, k_noise_scale, block_table, cache_lens, block_list, block_count}))
        return GDA_ERR_MISALIGNED;
    const size_t need = block_select_workspace_bytes(B, static_cast<int>(most), h_s, h_n);
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return GDA_ERR_WORKSPACE;
    BlockSelectArgs a{q_sig, q_noise, k_sig_bounds, k_noise_bounds, k_sig_scale, k_noise_scale, block_table, cache_lens,
                      block_list, block_count, B, max_pages, page_size, num_pages, block, keep, first, last, h_s, h_n, d,
                      static_cast<float>(4.0 / 127.0 / std::log(2.0) / std::sqrt(static_cast<double>(d))),
                      static_cast<float *>(workspace), nullptr};
    if ((st = current_device(&a.dev_err)) != GDA_OK) return st;
    return launch_block_select(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t gda_attn_decode_fp8_block_workspace_size(int B, int h_s, int h_n, int d, int dv) {
    if (B < 1 || h_s < 1 || h_n < 1 || d < 1 || dv < 1 || h_s % h_n != 0) return 0;
    if (B > 65535 || heads_above(h_s, h_n, 128)) return 0;
    if (!(d == 64 || d == 128) || !(dv == 64 || dv == 128 || dv == 256)) return 0;
    return decode_fp8_block_workspace_bytes(B, h_s, h_n, d, dv);
}

int gda_attn_decode_fp8_block(const void *q_sig, const void *q_noise, const void *k_sig_cache, const void *k_noise_cache,
                              const void *v_cache, const float *k_sig_scale, const float *k_noise_scale,
                              const float *v_scale, const int *cache_lens, const float *lambda, float lambda_init,
                              void *out, int B, int Lcap, int block, int h_s, int h_n, int d, int dv, float eps,
                              void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    DecodeFp8BlockArgs a{q_sig, q_noise, bytes_of(k_sig_cache), bytes_of(k_noise_cache), bytes_of(v_cache), k_sig_scale,
                         k_noise_scale, v_scale, cache_lens, lambda, lambda_init, out, B, 0, block, h_s, h_n, d, dv, eps,
                         workspace, nullptr};
    a.page_size = Lcap, a.max_pages = 1, a.num_pages = B;
    return decode_fp8_block(a, workspace_bytes, stream);
}

int gda_attn_decode_paged_fp8_block(const void *q_sig, const void *q_noise, const void *k_sig_pool,
                                    const void *k_noise_pool, const void *v_pool, const float *k_sig_scale,
                                    const float *k_noise_scale, const float *v_scale, const int *block_table,
                                    const int *cache_lens, const float *lambda, float lambda_init, void *out, int B,
                                    int max_pages, int page_size, int num_pages, int block, int h_s, int h_n, int d,
                                    int dv, float eps, void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    if (!block_table) return GDA_ERR_INVALID_ARG;
    DecodeFp8BlockArgs a{q_sig, q_noise, bytes_of(k_sig_pool), bytes_of(k_noise_pool), bytes_of(v_pool), k_sig_scale,
                         k_noise_scale, v_scale, cache_lens, lambda, lambda_init, out, B, 0, block, h_s, h_n, d, dv, eps,
                         workspace, nullptr};
    a.block_table = block_table, a.page_size = page_size, a.max_pages = max_pages, a.num_pages = num_pages;
    return decode_fp8_block(a, workspace_bytes, stream);
}

int gda_attn_decode_sparse_fp8_block(const void *q_sig, const void *q_noise, const void *k_sig_pool,
                                     const void *k_noise_pool, const void *v_pool, const float *k_sig_scale,
                                     const float *k_noise_scale, const float *v_scale, const int *block_table,
                                     const int *block_list, const int *block_count, const int *cache_lens,
                                     const float *lambda, float lambda_init, void *out, int B, int max_pages,
                                     int page_size, int num_pages, int block, int keep, int h_s, int h_n, int d, int dv,
                                     float eps, void *workspace, size_t workspace_bytes, gda_stream_t stream) {
    if (!block_list || !block_count) return GDA_ERR_INVALID_ARG;
    if (!block_table && (max_pages != 1 || num_pages != B)) return GDA_ERR_INVALID_ARG;
    DecodeFp8BlockArgs a{q_sig, q_noise, bytes_of(k_sig_pool), bytes_of(k_noise_pool), bytes_of(v_pool), k_sig_scale,
                         k_noise_scale, v_scale, cache_lens, lambda, lambda_init, out, B, 0, block, h_s, h_n, d, dv, eps,
                         workspace, nullptr};
    a.block_table = block_table, a.page_size = page_size, a.max_pages = max_pages, a.num_pages = num_pages;
    a.list = block_list, a.count = block_count, a.keep = keep;
    return decode_fp8_block(a, workspace_bytes, stream);
}

const char *gda_status_string(int status) {
    switch (status) {
        case GDA_OK: return "success";
        case GDA_ERR_INVALID_ARG: return "invalid argument";
        case GDA_ERR_UNSUPPORTED: return "unsupported configuration or device";
        case GDA_ERR_MISALIGNED: return "pointer not 16-byte aligned";
        case GDA_ERR_WORKSPACE: return "workspace missing or too small";
        case GDA_ERR_CUDA: return "CUDA runtime or driver error";
        case GDA_ERR_DEVICE_TIMEOUT: return "a kernel wait timed out";
        default: return "unknown status";
    }
}

int gda_last_cuda_error(void) { return g_last_cuda_error; }

int gda_device_error(int clear) {
    unsigned *err = nullptr;
    const int st = current_device(&err);
    if (st != GDA_OK) return st;
    if (cudaDeviceSynchronize() != cudaSuccess) {
        cudaGetLastError();
        return GDA_ERR_CUDA;
    }
    unsigned v = 0;
    if (cudaMemcpy(&v, err, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) {
        cudaGetLastError();
        return GDA_ERR_CUDA;
    }
    if (clear && cudaMemset(err, 0, sizeof(unsigned)) != cudaSuccess) {
        cudaGetLastError();
        return GDA_ERR_CUDA;
    }
    return static_cast<int>(v & 0x7fffffffu);
}

}  // extern "C"
