// ops_api.cu -- C entry points of the operators around the experts (include/moe.h): argument checks,
// workspaces and launches on the current device.  Host code only; the kernels are in rows.cu, norm.cu
// and mx4.cu.
#include <cuda.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "../../include/moe.h"
#include "common.cuh"
#include "kernels.h"
#include "ops.h"

using namespace moe;

namespace {

int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return code;
}

#define OPS_CHECK(cond, ...)                                          \
    do {                                                              \
        if (!(cond)) return fail(MOE_ERR_INVALID_ARG, __VA_ARGS__);   \
    } while (0)

// NVTX range around the call, then its launch's error.
struct Range {
    explicit Range(const char* name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};
int launched(const char* what, cudaError_t e) {
    return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool ok16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool null_or16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool null_or4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool dtype_ok(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_FP16 || d == MOE_DTYPE_FP32; }
int dtype_size(int d) { return d == MOE_DTYPE_FP32 ? 4 : 2; }

// The current device: sm_100 and its SM count.  Its context is made current too: in a thread that has made
// no CUDA call yet there is none, and the tensor-map encoder needs one.
int current_device(int* num_sms) {
    int dev = 0, major = 0, minor = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "current device: %s", cudaGetErrorString(e));
    if (major != 10 || minor != 0)
        return fail(MOE_ERR_UNSUPPORTED_DEVICE, "device %d is sm_%d%d; libmoe needs sm_100 (B200)", dev, major, minor);
    return MOE_OK;
}

constexpr int kMaxRowWidth = 65536;   // H of the moved rows

// Tokens per chunk of the sort: a whole round of its CTAs where that leaves no more CTAs than SMs.
int sort_chunk_tokens(int T, int k) { return std::max(kSortThreads / k, (T + kSortMaxChunks - 1) / kSortMaxChunks); }
int sort_chunks(int T, int k) { return (T + sort_chunk_tokens(T, k) - 1) / sort_chunk_tokens(T, k); }

int check_rows(int32_t dtype, int32_t T, int32_t k, int32_t H) {
    OPS_CHECK(dtype_ok(dtype), "unknown dtype %d", dtype);
    OPS_CHECK(T >= 0, "T must be >= 0 (got %d)", T);
    OPS_CHECK(k >= 1 && k <= 32, "k must be in [1, 32] (got %d)", k);
    OPS_CHECK((long long)T * k < (1ll << 30), "T * k must be below 2^30");
    OPS_CHECK(H >= 8 && H % 8 == 0 && H <= kMaxRowWidth, "H must be a multiple of 8 in [8, %d] (got %d)", kMaxRowWidth, H);
    return MOE_OK;
}

// 2-D map of 4-bit rows: [rows, bytes per row] uint8, box {128 bytes, box_rows}, 128-byte swizzle.
int encode_codes_map(CUtensorMap* m, const uint8_t* base, long long rows, int row_bytes, int box_rows) {
    EncodeTiledFn fn = tensor_map_encode_fn();
    if (!fn) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    const cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MOE_OK : fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

#define OPS_DEVICE(num_sms)                         \
    int num_sms = 0;                                \
    do {                                            \
        const int _rc = current_device(&num_sms);   \
        if (_rc != MOE_OK) return _rc;              \
    } while (0)

}  // namespace

extern "C" {

int moe_ops_status(void* stream) {
    OPS_DEVICE(sms);
    (void)sms;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t a = 0, b = 0, c = 0;
    cudaError_t e = cudaStreamSynchronize(st);
    static std::mutex one;   // a call's taken word is read before another call's take replaces it
    const std::lock_guard<std::mutex> lock(one);
    if (e == cudaSuccess) e = rows_take_status(&a, st);
    if (e == cudaSuccess) e = norm_take_status(&b, st);
    if (e == cudaSuccess) e = mx4_take_status(&c, st);
    if (e != cudaSuccess) return launched("moe_ops_status", e);
    if ((a | b | c) & MOE_STATUS_TIMEOUT) return fail(MOE_ERR_DEVICE_TIMEOUT, "a device-side wait timed out");
    if ((a | b | c) & MOE_STATUS_BOUNDS) return fail(MOE_ERR_DEVICE_BOUNDS, "a device-side index check failed");
    return MOE_OK;
}

size_t moe_dispatch_workspace(int32_t T, int32_t k, int32_t E) {
    if (T < 0 || k < 1 || k > 32 || E < 1 || E > 256 || (long long)T * k >= (1ll << 30)) return 0;
    return T * k <= kSmallPairs ? 0 : sizeof(int) * (size_t)sort_chunks(T, k) * E;
}

int moe_dispatch_rows(const void* x, int32_t dtype, int32_t T, int32_t H, const int32_t* idx, int32_t k, int32_t E,
                      void* rows, int32_t* offsets, int32_t* perm, int32_t* pos, void* workspace,
                      size_t workspace_bytes, void* stream) {
    const int rc = check_rows(dtype, T, k, H);
    if (rc != MOE_OK) return rc;
    OPS_CHECK(E >= 1 && E <= 256, "E must be in [1, 256] (got %d)", E);
    OPS_CHECK(ok4(offsets), "offsets is NULL or misaligned");
    const size_t need = moe_dispatch_workspace(T, k, E);
    if (T > 0) {
        OPS_CHECK(ok4(idx) && ok4(perm) && ok4(pos), "idx, perm or pos is NULL or misaligned");
        OPS_CHECK(!x == !rows, "x and rows must both be given, or neither");
        OPS_CHECK(null_or16(x) && null_or16(rows), "x and rows must be 16-byte aligned");
        OPS_CHECK(need == 0 || (ok16(workspace) && workspace_bytes >= need), "workspace of %zu bytes needed (got %zu)", need,
                  workspace_bytes);
    }
    OPS_DEVICE(sms);
    Range range("moe_dispatch_rows");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return launched("moe_dispatch_rows", cudaMemsetAsync(offsets, 0, sizeof(int) * (size_t)(E + 1), st));
    SortArgs a{};
    a.idx = idx;
    a.T = T; a.k = k; a.E = E; a.n = T * k;
    a.chunk_tokens = sort_chunk_tokens(T, k);
    a.nchunk = sort_chunks(T, k);
    a.offsets = offsets; a.perm = perm; a.pos = pos;
    a.hist = static_cast<int*>(workspace);
    a.x = static_cast<const uint4*>(x);
    a.rows = static_cast<uint4*>(rows);
    a.nvec = H * dtype_size(dtype) / 16;
    return launched("moe_dispatch_rows", launch_dispatch(a, sms, st));
}

static int combine(const char* name, const void* rows, int32_t dtype, int32_t n_rows, const int32_t* pos,
                   const float* gates, int32_t T, int32_t k, int32_t H, const void* base, void* out, void* stream) {
    const int rc = check_rows(dtype, T, k, H);
    if (rc != MOE_OK) return rc;
    OPS_CHECK(n_rows >= 0, "n_rows must be >= 0 (got %d)", n_rows);
    if (T == 0) return MOE_OK;
    OPS_CHECK(ok4(pos) && ok16(out) && null_or16(base) && null_or4(gates) && (n_rows == 0 || ok16(rows)),
              "%s: a pointer is NULL or misaligned", name);
    OPS_DEVICE(sms);
    (void)sms;
    Range range(name);
    const CombineArgs a{rows, n_rows, pos, gates, base, out, T, k, H};
    return launched(name, launch_combine(a, dtype, static_cast<cudaStream_t>(stream)));
}

int moe_dispatch_rows_backward(const void* drows, int32_t dtype, int32_t n_rows, const int32_t* pos, int32_t T,
                               int32_t k, int32_t H, void* dx, void* stream) {
    return combine("moe_dispatch_rows_backward", drows, dtype, n_rows, pos, nullptr, T, k, H, nullptr, dx, stream);
}

int moe_combine_weighted(const void* rows, int32_t dtype, int32_t n_rows, const int32_t* pos, const float* gates,
                         int32_t T, int32_t k, int32_t H, const void* base, void* out, void* stream) {
    OPS_CHECK(T <= 0 || gates, "gates is NULL");
    return combine("moe_combine_weighted", rows, dtype, n_rows, pos, gates, T, k, H, base, out, stream);
}

int moe_combine_weighted_backward(const void* dout, int32_t dtype, const void* rows, int32_t n_rows,
                                  const int32_t* pos, const float* gates, int32_t T, int32_t k, int32_t H,
                                  void* drows, float* dgates, void* stream) {
    const int rc = check_rows(dtype, T, k, H);
    if (rc != MOE_OK) return rc;
    OPS_CHECK(n_rows >= 0, "n_rows must be >= 0 (got %d)", n_rows);
    if (T == 0) return MOE_OK;
    OPS_CHECK(ok16(dout) && ok4(pos) && ok4(gates) && ok4(dgates) && (n_rows == 0 || (ok16(rows) && ok16(drows))),
              "moe_combine_weighted_backward: a pointer is NULL or misaligned");
    OPS_DEVICE(sms);
    (void)sms;
    Range range("moe_combine_weighted_backward");
    const CombineBwdArgs a{dout, rows, n_rows, pos, gates, drows, dgates, T, k, H};
    return launched("moe_combine_weighted_backward", launch_combine_bwd(a, dtype, static_cast<cudaStream_t>(stream)));
}

constexpr int kMaxNormWidth = 16384;

static int check_norm(int32_t h_dtype, int32_t y_dtype, int32_t T, int32_t H, int32_t norm_post) {
    OPS_CHECK(dtype_ok(h_dtype) && dtype_ok(y_dtype) && (h_dtype == y_dtype || h_dtype == MOE_DTYPE_FP32),
              "unsupported types: the residual (%d) must have the block's type (%d) or be fp32", h_dtype, y_dtype);
    OPS_CHECK(T >= 0, "T must be >= 0 (got %d)", T);
    OPS_CHECK(H >= 8 && H % 8 == 0 && H <= kMaxNormWidth, "H must be a multiple of 8 in [8, %d] (got %d)", kMaxNormWidth, H);
    OPS_CHECK(norm_post == 0 || norm_post == 1, "norm_post must be 0 or 1");
    return MOE_OK;
}

int moe_block_norm(const void* h, int32_t h_dtype, const void* y, int32_t y_dtype, int32_t T, int32_t H,
                   const float* w_post, int32_t norm_post, const float* gate, float scale, const float* w_pre, float eps,
                   void* h_out, void* n_out, float* r_post, float* r_pre, void* stream) {
    const int rc = check_norm(h_dtype, y_dtype, T, H, norm_post);
    if (rc != MOE_OK) return rc;
    OPS_CHECK(eps >= 0.f, "eps must be >= 0");
    if (T == 0) return MOE_OK;   // (an empty tensor's address is NULL)
    OPS_CHECK(y || (!w_post && !gate && !norm_post), "w_post, gate and norm_post need y");
    OPS_CHECK(!r_post || norm_post, "r_post needs norm_post");
    OPS_CHECK(ok16(h) && null_or16(y) && null_or16(w_post) && null_or16(w_pre) && null_or4(gate) && null_or16(h_out) &&
                  null_or16(n_out) && null_or4(r_post) && null_or4(r_pre),
              "moe_block_norm: a pointer is NULL or misaligned");
    OPS_DEVICE(sms);
    (void)sms;
    Range range("moe_block_norm");
    const NormArgs a{h, y, w_post, gate, w_pre, h_out, n_out, r_post, r_pre, T, H, norm_post, scale, eps};
    return launched("moe_block_norm", launch_block_norm(a, h_dtype, y_dtype, static_cast<cudaStream_t>(stream)));
}

size_t moe_block_norm_backward_workspace(int32_t T, int32_t H) {
    if (T < 0 || H < 8 || H % 8 != 0 || H > kMaxNormWidth) return 0;
    return sizeof(float) * 2 * (size_t)norm_bwd_ctas(T) * H;
}

int moe_block_norm_backward(const void* dn, const void* dh_out, const void* h_out, int32_t h_dtype, const void* y,
                            int32_t y_dtype, int32_t T, int32_t H, const float* r_pre, const float* r_post,
                            const float* w_pre, const float* w_post, int32_t norm_post, const float* gate, float scale,
                            void* dh, void* dy, float* dw_pre, float* dw_post, float* dgate, void* workspace,
                            size_t workspace_bytes, void* stream) {
    const int rc = check_norm(h_dtype, y_dtype, T, H, norm_post);
    if (rc != MOE_OK) return rc;
    OPS_CHECK(null_or16(dw_pre) && null_or16(dw_post), "dw_pre and dw_post must be 16-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T > 0) {   // (an empty tensor's address is NULL)
        OPS_CHECK(y || (!w_post && !gate && !norm_post && !dy && !dw_post && !dgate),
                  "w_post, gate, norm_post, dy, dw_post and dgate need y");
        OPS_CHECK(dn || (!dw_pre && !w_pre), "w_pre and dw_pre need dn");
        OPS_CHECK(!dn || (ok16(dn) && ok16(h_out) && ok4(r_pre)), "dn needs h_out and r_pre (16- and 4-byte aligned)");
        OPS_CHECK(!norm_post || ok4(r_post), "norm_post needs r_post");
        OPS_CHECK(null_or16(dh_out) && null_or16(y) && null_or16(w_pre) && null_or16(w_post) && null_or4(gate) &&
                      null_or16(dh) && null_or16(dy) && null_or4(dgate),
                  "moe_block_norm_backward: a pointer is misaligned");
        const size_t need = dw_pre || dw_post ? moe_block_norm_backward_workspace(T, H) : 0;
        OPS_CHECK(need == 0 || (ok16(workspace) && workspace_bytes >= need), "workspace of %zu bytes needed (got %zu)", need,
                  workspace_bytes);
    }
    OPS_DEVICE(sms);
    (void)sms;
    Range range("moe_block_norm_backward");
    if (T == 0) {   // the sums over no rows
        cudaError_t e = dw_pre ? cudaMemsetAsync(dw_pre, 0, sizeof(float) * H, st) : cudaSuccess;
        if (e == cudaSuccess && dw_post) e = cudaMemsetAsync(dw_post, 0, sizeof(float) * H, st);
        return launched("moe_block_norm_backward", e);
    }
    const NormBwdArgs a{dn, dh_out, h_out, y, r_pre, r_post, w_pre, w_post, gate, dh, dy, dw_pre, dw_post, dgate,
                        static_cast<float*>(workspace), T, H, norm_post, scale};
    return launched("moe_block_norm_backward", launch_block_norm_bwd(a, h_dtype, y_dtype, st));
}

constexpr int kMaxMx4Width = 65536;

int moe_mx4_quantize(const void* x, int32_t dtype, int32_t T, int32_t K, int32_t act, const int32_t* pos, int32_t k,
                     int32_t n_rows, uint8_t* codes, uint8_t* scales, void* stream) {
    OPS_CHECK(dtype_ok(dtype), "unknown dtype %d", dtype);
    OPS_CHECK(T >= 0 && n_rows >= 0, "T and n_rows must be >= 0");
    OPS_CHECK(K >= 32 && K % 32 == 0 && K <= kMaxMx4Width, "K must be a multiple of 32 in [32, %d] (got %d)", kMaxMx4Width, K);
    OPS_CHECK((long long)T * K < (1ll << 35), "T * K must be below 2^35");
    OPS_CHECK(act == MOE_ACT_NONE || act == MOE_ACT_SWIGLU, "unknown act %d", act);
    OPS_CHECK(!pos || (k >= 1 && k <= 32 && (long long)T * k < (1ll << 30)), "k must be in [1, 32] and T * k below 2^30");
    OPS_CHECK(pos || n_rows >= T, "n_rows = %d rows cannot hold T = %d", n_rows, T);
    if (T == 0) return MOE_OK;
    OPS_CHECK(ok16(x) && (n_rows == 0 || (ok16(codes) && ok16(scales))) && null_or4(pos),
              "moe_mx4_quantize: a pointer is NULL or misaligned");
    OPS_DEVICE(sms);
    (void)sms;
    Range range("moe_mx4_quantize");
    const Mx4QuantArgs a{x, T, K, act == MOE_ACT_SWIGLU, pos, k, n_rows, codes, scales};
    return launched("moe_mx4_quantize", launch_mx4_quantize(a, dtype, static_cast<cudaStream_t>(stream)));
}

int moe_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t K, void* out, int32_t dtype,
                       void* stream) {
    OPS_CHECK(dtype_ok(dtype), "unknown dtype %d", dtype);
    OPS_CHECK(rows >= 0 && rows < (1ll << 40), "rows must be in [0, 2^40)");
    OPS_CHECK(K >= 32 && K % 32 == 0 && K <= kMaxMx4Width, "K must be a multiple of 32 in [32, %d] (got %d)", kMaxMx4Width, K);
    if (rows == 0) return MOE_OK;
    OPS_CHECK(ok16(codes) && ok16(scales) && ok16(out), "moe_mx4_dequantize: a pointer is NULL or misaligned");
    OPS_DEVICE(sms);
    Range range("moe_mx4_dequantize");
    return launched("moe_mx4_dequantize",
                    launch_mx4_dequantize(codes, scales, rows, K, out, dtype, sms, static_cast<cudaStream_t>(stream)));
}

int moe_mx4_matmul(const uint8_t* codes, const uint8_t* scales, int32_t n_rows, int32_t K, const uint8_t* w_codes,
                   const uint8_t* w_scales, int32_t E, int32_t N, const int32_t* offsets, void* y, int32_t dtype,
                   void* stream) {
    OPS_CHECK(dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_FP32, "y must be bf16 or fp32 (dtype %d)", dtype);
    OPS_CHECK(n_rows >= 0 && n_rows <= (1 << 30), "n_rows must be in [0, 2^30]");
    OPS_CHECK(K >= 32 && K % 32 == 0 && K <= kMaxMx4Width, "K must be a multiple of 32 in [32, %d] (got %d)", kMaxMx4Width, K);
    OPS_CHECK(E >= 1 && E <= 256, "E must be in [1, 256] (got %d)", E);
    OPS_CHECK(N >= 8 && N % 8 == 0 && (long long)E * N < (1ll << 31), "N must be a multiple of 8 with E * N < 2^31 (got %d)", N);
    OPS_CHECK(((long long)n_rows / 64 + E) * ((N + 127) / 128) < (1ll << 30), "too many tiles: n_rows = %d, N = %d", n_rows, N);
    if (n_rows == 0) return MOE_OK;
    OPS_CHECK(ok16(codes) && ok16(scales) && ok16(w_codes) && ok16(w_scales) && ok4(offsets) && ok16(y),
              "moe_mx4_matmul: a pointer is NULL or misaligned");
    OPS_DEVICE(sms);
    Range range("moe_mx4_matmul");
    CUtensorMap tm_w, tm_x;
    int rc = encode_codes_map(&tm_w, w_codes, (long long)E * N, K / 2, 128);
    if (rc == MOE_OK) rc = encode_codes_map(&tm_x, codes, n_rows, K / 2, kMx4BoxRows);
    if (rc != MOE_OK) return rc;
    const Mx4MatmulArgs a{scales, w_scales, offsets, y, n_rows, K, N, E};
    return launched("moe_mx4_matmul", launch_mx4_matmul(a, tm_w, tm_x, dtype, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
