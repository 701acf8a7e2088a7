// ops.h -- internal interface between the C entry points of the operators around the experts
// (ops_api.cu) and their kernels (rows.cu, norm.cu, mx4.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encode_fn();   // cuTensorMapEncodeTiled (defined in api.cu; NULL if unavailable)

// ---- rows.cu: pairs sorted by expert, rows moved there and back -----------------------------------
constexpr int kSortThreads = 1024;       // pairs ranked at a time by one CTA of the general sort
constexpr int kSortMaxChunks = 148;      // the tokens are split into at most this many chunks (one CTA per SM)
constexpr int kSmallPairs = 4096;        // up to this many pairs one launch sorts and copies

struct SortArgs {
    const int* idx;
    int T, k, E;
    int n;          // T * k
    int chunk_tokens, nchunk;   // the general sort's chunks, of whole tokens
    int* offsets;
    int* perm;
    int* pos;
    int* hist;      // [nchunk][E] workspace of the general sort
    const uint4* x; // [T][nvec] rows as 16-byte vectors; NULL: sort only
    uint4* rows;
    int nvec;
};

cudaError_t launch_dispatch(const SortArgs& a, int num_sms, cudaStream_t st);

struct CombineArgs {
    const void* rows;
    int n_rows;
    const int* pos;
    const float* gates;     // NULL: every weight 1
    const void* base;       // NULL: zeros
    void* out;
    int T, k, H;
};
cudaError_t launch_combine(const CombineArgs& a, int dtype, cudaStream_t st);

struct CombineBwdArgs {
    const void* dout;
    const void* rows;
    int n_rows;
    const int* pos;
    const float* gates;
    void* drows;
    float* dgates;
    int T, k, H;
};
cudaError_t launch_combine_bwd(const CombineBwdArgs& a, int dtype, cudaStream_t st);
cudaError_t rows_take_status(uint32_t* host, cudaStream_t st);

// ---- norm.cu: the norms before and after a block ---------------------------------------------------
struct NormArgs {
    const void* h;
    const void* y;
    const float* w_post;
    const float* gate;
    const float* w_pre;
    void* h_out;
    void* n_out;
    float* r_post;
    float* r_pre;
    int T, H, norm_post;
    float scale, eps;
};
cudaError_t launch_block_norm(const NormArgs& a, int h_dtype, int y_dtype, cudaStream_t st);

constexpr int kNormBwdCtas = 148;   // most blocks of the backward pass (one per SM)
constexpr int kNormBwdStages = 4;   // most rows in flight per group of warps
struct NormBwdArgs {
    const void* dn;
    const void* dh_out;
    const void* h_out;
    const void* y;
    const float* r_pre;
    const float* r_post;
    const float* w_pre;
    const float* w_post;
    const float* gate;
    void* dh;
    void* dy;
    float* dw_pre;
    float* dw_post;
    float* dgate;
    float* part;     // [2][ctas][H] workspace
    int T, H, norm_post;
    float scale;
};
int norm_bwd_ctas(int T);
cudaError_t launch_block_norm_bwd(const NormBwdArgs& a, int h_dtype, int y_dtype, cudaStream_t st);
cudaError_t norm_take_status(uint32_t* host, cudaStream_t st);

// ---- mx4.cu: microscaled 4-bit floating point ------------------------------------------------------
struct Mx4QuantArgs {
    const void* x;
    int T, K;
    int swiglu;       // 1: x rows are [gate | up], 2K wide
    const int* pos;   // [T][k] destination rows, or NULL: row t
    int k;
    int n_rows;
    uint8_t* codes;   // [n_rows][K / 2]
    uint8_t* scales;  // [n_rows][K / 32]
};
cudaError_t launch_mx4_quantize(const Mx4QuantArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, long long rows, int K, void* out,
                                  int dtype, int num_sms, cudaStream_t st);

struct Mx4MatmulArgs {
    const uint8_t* scales;
    const uint8_t* w_scales;
    const int* offsets;
    void* y;
    int R, K, N, E;
};
constexpr int kMx4BoxRows = 32;    // rows of the token tile's TMA box
cudaError_t launch_mx4_matmul(const Mx4MatmulArgs& a, const CUtensorMap& tm_w, const CUtensorMap& tm_x, int dtype,
                              int num_sms, cudaStream_t st);
cudaError_t mx4_take_status(uint32_t* host, cudaStream_t st);

}  // namespace moe
