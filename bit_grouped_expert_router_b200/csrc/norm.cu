// norm.cu -- the norms before and after a block, fused with its gate and the residual, and their
// gradient.  With h the residual stream, y the block's output and everything optional but h:
//
//   a  = y * r_post * w_post            r_post = 1 / sqrt(mean(y^2) + eps)      (norm_post, else 1)
//   h' = h + scale * gate_t * a         the new residual
//   n  = h' * r_pre * w_pre             r_pre = 1 / sqrt(mean(h'^2) + eps): the next block's input
//
// and backwards, from dn and the residual's own gradient dh'_in:
//
//   u  = dn * w_pre;  z = h' r_pre;  dh' = dh'_in + r_pre (u - z mean(u z));  dw_pre = sum_t dn z
//   da = scale gate_t dh';  x = y r_post;  dgate_t = scale <dh', a>;  dw_post = sum_t da x
//   v  = da * w_post;  dy = r_post (v - x mean(v x))  (norm_post, else v);  dh = dh'
//
// Bound by the bytes of the rows: each is read once, kept in registers across the row's two sums,
// and each result written once.  Sums and row factors are fp32 whatever the rows' type.
#include "ops_common.cuh"

namespace moe {

namespace {

// G warps share a row of up to G * 32 * 8 * V values; blocks of 256 threads hold 8 / G rows
// (G <= 8), wider rows have a block of G warps to themselves.
template <int G, int V> struct NormCfg {
    static constexpr int kThreads = G > 8 ? G * 32 : 256;
    static constexpr int kRows = G > 8 ? 1 : 8 / G;
    static constexpr int kSpan = G * 32 * 8;   // values covered by one piece of every thread
};

// Sum of NV values over the G warps of a row, every thread gets all sums.  red: [2][NV][G] per row,
// `flip` alternates between its halves so one barrier per sum is enough.
template <int G, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float* red, int& flip) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = warp_sum(v[i]);
    if constexpr (G > 1) {
        const int w = (threadIdx.x >> 5) % G;
        float* at = red + flip * 2 * G;
        flip ^= 1;
        if (lane_id() == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) at[i * G + w] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < G; ++j) s += at[i * G + j];
            v[i] = s;
        }
    }
}

template <typename TH, typename TY, int G, int V>
__global__ void __launch_bounds__(NormCfg<G, V>::kThreads) block_norm_kernel(NormArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    using C = NormCfg<G, V>;
    static_assert(G == 1 || C::kRows == 1, "rows of several warps have the block's barrier to themselves");
    __shared__ float red[4 * G];
    int flip = 0;
    const int g = threadIdx.x / (G * 32), l = threadIdx.x % (G * 32);
    const long long t = (long long)blockIdx.x * C::kRows + g;
    if (t >= a.T) return;   // a whole warp (G = 1) or no thread (one row per block)
    const size_t row = (size_t)t * a.H;
    Vec<TH, 8> hv[V];
    Vec<TY, 8> yv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * C::kSpan + l * 8;
        if (c < a.H) {
            hv[i].load(static_cast<const TH*>(a.h) + row + c);
            if (a.y) yv[i].load(static_cast<const TY*>(a.y) + row + c);
        }
    }
    float f = a.scale;
    if (a.gate) f *= a.gate[t];
    if (a.norm_post) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * C::kSpan + l * 8 < a.H) {
                float y[8];
                yv[i].get(y);
#pragma unroll
                for (int q = 0; q < 8; ++q) s[0] = fmaf(y[q], y[q], s[0]);
            }
        row_sum<G, 1>(s, red, flip);
        const float r = 1.f / sqrtf(s[0] / (float)a.H + a.eps);
        if (a.r_post && l == 0) a.r_post[t] = r;
        f *= r;
    }
    float h[V][8];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * C::kSpan + l * 8;
        if (c >= a.H) continue;
        hv[i].get(h[i]);
        if (a.y) {
            float y[8];
            yv[i].get(y);
            if (a.w_post) {
                Vec<float, 8> w;
                w.load(a.w_post + c);
                float wf[8];
                w.get(wf);
#pragma unroll
                for (int q = 0; q < 8; ++q) y[q] *= wf[q];
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) h[i][q] = fmaf(f, y[q], h[i][q]);
        }
        if (a.h_out) {
            Vec<TH, 8> o;
            o.set(h[i]);
            o.store(static_cast<TH*>(a.h_out) + row + c);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) s[0] = fmaf(h[i][q], h[i][q], s[0]);
    }
    if (!a.n_out && !a.r_pre) return;
    row_sum<G, 1>(s, red, flip);
    const float r = 1.f / sqrtf(s[0] / (float)a.H + a.eps);
    if (a.r_pre && l == 0) a.r_pre[t] = r;
    if (!a.n_out) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * C::kSpan + l * 8;
        if (c >= a.H) continue;
        float n[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) n[q] = h[i][q] * r;
        if (a.w_pre) {
            Vec<float, 8> w;
            w.load(a.w_pre + c);
            float wf[8];
            w.get(wf);
#pragma unroll
            for (int q = 0; q < 8; ++q) n[q] *= wf[q];
        }
        Vec<TY, 8> o;
        o.set(n);
        o.store(static_cast<TY*>(a.n_out) + row + c);
    }
}

// Blocks walk the rows and keep their share of the two weight gradients in registers; each block
// leaves one partial row per gradient and norm_reduce_kernel adds those in block order, so the
// sums do not change from run to run.
template <typename TH, typename TY, int G, int V>
__global__ void __launch_bounds__(NormCfg<G, V>::kThreads) block_norm_bwd_kernel(NormBwdArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    using C = NormCfg<G, V>;
    __shared__ float red[4 * G];
    __shared__ float fold[G == 1 ? 256 * V : 1];
    int flip = 0;
    const int g = threadIdx.x / (G * 32), l = threadIdx.x % (G * 32);
    const float inv = 1.f / (float)a.H;
    float gpre[V][8], gpost[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) gpre[i][q] = gpost[i][q] = 0.f;
    for (long long t = (long long)blockIdx.x * C::kRows + g; t < a.T; t += (long long)gridDim.x * C::kRows) {
        const size_t row = (size_t)t * a.H;
        Vec<TH, 8> hv[V], iv[V];
        Vec<TY, 8> nv[V], yv[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * C::kSpan + l * 8;
            if (c >= a.H) continue;
            if (a.dn) {
                hv[i].load(static_cast<const TH*>(a.h_out) + row + c);
                nv[i].load(static_cast<const TY*>(a.dn) + row + c);
            }
            if (a.dh_out) iv[i].load(static_cast<const TH*>(a.dh_out) + row + c);
            if (a.y) yv[i].load(static_cast<const TY*>(a.y) + row + c);
        }
        const float r = a.dn ? a.r_pre[t] : 0.f;
        float d[V][8];   // dh'
        if (a.dn) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * C::kSpan + l * 8;
                if (c >= a.H) continue;
                float z[8];
                hv[i].get(z);
                nv[i].get(d[i]);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    z[q] *= r;
                    gpre[i][q] = fmaf(d[i][q], z[q], gpre[i][q]);
                }
                if (a.w_pre) {
                    Vec<float, 8> w;
                    w.load(a.w_pre + c);
                    float wf[8];
                    w.get(wf);
#pragma unroll
                    for (int q = 0; q < 8; ++q) d[i][q] *= wf[q];
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) s[0] = fmaf(d[i][q], z[q], s[0]);
            }
            row_sum<G, 1>(s, red, flip);
            const float mean = s[0] * inv;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (i * C::kSpan + l * 8 >= a.H) continue;
                float z[8];
                hv[i].get(z);
#pragma unroll
                for (int q = 0; q < 8; ++q) d[i][q] = r * (d[i][q] - z[q] * r * mean);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int q = 0; q < 8; ++q) d[i][q] = 0.f;
        }
        const float rp = a.norm_post ? a.r_post[t] : 1.f;
        const float gt = a.gate ? a.gate[t] : 1.f;
        const float f = a.scale * gt;
        float s[1] = {0.f};   // <dh' w_post, x>: <v, x> but for the factor f, and <dh', a>
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * C::kSpan + l * 8;
            if (c >= a.H) continue;
            if (a.dh_out) {
                float in[8];
                iv[i].get(in);
#pragma unroll
                for (int q = 0; q < 8; ++q) d[i][q] += in[q];
            }
            if (a.dh) {
                Vec<TH, 8> o;
                o.set(d[i]);
                o.store(static_cast<TH*>(a.dh) + row + c);
            }
            if (!a.y) continue;
            float x[8], wf[8];
            yv[i].get(x);
            if (a.w_post) {
                Vec<float, 8> w;
                w.load(a.w_post + c);
                w.get(wf);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                x[q] *= rp;
                gpost[i][q] = fmaf(f * d[i][q], x[q], gpost[i][q]);
                if (a.w_post) d[i][q] *= wf[q];
                s[0] = fmaf(d[i][q], x[q], s[0]);
            }
        }
        if (!a.y) continue;
        if (a.norm_post || a.dgate) row_sum<G, 1>(s, red, flip);
        if (a.dgate && l == 0) a.dgate[t] = a.scale * s[0];
        if (a.dy) {
            const float mean = a.norm_post ? s[0] * inv : 0.f, fr = f * rp;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * C::kSpan + l * 8;
                if (c >= a.H) continue;
                float y[8];
                yv[i].get(y);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    d[i][q] = fr * (a.norm_post ? d[i][q] - y[q] * rp * mean : d[i][q]);
                Vec<TY, 8> o;
                o.set(d[i]);
                o.store(static_cast<TY*>(a.dy) + row + c);
            }
        }
    }
    for (int which = 0; which < 2; ++which) {
        if (which == 0 ? !a.dw_pre : !a.dw_post) continue;
        float* out = a.part + ((size_t)which * gridDim.x + blockIdx.x) * a.H;
        if constexpr (G == 1) {   // the block's eight warps in turn
            for (int w = 0; w < 8; ++w) {
                __syncthreads();
                if (g == w) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const float v = which == 0 ? gpre[i][q] : gpost[i][q];
                            float* at = fold + (i * 8 + q) * 32 + l;
                            *at = w == 0 ? v : *at + v;
                        }
                }
            }
            __syncthreads();
            for (int c = threadIdx.x; c < a.H; c += 256)
                out[c] = fold[((c / C::kSpan) * 8 + (c & 7)) * 32 + ((c % C::kSpan) >> 3)];
            __syncthreads();
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * C::kSpan + l * 8;
                if (c >= a.H) continue;
                Vec<float, 8> o;
                if (which == 0) o.set(gpre[i]);
                else o.set(gpost[i]);
                o.store(out + c);
            }
        }
    }
}

// dw[c] = sum over the blocks' partial rows, in a fixed order: 32 columns per block, 32 threads per
// column each over every 32nd row, then those 32 sums in order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* __restrict__ part, int rows, int H,
                                                           float* dw_pre, float* dw_post) {
    griddep_wait();
    griddep_launch_dependents();
    float* dw = blockIdx.y == 0 ? dw_pre : dw_post;
    if (!dw) return;
    __shared__ float s[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x, r0 = threadIdx.y;
    float v = 0.f;
    if (c < H)
        for (int r = r0; r < rows; r += 32) v += part[((size_t)blockIdx.y * rows + r) * H + c];
    s[r0][threadIdx.x] = v;
    __syncthreads();
    if (r0 == 0 && c < H) {
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) sum += s[r][threadIdx.x];
        dw[c] = sum;
    }
}

template <typename F> cudaError_t with_types(int h_dtype, int y_dtype, F f) {
    if (h_dtype == y_dtype) return with_dtype(h_dtype, [&](auto t) { return f(t, t); });
    if (h_dtype != MOE_DTYPE_FP32) return cudaErrorInvalidValue;
    return with_dtype(y_dtype, [&](auto t) { return f(float(), t); });
}

template <int G_, int V_> struct Geom {
    static constexpr int G = G_, V = V_;
};
// Warps per row by its width: narrow rows one warp each (no barrier), then a block of 256 with one,
// two or four pieces per thread, then 512 threads.
template <typename F> cudaError_t with_width(int H, F f) {
    if (H <= 256) return f(Geom<1, 1>());
    if (H <= 1024) return f(Geom<1, 4>());
    if (H <= 2048) return f(Geom<8, 1>());
    if (H <= 4096) return f(Geom<8, 2>());
    if (H <= 8192) return f(Geom<16, 2>());
    return f(Geom<16, 4>());
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, int h_dtype, int y_dtype, cudaStream_t st) {
    return with_types(h_dtype, y_dtype, [&](auto th, auto ty) {
        return with_width(a.H, [&](auto w) {
            using W = decltype(w);
            using C = NormCfg<W::G, W::V>;
            return launch_pdl(block_norm_kernel<decltype(th), decltype(ty), W::G, W::V>,
                              dim3((a.T + C::kRows - 1) / C::kRows), dim3(C::kThreads), 0, st, a);
        });
    });
}

int norm_bwd_ctas(int T, int H) {
    const int rows = H <= 1024 ? 8 : 1;
    const int want = (T + rows - 1) / rows;
    return want < kNormBwdCtas ? want : kNormBwdCtas;
}

cudaError_t launch_block_norm_bwd(const NormBwdArgs& a, int h_dtype, int y_dtype, cudaStream_t st) {
    const int ctas = norm_bwd_ctas(a.T, a.H);
    cudaError_t e = with_types(h_dtype, y_dtype, [&](auto th, auto ty) {
        return with_width(a.H, [&](auto w) {
            using W = decltype(w);
            using C = NormCfg<W::G, W::V>;
            return launch_pdl(block_norm_bwd_kernel<decltype(th), decltype(ty), W::G, W::V>, dim3(ctas),
                              dim3(C::kThreads), 0, st, a);
        });
    });
    if (e == cudaSuccess && (a.dw_pre || a.dw_post))
        e = launch_pdl(norm_reduce_kernel, dim3((a.H + 31) / 32, a.dw_post ? 2 : 1), dim3(32, 32), 0, st,
                       (const float*)a.part, ctas, a.H, a.dw_pre, a.dw_post);
    return e;
}

}  // namespace moe
