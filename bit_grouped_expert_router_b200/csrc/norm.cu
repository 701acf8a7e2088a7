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
// Bound by the bytes of the rows: each is read once, kept on the chip across the row's two sums, and
// each result written once (forward, 16384 x 2048 bf16 with both norms: 45 us, 6.0 TB/s; gradient, 4096 x
// 2048 with an fp32 stream: 32 us, 4.7 TB/s).  Sums and row factors are fp32 whatever the rows' type.
#include <type_traits>

#include "ops_common.cuh"

namespace moe {

namespace {

// G warps share a row of up to G * 32 * 8 * V values, V pieces of eight per thread; blocks of 128 threads
// hold 4 / G rows, wider rows have a block of G warps to themselves.
template <int G, int V> struct NormCfg {
    static constexpr int kThreads = G > 4 ? G * 32 : 128;
    static constexpr int kRows = G > 4 ? 1 : 4 / G;
    static constexpr int kSpan = G * 32 * 8;   // values covered by one piece of every thread
};

// Sum of v over the G warps of a row, the same in every thread.  red: [rows][2][G]; `flip` alternates
// between a row's halves, so one barrier of the row's warps per sum is enough.
template <int G>
__device__ __forceinline__ float row_sum(float v, float* red, int& flip, int row) {
    v = warp_sum(v);
    if constexpr (G > 1) {
        float* at = red + (row * 2 + flip) * G;
        flip ^= 1;
        if (lane_id() == 0) at[(threadIdx.x >> 5) % G] = v;
        named_bar(1 + row, G * 32);
        // lane i takes warp i % G's sum; the exchanges leave the same total, added in the same order, everywhere
        v = at[lane_id() % G];
#pragma unroll
        for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    }
    return v;
}

__device__ __forceinline__ void load_weights(const float* p, float (&v)[8]) {
    Vec<float, 8> w;
    w.load(p);
    w.get(v);
}

template <typename TH, typename TY, int G, int V>
__global__ void __launch_bounds__(NormCfg<G, V>::kThreads) block_norm_kernel(NormArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    using C = NormCfg<G, V>;
    __shared__ float red[C::kRows * 2 * G];
    int flip = 0;
    const int g = threadIdx.x / (G * 32), l = threadIdx.x % (G * 32);
    const float inv = 1.f / (float)a.H;
    const long long t = (long long)blockIdx.x * C::kRows + g;
    if (t >= a.T) return;   // all warps of the row
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
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * C::kSpan + l * 8 < a.H) {
                float y[8];
                yv[i].get(y);
#pragma unroll
                for (int q = 0; q < 8; ++q) s = fmaf(y[q], y[q], s);
            }
        s = row_sum<G>(s, red, flip, g);
        const float r = rsqrtf(fmaf(s, inv, a.eps));
        if (a.r_post && l == 0) a.r_post[t] = r;
        f *= r;
    }
    float h[V][8];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * C::kSpan + l * 8;
        if (c >= a.H) continue;
        hv[i].get(h[i]);
        if (a.y) {
            float y[8];
            yv[i].get(y);
            if (a.w_post) {
                float wf[8];
                load_weights(a.w_post + c, wf);
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
        for (int q = 0; q < 8; ++q) s = fmaf(h[i][q], h[i][q], s);
    }
    if (!a.n_out && !a.r_pre) return;
    s = row_sum<G>(s, red, flip, g);
    const float r = rsqrtf(fmaf(s, inv, a.eps));
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
            float wf[8];
            load_weights(a.w_pre + c, wf);
#pragma unroll
            for (int q = 0; q < 8; ++q) n[q] *= wf[q];
        }
        Vec<TY, 8> o;
        o.set(n);
        o.store(static_cast<TY*>(a.n_out) + row + c);
    }
}

// One block per SM, in groups of G warps that each walk rows of their own and keep their share of the two
// weight gradients; the block folds its groups' shares and leaves one partial row per gradient, and
// norm_reduce_kernel adds those in block order, so the sums do not change from run to run.  (Blocks of
// one row with a partial each, 592 of them: 45.2 us for 4096 x 2048, a third of it for the partials.)
//
// Bulk copies bring a group's next rows into its ring of `stages` shared-memory buffers while this one is
// worked on, so the loads in flight do not hang on the registers a row needs.  The weights lie behind the
// rings (read from global memory for every row they cost 12 of 42 us: the rings leave the first cache
// level no room).  Rows too wide for two buffers and the weights are read from global memory (RING false).
struct BwdRing {
    int stages;
    int n_off, i_off, y_off;   // of dn, dh_out and y in a stage (h_out first)
    int stage_bytes;
    int w_off;                 // of the weights' copies behind the rings: w_pre, then w_post
};

template <int G> struct BwdCfg {
    static constexpr int kMaxThreads = G == 32 ? 1024 : 512;
    static constexpr int kMaxGroups = kMaxThreads / (G * 32);
};

// Whether `ok` holds in all threads of the group; a barrier of the group.
template <int G> __device__ __forceinline__ bool group_all(bool ok, int g) {
    if constexpr (G == 1) return __all_sync(0xffffffffu, ok);
    else return !named_bar_or(1 + g, G * 32, !ok);
}

template <typename TH, typename TY, int G, int V, bool RING>
__global__ void __launch_bounds__(BwdCfg<G>::kMaxThreads, 1) block_norm_bwd_kernel(NormBwdArgs a, BwdRing ring) {
    constexpr int kSpan = G * 32 * 8, kMaxGroups = BwdCfg<G>::kMaxGroups;
    __shared__ float red[kMaxGroups * 2 * G];
    __shared__ __align__(8) uint64_t bars[kMaxGroups * kNormBwdStages];
    __shared__ int abort_word;
    extern __shared__ __align__(16) uint8_t dyn[];   // rings [group][stage], then the fold; or sums (kShared)
    const int groups = blockDim.x / (G * 32), threads = blockDim.x;
    const int g = threadIdx.x / (G * 32), l = threadIdx.x % (G * 32);
    uint64_t* full = bars + g * kNormBwdStages;
    uint8_t* mine = dyn + (size_t)g * ring.stages * ring.stage_bytes;
    int flip = 0;
    const float inv = 1.f / (float)a.H;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxGroups * kNormBwdStages; ++i) mbar_init(&bars[i], 1);
        abort_word = 0;
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    // The block's sums for the two weight gradients: in registers, for the widest rows (1024 threads of 64
    // registers) in shared memory, every thread its own columns either way.
    constexpr bool kShared = G == 32;
    float4* sums = reinterpret_cast<float4*>(dyn);   // [2][V][2][threads]
    float gsum[2][kShared ? 1 : V][8];
    if constexpr (kShared) {
        for (int i = 0; i < 4 * V; ++i) sums[i * threads + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int q = 0; q < 8; ++q) gsum[0][i][q] = gsum[1][i][q] = 0.f;
    }
    auto add = [&](auto which, int i, const float (&u)[8], const float (&v)[8]) {   // += u v
        constexpr int kWhich = decltype(which)::value;
        if constexpr (kShared) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4& at = sums[((kWhich * V + i) * 2 + h) * threads + threadIdx.x];
                float4 o = at;
                o.x = fmaf(u[4 * h], v[4 * h], o.x);
                o.y = fmaf(u[4 * h + 1], v[4 * h + 1], o.y);
                o.z = fmaf(u[4 * h + 2], v[4 * h + 2], o.z);
                o.w = fmaf(u[4 * h + 3], v[4 * h + 3], o.w);
                at = o;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) gsum[kWhich][i][q] = fmaf(u[q], v[q], gsum[kWhich][i][q]);
        }
    };
    using Pre = std::integral_constant<int, 0>;
    using Post = std::integral_constant<int, 1>;
    // the group's n-th row is blockIdx.x + (g + n groups) gridDim.x
    const long long first = blockIdx.x + (long long)g * gridDim.x, stride = (long long)groups * gridDim.x;
    auto issue = [&](int n) {   // that row into its stage (one thread of the group)
        const long long t = first + n * stride;
        if (t >= a.T) return;
        const int s = n % ring.stages;
        uint8_t* st = mine + s * ring.stage_bytes;
        const size_t at = (size_t)t * a.H;
        const uint32_t nh = a.H * sizeof(TH), ny = a.H * sizeof(TY);
        mbar_arrive_expect_tx(&full[s], (a.dn ? nh + ny : 0) + (a.dh_out ? nh : 0) + (a.y ? ny : 0));
        if (a.dn) {
            bulk_g2s(st, static_cast<const TH*>(a.h_out) + at, nh, &full[s]);
            bulk_g2s(st + ring.n_off, static_cast<const TY*>(a.dn) + at, ny, &full[s]);
        }
        if (a.dh_out) bulk_g2s(st + ring.i_off, static_cast<const TH*>(a.dh_out) + at, nh, &full[s]);
        if (a.y) bulk_g2s(st + ring.y_off, static_cast<const TY*>(a.y) + at, ny, &full[s]);
    };
    const float *wpre = a.w_pre, *wpost = a.w_post;
    if constexpr (RING) {
        if (l == 0)
            for (int n = 0; n < ring.stages - 1; ++n) issue(n);
        float4* to = reinterpret_cast<float4*>(dyn + ring.w_off);
        for (int i = threadIdx.x; i < a.H / 4; i += threads) {
            if (a.w_pre) to[i] = reinterpret_cast<const float4*>(a.w_pre)[i];
            if (a.w_post) to[a.H / 4 + i] = reinterpret_cast<const float4*>(a.w_post)[i];
        }
        wpre = reinterpret_cast<const float*>(to);
        wpost = wpre + a.H;
        __syncthreads();
    }
    float r_next = 0.f, rp_next = 1.f, gate_next = 1.f;   // the next row's factors, a row ahead as well
    auto factors = [&](long long t) {
        if (t >= a.T) return;
        if (a.dn) r_next = a.r_pre[t];
        if (a.norm_post) rp_next = a.r_post[t];
        if (a.gate) gate_next = a.gate[t];
    };
    factors(first);
    int n = 0;
    for (long long t = first; t < a.T; t += stride, ++n) {
        const size_t row = (size_t)t * a.H;
        const float r = r_next, rp = rp_next, f = a.scale * gate_next, fr = f * rp;
        factors(t + stride);
        const TH *hrow, *irow;
        const TY *nrow, *yrow;
        if constexpr (RING) {
            const int s = n % ring.stages;
            const bool ok = mbar_wait(&full[s], (n / ring.stages) & 1u, &abort_word, g_ops_status);
            // all of the group's threads are past the row before: its stage takes the row stages - 1 ahead
            if (!group_all<G>(ok, g)) break;
            if (l == 0) issue(n + ring.stages - 1);
            const uint8_t* st = mine + s * ring.stage_bytes;
            hrow = reinterpret_cast<const TH*>(st);
            nrow = reinterpret_cast<const TY*>(st + ring.n_off);
            irow = reinterpret_cast<const TH*>(st + ring.i_off);
            yrow = reinterpret_cast<const TY*>(st + ring.y_off);
        } else {
            hrow = static_cast<const TH*>(a.h_out) + row;
            nrow = static_cast<const TY*>(a.dn) + row;
            irow = static_cast<const TH*>(a.dh_out) + row;
            yrow = static_cast<const TY*>(a.y) + row;
        }
        float d[V][8];   // dh'
        if (a.dn) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * kSpan + l * 8;
                if (c >= a.H) continue;
                Vec<TH, 8> hv;
                Vec<TY, 8> nv;
                hv.load(hrow + c);
                nv.load(nrow + c);
                float z[8];
                hv.get(z);
                nv.get(d[i]);
#pragma unroll
                for (int q = 0; q < 8; ++q) z[q] *= r;
                add(Pre(), i, d[i], z);
                if (a.w_pre) {
                    float wf[8];
                    load_weights(wpre + c, wf);
#pragma unroll
                    for (int q = 0; q < 8; ++q) d[i][q] *= wf[q];
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) s = fmaf(d[i][q], z[q], s);
            }
            s = row_sum<G>(s, red, flip, g);
            const float k = -(s * inv) * r;   // (z = h' r comes first: r^2 alone may leave the range of fp32)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * kSpan + l * 8;
                if (c >= a.H) continue;
                Vec<TH, 8> hv;
                hv.load(hrow + c);
                float h[8];
                hv.get(h);
#pragma unroll
                for (int q = 0; q < 8; ++q) d[i][q] = fmaf(h[q] * r, k, r * d[i][q]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int q = 0; q < 8; ++q) d[i][q] = 0.f;
        }
        float s = 0.f;   // <dh' w_post, y>: times r_post, <v, x> but for the factor f, and <dh', a>
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * kSpan + l * 8;
            if (c >= a.H) continue;
            if (a.dh_out) {
                Vec<TH, 8> iv;
                iv.load(irow + c);
                float in[8];
                iv.get(in);
#pragma unroll
                for (int q = 0; q < 8; ++q) d[i][q] += in[q];
            }
            if (a.dh) {
                Vec<TH, 8> o;
                o.set(d[i]);
                o.store(static_cast<TH*>(a.dh) + row + c);
            }
            if (!a.y) continue;
            Vec<TY, 8> yv;
            yv.load(yrow + c);
            float y[8], x[8];
            yv.get(y);
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = fr * y[q];
            add(Post(), i, d[i], x);
            if (a.w_post) {
                float wf[8];
                load_weights(wpost + c, wf);
#pragma unroll
                for (int q = 0; q < 8; ++q) d[i][q] *= wf[q];
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) s = fmaf(d[i][q], y[q], s);
        }
        if (!a.y) continue;
        if (a.norm_post || a.dgate) s = row_sum<G>(s, red, flip, g) * rp;
        if (a.dgate && l == 0) a.dgate[t] = a.scale * s;
        if (a.dy) {
            const float k = a.norm_post ? -(s * inv) * fr : 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * kSpan + l * 8;
                if (c >= a.H) continue;
                Vec<TY, 8> yv;
                yv.load(yrow + c);
                float y[8];
                yv.get(y);
#pragma unroll
                for (int q = 0; q < 8; ++q) d[i][q] = fr * d[i][q];
                if (a.norm_post) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) d[i][q] = fmaf(y[q] * rp, k, d[i][q]);
                }
                Vec<TY, 8> o;
                o.set(d[i]);
                o.store(static_cast<TY*>(a.dy) + row + c);
            }
        }
    }
    if (RING && l == 0 && abort_word)   // copies still in flight land before the block ends
        for (int i = 0; i < ring.stages - 1; ++i)
            if (first + (n + i) * stride < a.T) mbar_drain(&full[(n + i) % ring.stages], ((n + i) / ring.stages) & 1u);
    float* fold = reinterpret_cast<float*>(dyn);   // the rings are free by then
    for (int which = 0; which < 2; ++which) {
        if (which == 0 ? !a.dw_pre : !a.dw_post) continue;
        float* out = a.part + ((size_t)which * gridDim.x + blockIdx.x) * a.H;
        for (int w = 0; w < groups; ++w) {   // the groups in turn
            __syncthreads();
            if (g != w) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * kSpan + l * 8;
                if (c >= a.H) continue;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 v;
                    if constexpr (kShared) {
                        v = sums[((which * V + i) * 2 + h) * threads + threadIdx.x];
                    } else {
                        const float* u = which == 0 ? &gsum[0][i][4 * h] : &gsum[1][i][4 * h];
                        v = make_float4(u[0], u[1], u[2], u[3]);
                    }
                    if (w > 0) {
                        const float4 o = reinterpret_cast<const float4*>(fold + c)[h];
                        v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
                    }
                    if (w == groups - 1) reinterpret_cast<float4*>(out + c)[h] = v;
                    else reinterpret_cast<float4*>(fold + c)[h] = v;
                }
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
// Many rows: 16 or 32 values per thread, so that the sums across threads, the factors and the barriers (some
// 130 instructions a thread and row) are spread over them.  33.5 M bf16 values with both norms, in us, at
// widths 1024 / 2048 / 4096 / 8192 / 16384: this choice 46 / 45 / 47 / 48 / 56; 64 values each 46 / 50 / 52 / 52 / 66;
// 16 values each 67 / 45 / 48 / 57 / 69; 8 values at 2048: 51, bound by its instructions, 41 a value.
template <typename F> cudaError_t with_width(int H, F f) {
    if (H <= 256) return f(Geom<1, 1>());
    if (H <= 512) return f(Geom<1, 2>());
    if (H <= 1024) return f(Geom<1, 4>());
    if (H <= 2048) return f(Geom<4, 2>());
    if (H <= 4096) return f(Geom<4, 4>());
    if (H <= 8192) return f(Geom<8, 4>());
    return f(Geom<16, 4>());
}
// Few rows, bound by the latency of one: as many warps per row as its values allow.  Few / many rows' choice, in us
// (both norms, bf16): 512 x 2048 3.0 / 3.2 and 2048 x 2048 8.3 / 8.5, 128 x 1024 2.1 / 3.6 and 2048 x 1024 4.3 / 4.5,
// 1024 x 512 2.5 / 2.8 and 2048 x 512 4.0 / 3.1, 256 x 4096 3.1 / 4.2 and 1024 x 4096 9.3 / 7.6.
bool many_rows(int T, int H) { return T >= 2048 || (long long)T * H >= 1 << 21; }
template <typename F> cudaError_t with_width_few(int H, F f) {
    if (H <= 256) return f(Geom<1, 1>());
    if (H <= 512) return f(Geom<2, 1>());
    if (H <= 1024) return f(Geom<4, 1>());
    if (H <= 2048) return f(Geom<8, 1>());
    if (H <= 4096) return f(Geom<16, 1>());
    if (H <= 8192) return f(Geom<32, 1>());
    return f(Geom<32, 2>());
}
// The backward pass: 16 values per thread and as many sums for the weight gradients.
template <typename F> cudaError_t with_width_bwd(int H, F f) {
    if (H <= 256) return f(Geom<1, 1>());
    if (H <= 512) return f(Geom<1, 2>());
    if (H <= 1024) return f(Geom<2, 2>());
    if (H <= 2048) return f(Geom<4, 2>());
    if (H <= 4096) return f(Geom<8, 2>());
    if (H <= 8192) return f(Geom<16, 2>());
    return f(Geom<32, 2>());
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, int h_dtype, int y_dtype, cudaStream_t st) {
    return with_types(h_dtype, y_dtype, [&](auto th, auto ty) {
        auto launch = [&](auto w) {
            using W = decltype(w);
            using C = NormCfg<W::G, W::V>;
            return launch_pdl(block_norm_kernel<decltype(th), decltype(ty), W::G, W::V>,
                              dim3((a.T + C::kRows - 1) / C::kRows), dim3(C::kThreads), 0, st, a);
        };
        return many_rows(a.T, a.H) ? with_width(a.H, launch) : with_width_few(a.H, launch);
    });
}

constexpr int kBwdSmem = 220 * 1024;   // dynamic shared memory of the backward pass; the static arrays have 7 KB beside it

int norm_bwd_ctas(int T) { return T < kNormBwdCtas ? T : kNormBwdCtas; }

cudaError_t launch_block_norm_bwd(const NormBwdArgs& a, int h_dtype, int y_dtype, cudaStream_t st) {
    const int ctas = norm_bwd_ctas(a.T);
    cudaError_t e = with_types(h_dtype, y_dtype, [&](auto th, auto ty) {
        return with_width_bwd(a.H, [&](auto w) {
            using W = decltype(w);
            const int nh = a.H * (int)sizeof(th), ny = a.H * (int)sizeof(ty);
            BwdRing ring{0, nh, nh + ny, 2 * nh + ny, 2 * (nh + ny), 0};
            const int room = kBwdSmem - 8 * a.H;   // for the rings, beside the weights
            int groups = BwdCfg<W::G>::kMaxGroups;
            auto kernel = block_norm_bwd_kernel<decltype(th), decltype(ty), W::G, W::V, false>;
            constexpr int kSums = W::G == 32 ? (int)sizeof(float) * 2 * W::V * 8 * BwdCfg<W::G>::kMaxThreads : 0;
            size_t smem = W::G == 32 ? kSums : sizeof(float) * a.H;
            if constexpr (W::G < 32) {
                if (room / ring.stage_bytes >= 2) {
                    // two stages for as many groups as fit, then more stages
                    groups = room / (2 * ring.stage_bytes) < groups ? room / (2 * ring.stage_bytes) : groups;
                    const int stages = room / (groups * ring.stage_bytes);
                    ring.stages = stages < kNormBwdStages ? stages : kNormBwdStages;
                    ring.w_off = groups * ring.stages * ring.stage_bytes;
                    smem = (size_t)ring.w_off + 8 * (size_t)a.H;
                    kernel = block_norm_bwd_kernel<decltype(th), decltype(ty), W::G, W::V, true>;
                }
            }
            // The most that any width of this kernel takes, not this call's size: the attribute belongs to the kernel, and
            // another thread's call of another width may set it between this and the launch.
            const cudaError_t er = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                        W::G == 32 ? kSums : kBwdSmem);
            if (er != cudaSuccess) return er;
            return launch_pdl(kernel, dim3(ctas), dim3(groups * W::G * 32), smem, st, a, ring);
        });
    });
    if (e == cudaSuccess && (a.dw_pre || a.dw_post))
        e = launch_pdl(norm_reduce_kernel, dim3((a.H + 31) / 32, a.dw_post ? 2 : 1), dim3(32, 32), 0, st,
                       (const float*)a.part, ctas, a.H, a.dw_pre, a.dw_post);
    return e;
}

cudaError_t norm_take_status(uint32_t* host, cudaStream_t st) { return take_status(host, st); }

}  // namespace moe
