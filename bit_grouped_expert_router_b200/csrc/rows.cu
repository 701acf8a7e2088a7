// rows.cu -- (token, slot) pairs sorted by expert, token rows copied into that order and expert rows
// summed back, with the gradients of both.
//
//   dispatch          pos = place of pair (t, j) in the stable order by expert; rows[pos[t,j]] = x[t]
//   its gradient      dx[t] = sum_j drows[pos[t,j]]                       (combine with weights 1)
//   combine           out[t] = base[t] + sum_j gates[t,j] rows[pos[t,j]]
//   its gradient      drows[pos[t,j]] = gates[t,j] dout[t];  dgates[t,j] = <dout[t], rows[pos[t,j]]>
//
// All four move k rows of H values per token and compute next to nothing: they are bound by those
// bytes, so every row is read once and written once, 16 bytes per thread, and nothing is summed
// with atomics (results do not change from run to run).
#include "ops_common.cuh"

namespace moe {

namespace {

__device__ __forceinline__ int sort_key(int e, int E) {   // the pair's expert, -1 for none
    if (e >= E) {
        set_status(g_ops_status, MOE_STATUS_BOUNDS);
        return -1;
    }
    return e < 0 ? -1 : e;
}

__device__ __forceinline__ int warp_scan(int v) {   // inclusive
    const int lane = lane_id();
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    return v;
}

// off[e] = sum of tot[0..e), off[E] = all, over the block's first 256 threads (E <= 256).
__device__ __forceinline__ void scan_experts(const int* tot, int* off, int* wsum, int E) {
    const int tid = threadIdx.x, warp = tid >> 5;
    int v = 0, inc = 0;
    if (warp < 8) {
        v = tid < E ? tot[tid] : 0;
        inc = warp_scan(v);
        if (lane_id() == 31) wsum[warp] = inc;
    }
    __syncthreads();
    if (warp < 8) {
        for (int w = 0; w < warp; ++w) inc += wsum[w];
        if (tid < E) off[tid] = inc - v;
        if (tid == E - 1) off[E] = inc;
    }
    __syncthreads();
}

// Ranks up to blockDim.x pairs (one per thread, expert e or -1) in thread order behind nxt[e], the
// next free place of each expert, and moves nxt on.  wcnt: [warps][E].  Returns the pair's place.
__device__ __forceinline__ int rank_pairs(int e, int* nxt, int* wcnt, int E, int nwarps) {
    const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
    for (int i = tid; i < nwarps * E; i += blockDim.x) wcnt[i] = 0;
    __syncthreads();
    const unsigned same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && lane == __ffs(same) - 1) wcnt[warp * E + e] = __popc(same);
    __syncthreads();
    for (int i = tid; i < E; i += blockDim.x) {
        int run = nxt[i];
        for (int w0 = 0; w0 < nwarps; w0 += 8) {   // eight loads before their stores
            int v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = w0 + u < nwarps ? wcnt[(w0 + u) * E + i] : 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (w0 + u < nwarps) wcnt[(w0 + u) * E + i] = run;
                run += v[u];
            }
        }
        nxt[i] = run;
    }
    __syncthreads();
    return e >= 0 ? wcnt[warp * E + e] + __popc(same & ((1u << lane) - 1u)) : -1;
}

// Few pairs: every CTA counts all of them, ranks its own (whole tokens, at most 256 pairs) and
// copies their rows: one launch, bound by its latency (one token of 8 x 2048 bf16: 3.4 us).
__global__ void __launch_bounds__(256) dispatch_small_kernel(SortArgs a, int tokens_per_cta) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ int tot[256], before[256], off[257], wsum[8], wcnt[8 * 256], place[256];
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * tokens_per_cta, nt = min(tokens_per_cta, a.T - t0);
    const int lo = t0 * a.k, mine = nt * a.k;
    tot[tid] = 0;
    before[tid] = 0;
    __syncthreads();
    for (int i0 = tid; i0 < a.n; i0 += 8 * 256) {   // eight loads in flight
        int e[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) e[u] = i0 + 256 * u < a.n ? a.idx[i0 + 256 * u] : -1;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            e[u] = sort_key(e[u], a.E);
            if (e[u] < 0) continue;
            atomicAdd(&tot[e[u]], 1);
            if (i0 + 256 * u < lo) atomicAdd(&before[e[u]], 1);
        }
    }
    __syncthreads();
    scan_experts(tot, off, wsum, a.E);
    if (tid < a.E) before[tid] += off[tid];
    __syncthreads();
    const int e = tid < mine ? sort_key(a.idx[lo + tid], a.E) : -1;
    const int p = rank_pairs(e, before, wcnt, a.E, 8);
    const int kept = off[a.E];
    if (tid < mine) {
        place[tid] = p;
        a.pos[lo + tid] = p;
        if (p >= 0) a.perm[p] = lo + tid;
        if (lo + tid >= kept) a.perm[lo + tid] = -1;
    }
    if (blockIdx.x == 0)
        for (int i = tid; i <= a.E; i += 256) a.offsets[i] = off[i];
    if (!a.rows) return;
    __syncthreads();
    for (int i = tid; i < nt * a.nvec; i += 256) {
        const int t = i / a.nvec, c = i - t * a.nvec;
        const uint4 v = a.x[(size_t)(t0 + t) * a.nvec + c];
        for (int j = 0; j < a.k; ++j) {
            const int q = place[t * a.k + j];
            if (q >= 0) a.rows[(size_t)q * a.nvec + c] = v;
        }
    }
}

// hist[b][e] = pairs of expert e in chunk b.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ int cnt[256];
    const int tid = threadIdx.x;
    if (tid < a.E) cnt[tid] = 0;
    __syncthreads();
    const int lo = blockIdx.x * a.chunk_tokens * a.k, hi = min(a.n, lo + a.chunk_tokens * a.k);
    for (int i = lo + tid; i < hi; i += kSortThreads) {
        const int e = sort_key(a.idx[i], a.E);
        if (e >= 0) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    if (tid < a.E) a.hist[(size_t)blockIdx.x * a.E + tid] = cnt[tid];
}

// One CTA per chunk (of whole tokens): the experts' totals and the pairs of earlier chunks from the counts
// of all chunks, then the chunk's places in pair order, up to kSortThreads pairs at a time.
__global__ void __launch_bounds__(kSortThreads) sort_rank_kernel(SortArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ int part[4][256], partb[4][256], off[257], wsum[8];
    __shared__ int wcnt[(kSortThreads / 32) * 256];
    const int tid = threadIdx.x, b = blockIdx.x;
    {
        const int e = tid & 255, quarter = tid >> 8;
        const int b_lo = quarter * a.nchunk / 4, b_hi = (quarter + 1) * a.nchunk / 4;
        int sum = 0, before = 0;
        if (e < a.E) {
            constexpr int U = 20;   // loads in flight
            for (int b0 = b_lo; b0 < b_hi; b0 += U) {
                int v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) v[u] = b0 + u < b_hi ? a.hist[(size_t)(b0 + u) * a.E + e] : 0;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (b0 + u < b) before += v[u];
                    sum += v[u];
                }
            }
        }
        part[quarter][e] = sum;
        partb[quarter][e] = before;
    }
    __syncthreads();
    if (tid < 256) {
        part[0][tid] += part[1][tid] + part[2][tid] + part[3][tid];
        partb[0][tid] += partb[1][tid] + partb[2][tid] + partb[3][tid];
    }
    __syncthreads();
    scan_experts(part[0], off, wsum, a.E);
    int* nxt = partb[0];
    if (tid < a.E) nxt[tid] += off[tid];
    const int kept = off[a.E];
    if (b == 0)
        for (int i = tid; i <= a.E; i += kSortThreads) a.offsets[i] = off[i];
    const int t0 = b * a.chunk_tokens, t1 = min(a.T, t0 + a.chunk_tokens), round = kSortThreads / a.k;
    for (int t = t0; t < t1; t += round) {
        __syncthreads();   // nxt is ready, wcnt is free
        const int nt = min(round, t1 - t), pairs = nt * a.k, lo = t * a.k;
        const int e = tid < pairs ? sort_key(a.idx[lo + tid], a.E) : -1;
        const int p = rank_pairs(e, nxt, wcnt, a.E, (pairs + 31) / 32);
        if (tid < pairs) {
            a.pos[lo + tid] = p;
            if (p >= 0) a.perm[p] = lo + tid;
            if (lo + tid >= kept) a.perm[lo + tid] = -1;
        }
    }
}

// Threads of the row kernels: a row of n pieces gets min(n, 256) threads of a 256-thread block, so
// a block serves 256 / n rows, or one row in passes of 256 pieces.
struct RowSplit {
    int t, c, step;   // the thread's row (-1: none), its first piece, the distance to its next
    __device__ RowSplit(int n, int T) {
        const int per = min(n, 256), rows = 256 / per, r = threadIdx.x / per;
        const long long row = (long long)blockIdx.x * rows + r;
        t = r < rows && row < T ? (int)row : -1;
        c = threadIdx.x - r * per;
        step = per;
    }
    static dim3 grid(int n, int T) {
        const int rows = 256 / (n < 256 ? n : 256);
        return dim3((T + rows - 1) / rows);
    }
};

// A block's threads hold a token's row, a piece each, and store it k times.  Blocks run in token order, so
// the rows written at a time lie close together in each expert's segment (16384 tokens of 8 x 2048 bf16:
// 97 us, 6.2 TB/s; each SM on a range of tokens of its own, in the kernel that ranks them: 111 us with
// these stores, 108 us with bulk copies through shared memory).
__global__ void __launch_bounds__(256) dispatch_copy_kernel(const uint4* __restrict__ x, const int* __restrict__ pos,
                                                            int T, int k, int nvec, uint4* __restrict__ rows) {
    griddep_wait();
    griddep_launch_dependents();
    const RowSplit s(nvec, T);
    if (s.t < 0) return;
    for (int c = s.c; c < nvec; c += s.step) {
        const uint4 v = x[(size_t)s.t * nvec + c];
        for (int j0 = 0; j0 < k; j0 += 8) {
            int p[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) p[u] = j0 + u < k ? pos[(size_t)s.t * k + j0 + u] : -1;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (p[u] >= 0) rows[(size_t)p[u] * nvec + c] = v;
        }
    }
}

// A thread sums one 16-byte piece of a token's k rows in fp32, in slot order, four loads in flight and
// five blocks per SM to hide the chain from place to row (4099 tokens of 8 x 2048 bf16: 27.5 us,
// 5.5 TB/s; eight loads and the 3 blocks their registers leave: 39.4 us; four and 6: spills, 40.7 us).
constexpr int kSumRows = 4;
template <typename T>
__global__ void __launch_bounds__(256, 5) combine_kernel(CombineArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int N = 16 / (int)sizeof(T);
    const int n = a.H / N;
    const RowSplit s(n, a.T);
    if (s.t < 0) return;
    const T* rows = static_cast<const T*>(a.rows);
    for (int c = s.c; c < n; c += s.step) {
        float acc[N];
        Vec<T, N> v;
        if (a.base) {
            v.load(static_cast<const T*>(a.base) + (size_t)s.t * a.H + c * N);
            v.get(acc);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = 0.f;
        }
        for (int j0 = 0; j0 < a.k; j0 += kSumRows) {
            int p[kSumRows];
            float g[kSumRows];
            Vec<T, N> r[kSumRows];
#pragma unroll
            for (int u = 0; u < kSumRows; ++u) {
                const size_t at = (size_t)s.t * a.k + j0 + u;
                p[u] = j0 + u < a.k ? a.pos[at] : -1;
                g[u] = a.gates && p[u] >= 0 ? a.gates[at] : 1.f;
                if (p[u] >= a.n_rows) {
                    set_status(g_ops_status, MOE_STATUS_BOUNDS);
                    p[u] = -1;
                }
            }
#pragma unroll
            for (int u = 0; u < kSumRows; ++u)
                if (p[u] >= 0) r[u].load(rows + (size_t)p[u] * a.H + c * N);
#pragma unroll
            for (int u = 0; u < kSumRows; ++u) {
                if (p[u] < 0) continue;
                float f[N];
                r[u].get(f);
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = fmaf(g[u], f[i], acc[i]);
            }
        }
        v.set(acc);
        v.store(static_cast<T*>(a.out) + (size_t)s.t * a.H + c * N);
    }
}

// One warp per pair: the pair's row is read once for the gate's gradient and its gradient written.
// The k warps of a token sit next to each other, so dout[t] comes from HBM once and from the first
// cache level after that (4096 tokens of 8 x 2048 bf16: 46.6 us, 6.1 TB/s).
template <typename T>
__global__ void __launch_bounds__(256) combine_bwd_kernel(CombineBwdArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int N = 16 / (int)sizeof(T), U = 4;
    const long long pair = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (pair >= (long long)a.T * a.k) return;
    const int lane = lane_id();
    int p = a.pos[pair];
    if (p >= a.n_rows) {
        if (lane == 0) set_status(g_ops_status, MOE_STATUS_BOUNDS);
        p = -1;
    }
    if (p < 0) {
        if (lane == 0) a.dgates[pair] = 0.f;
        return;
    }
    const float g = a.gates[pair];
    const T* d = static_cast<const T*>(a.dout) + (size_t)(pair / a.k) * a.H;
    const T* r = static_cast<const T*>(a.rows) + (size_t)p * a.H;
    T* o = static_cast<T*>(a.drows) + (size_t)p * a.H;
    float dot = 0.f;
    for (int h0 = lane * N; h0 < a.H; h0 += 32 * N * U) {
        Vec<T, N> dv[U], rv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + 32 * N * u;
            if (h < a.H) {
                rv[u].load(r + h);
                dv[u].load(d + h);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + 32 * N * u;
            if (h >= a.H) break;
            float df[N], rf[N];
            dv[u].get(df);
            rv[u].get(rf);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                dot = fmaf(df[i], rf[i], dot);
                df[i] *= g;
            }
            dv[u].set(df);
            dv[u].store(o + h);
        }
    }
    dot = warp_sum(dot);
    if (lane == 0) a.dgates[pair] = dot;
}

}  // namespace

cudaError_t launch_dispatch(const SortArgs& a, int num_sms, cudaStream_t st) {
    if (a.n <= kSmallPairs) {
        // as many CTAs as SMs where there are tokens for them, whole tokens each (k <= 32, so at
        // most 256 pairs)
        int tokens = (a.T + num_sms - 1) / num_sms;
        tokens = tokens * a.k > 256 ? 256 / a.k : tokens;
        return launch_pdl(dispatch_small_kernel, dim3((a.T + tokens - 1) / tokens), dim3(256), 0, st, a, tokens);
    }
    cudaError_t e = launch_pdl(sort_count_kernel, dim3(a.nchunk), dim3(kSortThreads), 0, st, a);
    if (e == cudaSuccess) e = launch_pdl(sort_rank_kernel, dim3(a.nchunk), dim3(kSortThreads), 0, st, a);
    if (e == cudaSuccess && a.rows)
        e = launch_pdl(dispatch_copy_kernel, RowSplit::grid(a.nvec, a.T), dim3(256), 0, st, a.x, (const int*)a.pos, a.T,
                       a.k, a.nvec, a.rows);
    return e;
}

cudaError_t launch_combine(const CombineArgs& a, int dtype, cudaStream_t st) {
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return launch_pdl(combine_kernel<T>, RowSplit::grid(a.H * (int)sizeof(T) / 16, a.T), dim3(256), 0, st, a);
    });
}

cudaError_t launch_combine_bwd(const CombineBwdArgs& a, int dtype, cudaStream_t st) {
    const long long pairs = (long long)a.T * a.k;
    return with_dtype(dtype, [&](auto t) {
        return launch_pdl(combine_bwd_kernel<decltype(t)>, dim3((unsigned)((pairs + 7) / 8)), dim3(256), 0, st, a);
    });
}

cudaError_t rows_take_status(uint32_t* host, cudaStream_t st) { return take_status(host, st); }

}  // namespace moe
