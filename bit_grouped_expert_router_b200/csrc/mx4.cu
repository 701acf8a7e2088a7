// mx4.cu -- microscaled 4-bit floating point (MXFP4): rows quantised, read back, and multiplied by
// each expert's matrix on the tensor cores in that form.
//
// Blocks of 32 values along a row share a scale 2^(s - 127); each value is a 4-bit E2M1 number times
// it.  The product's operands go to the tensor core as they are stored: kind::mxf4 multiplies the
// 4-bit values and applies both scales per 32 columns, accumulating in fp32.
#include <type_traits>

#include "ops_common.cuh"

namespace moe {

namespace {

// ---- quantisation ---------------------------------------------------------------------------------
// Two neighbouring threads share a block of 32 values, sixteen each: their largest magnitude by one
// exchange, eight bytes of codes per thread.  Codes and scales of consecutive blocks lie next to each other, so rows
// matter only where they are halved (SwiGLU) or sent elsewhere (pos: a token is read and quantised once
// and written to all of its places).  Bound by those bytes: 131072 x 512 bf16 in 25.7 us.

// Two values as E2M1 codes (round to nearest, ties to even, magnitudes above 6 to 6), the first in the
// low four bits; eight of them as a word.
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint32_t e2m1_pack(const float (&v)[8]) {
    return e2m1_pair(v[0], v[1]) | (e2m1_pair(v[2], v[3]) << 8) | (e2m1_pair(v[4], v[5]) << 16) |
           (e2m1_pair(v[6], v[7]) << 24);
}

// Largest magnitude as fp32 bits.  Magnitudes order like their bits in every type, infinities and NaN
// above all finite ones; 16-bit values are compared two at a time.
__device__ __forceinline__ uint32_t top_bits(const Vec<float, 8> (&x)[2]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 q = x[i >> 1].w[i & 1];
        m = max(max(m, max(q.x & 0x7FFFFFFFu, q.y & 0x7FFFFFFFu)), max(q.z & 0x7FFFFFFFu, q.w & 0x7FFFFFFFu));
    }
    return m;
}
template <typename T> __device__ __forceinline__ uint32_t top_bits(const Vec<T, 8> (&x)[2]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 q = x[i].w[0];
        m = __vmaxu2(__vmaxu2(m, __vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu)),
                     __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu));
    }
    float lo, hi;
    Elem<T>::unpack(max(m >> 16, m & 0xFFFFu), lo, hi);
    return __float_as_uint(lo);
}

// 1 / x to one unit in the last place, for x in [1, 2^126]: neither it nor the quotient is subnormal there, so the
// instruction that flushes those gives what the one that keeps them gives, in fewer steps (32768 x 512 outputs of
// SwiGLU: 15.5 us; with that one, and the largest magnitude taken in integers, 19.0 us).
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// silu(g) u = g u / (1 + exp(-g)).  Below kSiluTail (exp(64) < 2^93 lies inside the reciprocal's range) 1 + exp(-g) is
// exp(-g) to fp32's last bit, and the quotient alone would end at -87 though a large u can bring the product back into
// range: there it is g exp(g / 2) u exp(g / 2), whose factors are ordinary numbers down to -174.
constexpr float kSiluTail = -64.f;
template <bool TAIL> __device__ __forceinline__ float silu_times(float g, float u) {
    if (TAIL && g < kSiluTail) {
        const float h = expf(0.5f * g);
        return g * h * u * h;
    }
    return g * reciprocal(1.f + expf(-g)) * u;
}
// Whether a value is below kSiluTail (a negative NaN may pass for one), by its bits: those of negative numbers
// order by magnitude, above all positive ones.
__device__ __forceinline__ bool below_tail(const Vec<float, 8> (&x)[2]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 q = x[i >> 1].w[i & 1];
        m = max(max(m, max(q.x, q.y)), max(q.z, q.w));
    }
    return m > 0xC2800000u;
}
template <typename T> __device__ __forceinline__ bool below_tail(const Vec<T, 8> (&x)[2]) {
    constexpr uint32_t kTail = std::is_same_v<T, __half> ? 0xD400u : 0xC280u;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 q = x[i].w[0];
        m = __vmaxu2(__vmaxu2(m, __vmaxu2(q.x, q.y)), __vmaxu2(q.z, q.w));
    }
    return max(m >> 16, m & 0xFFFFu) > kTail;
}
// max(a, |b|), NaN if either is.
__device__ __forceinline__ float max_magnitude(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

// Items per thread: two, so that enough loads are in flight, but one where the places add loads and most bytes are
// written (4096 and 16384 tokens of 2048 to 8 rows each: 10.7 and 35.9 us with one item, 11.8 and 39.7 with two;
// 131072 x 512 in order: 26.0 and 25.7 us).
__host__ __device__ constexpr int quant_items(bool pos) { return pos ? 1 : 2; }

// The loaded items quantised and stored.
template <typename T, bool SWIGLU, bool POS, bool TAIL>
__device__ __forceinline__ void quantize_items(const Mx4QuantArgs& a, uint32_t items, uint32_t i0,
                                               const Vec<T, 8> (&x)[quant_items(POS)][2],
                                               const Vec<T, 8> (&up)[SWIGLU ? quant_items(POS) : 1][2],
                                               const uint32_t (&tok)[quant_items(POS)],
                                               const uint32_t (&col)[quant_items(POS)]) {
    constexpr int kQuantItems = quant_items(POS);
    const uint32_t n = (uint32_t)a.K / 16;
#pragma unroll
    for (int u = 0; u < kQuantItems; ++u) {   // every thread takes part in the exchanges
        const uint32_t i = i0 + u * 256u;
        const bool on = i < items;
        float v[2][8];
        uint32_t top = 0;
        if (on) {
            if constexpr (SWIGLU) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float g[8], p[8], most = 0.f;
                    x[u][h].get(g);
                    up[u][h].get(p);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        v[h][q] = silu_times<TAIL>(g[q], p[q]);
                        most = max_magnitude(most, v[h][q]);
                    }
                    top = max(top, __float_as_uint(most));
                }
            } else {
                top = top_bits(x[u]);
                x[u][0].get(v[0]);
                x[u][1].get(v[1]);
            }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        if (!on) continue;
        // s - 127 = exponent of the largest magnitude - 2, at least -127; 2^(127 - s) is exact
        const bool bad = top >= 0x7F800000u;
        const int s = bad ? 255 : max((int)(top >> 23) - 2, 0);
        uint2 w = make_uint2(0u, 0u);
        if (!bad) {
            const float scale = __uint_as_float((uint32_t)(254 - s) << 23);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                v[0][q] *= scale;
                v[1][q] *= scale;
            }
            w = make_uint2(e2m1_pack(v[0]), e2m1_pack(v[1]));
        }
        const bool first = (i & 1u) == 0;
        if constexpr (!POS) {
            reinterpret_cast<uint2*>(a.codes)[i] = w;
            if (first) a.scales[i / 2] = (uint8_t)s;
        } else {
            for (int j0 = 0; j0 < a.k; j0 += 8) {
                int p[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    p[c] = j0 + c < a.k ? a.pos[(size_t)tok[u] * a.k + j0 + c] : -1;
                    if (p[c] >= a.n_rows) {
                        set_status(g_ops_status, MOE_STATUS_BOUNDS);
                        p[c] = -1;
                    }
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (p[c] < 0) continue;
                    reinterpret_cast<uint2*>(a.codes)[(size_t)p[c] * n + col[u]] = w;
                    if (first) a.scales[(size_t)p[c] * (n / 2) + col[u] / 2] = (uint8_t)s;
                }
            }
        }
    }
}

template <typename T, bool SWIGLU, bool POS>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(Mx4QuantArgs a, uint32_t items) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kQuantItems = quant_items(POS);
    const uint32_t n = (uint32_t)a.K / 16;   // items of sixteen values per row: even, like all counts here
    const uint32_t i0 = blockIdx.x * (256u * kQuantItems) + threadIdx.x;
    Vec<T, 8> x[kQuantItems][2], up[SWIGLU ? kQuantItems : 1][2];
    uint32_t tok[kQuantItems], col[kQuantItems];
#pragma unroll
    for (int u = 0; u < kQuantItems; ++u) {
        const uint32_t i = i0 + u * 256u;
        if (i >= items) continue;
        tok[u] = SWIGLU || POS ? i / n : 0;
        col[u] = SWIGLU || POS ? i - tok[u] * n : 0;
        const T* at = static_cast<const T*>(a.x) +
                      (SWIGLU ? (size_t)tok[u] * 2 * a.K + (size_t)col[u] * 16 : (size_t)i * 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            x[u][h].load(at + 8 * h);
            if constexpr (SWIGLU) up[u][h].load(at + a.K + 8 * h);
        }
    }
    if constexpr (SWIGLU) {   // gates in silu's tail, rare, have a copy of the rest to themselves: a branch around each
                              // activation, or the sum of exponentials that needs none, cost 1.7 to 2.4 of 15.5 us
        bool tail = false;
#pragma unroll
        for (int u = 0; u < kQuantItems; ++u) tail |= i0 + u * 256u < items && below_tail(x[u]);
        if (__any_sync(0xffffffffu, tail)) return quantize_items<T, SWIGLU, POS, true>(a, items, i0, x, up, tok, col);
    }
    quantize_items<T, SWIGLU, POS, false>(a, items, i0, x, up, tok, col);
}

// ---- values ---------------------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, size_t pieces,
                                                             T* __restrict__ out) {
    griddep_wait();
    griddep_launch_dependents();
    for (size_t i = blockIdx.x * (size_t)256 + threadIdx.x; i < pieces; i += (size_t)gridDim.x * 256) {
        const uint32_t w = codes[i];
        const uint32_t s = scales[i / 4];
        // 2^(s - 127): a subnormal for s = 0, NaN for s = 255
        const float scale = __uint_as_float(s == 255u ? 0x7FFFFFFFu : s ? s << 23 : 0x00400000u);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // E2M1 bits as the top of an fp32: sign, then exponent and mantissa in places 24..22 of a
            // number scaled by 2^-126; the product by 2^126 is exact for the subnormal codes too
            const uint32_t c = w >> (4 * j);
            const float m = __uint_as_float(((c & 8u) << 28) | ((c & 7u) << 22)) * 0x1p126f;
            v[j] = m * scale;
        }
        Vec<T, 8> o;
        o.set(v);
        o.store(out + i * 8);
    }
}

// ---- grouped product ------------------------------------------------------------------------------
// Work unit = 128 output features x up to 224 rows of one expert.  The weights are the M = 128
// operand and the rows the N operand, so a short segment costs a narrow instruction (N = 16 and up)
// instead of a padded one.  A persistent CTA walks units; per step of 256 columns
//   warp 0       TMA: the 128 x 128-byte weight tile and the row tile (boxes of 32 rows), 128-byte swizzle
//   warps 8-11   the scales: a thread loads those of its rows 32 bytes at a time (four steps), ahead of their use,
//                and writes them in the order tcgen05.cp wants (512 bytes per 128 rows and 128 columns:
//                row r at 16 (r % 32) + 4 (r / 32)), to a ring of their own
//   warp 1       tcgen05.cp of the scales to tensor memory, then four MMAs of 64 columns
//   warps 4-7, 12-15  epilogue of the unit before: tensor memory -> shared memory -> row stores
// Tensor memory: two accumulators of 224 columns (the epilogue of one overlaps the MMAs of the next) and
// 2 x 32 columns of scales, alternating by step.
//
// What bounds it: the weights from HBM while the rows are few (1024 rows over 256 experts of 1024 x 2048: 47.7 us of
// 43.0), then the traffic from L2 (weights once per row tile, rows once per feature tile: 699 MB of it in the 73 us of
// 32768 x 1024 x 2048 over 256 experts), and, run after run, the power cap (1.65 GHz and 87 us there).  Short rows and
// many results (32768 x 2048 x 512: 62 us of 43.6, in fp32 104 of 64.1) leave DRAM and L2 about half busy; what holds
// them is not known.  Pairs of CTAs on one tile of 256 features (cta_group::2), which read the rows half as often,
// gained 3 to 5% from 131072 rows on and lost 1 to 30% below: their barriers and commits cross CTAs every step.
constexpr int kTM = 128;             // features per unit
constexpr int kStep = 256;           // columns per step: 128 bytes of codes per row
constexpr int kSfSteps = 4;          // steps whose scales come together: a 32-byte sector of every row
constexpr int kSfRing = 2;
constexpr int kSfBytes = 2 * (512 + 2 * 512);   // per step: 512 B of weight scales, 2 x 512 B of row scales, twice
constexpr int kThreadsMm = 512;
constexpr int kTmemSf = 448;         // first tensor-memory column of the scales
constexpr int kOutPitch = kTM * 2 + 16, kOutBytes = 32 * kOutPitch;   // a bf16 chunk of the epilogue

// TN: most rows per unit.  224 where experts have many rows; with 64 the ring has seven stages instead of four,
// and more of the weights are in flight where they are all there is to load (see launch_mx4_matmul).
template <int TN> struct MmCfg {
    static constexpr int kRing = TN > 64 ? 4 : 7;
    static constexpr int kABytes = kTM * 128, kBBytes = TN * 128, kStageBytes = kABytes + kBBytes;
    static constexpr int kSfAt = kRing * kStageBytes, kOutAt = kSfAt + kSfRing * kSfSteps * kSfBytes;
    static constexpr int kSmem = 1024 + kOutAt + 2 * kOutBytes;
    static_assert(kStageBytes % 1024 == 0, "stages keep the swizzle's alignment");
    static_assert(2 * TN <= kTmemSf, "two accumulators in front of the scales");
};

struct Unit {
    int e, mt, row0, rows;   // expert, feature tile, first row, rows (1..TN)
};

// The units of a persistent CTA, first + n stride of the list: experts in order, row tiles within an expert (its
// 16-row groups dealt evenly over them), feature tiles within a row tile.  A warp walks them together: its
// lanes look up 32 units at a time, one each, and hand them round (a search and three divisions for every
// unit, in every warp, cost 0.3 us of the 2.3 us between units of two steps).
template <int TN> struct UnitWalk {
    const int *ustart, *seg, *len;   // first unit of an expert, its first row, its rows
    const Unit* first;               // the CTA's first unit, found while the list was made
    int E, MT, total, stride, u;
    int n = 0;
    Unit mine = {0, 0, 0, 0};

    __device__ bool more() const { return u < total; }
    __device__ Unit next() {
        const int k = n == 0 ? 0 : (n - 1) & 31;
        if (n == 0) {
            mine = *first;
        } else if (k == 0) {
            const uint32_t v = (uint32_t)u + lane_id() * (uint32_t)stride;
            if (v < (uint32_t)total) mine = find((int)v);
        }
        ++n;
        u += stride;
        Unit r;   // (exchanged, so that the compiler may keep it in uniform registers)
        r.e = __shfl_sync(0xffffffffu, mine.e, k);
        r.mt = __shfl_sync(0xffffffffu, mine.mt, k);
        r.row0 = __shfl_sync(0xffffffffu, mine.row0, k);
        r.rows = __shfl_sync(0xffffffffu, mine.rows, k);
        return r;
    }

    // Unit w of expert e, which has `rows` rows from `row` on.
    static __device__ Unit unit_of(int e, int w, int row, int rows, int MT) {
        const int groups = (rows + 15) / 16, tiles = (rows + TN - 1) / TN, tile = w / MT;
        const int each = groups / tiles, left = groups - each * tiles;   // the first `left` tiles have one group more
        const int g0 = each * tile + min(tile, left), g1 = g0 + each + (tile < left ? 1 : 0);
        Unit r;
        r.e = e;
        r.mt = w - tile * MT;
        r.row0 = row + 16 * g0;
        r.rows = min(rows, 16 * g1) - 16 * g0;
        return r;
    }

private:
    __device__ Unit find(int v) const {
        int lo = 0, hi = E;   // ustart[lo] <= v < ustart[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (ustart[mid] <= v) lo = mid;
            else hi = mid;
        }
        return unit_of(lo, v - ustart[lo], seg[lo], len[lo], MT);
    }
};

// The asynchronous instructions below are issued by one lane (`lead`) of a warp that runs their code
// as a whole: under a branch on the lane the compiler moves every operand from vector to uniform
// registers first, which cost about 100 cycles an MMA (measured: 4 MMAs of N = 128 in 453 cycles, 254
// this way; the tensor core itself needs 256).
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// 32 rows x 16 bytes of shared memory to 4 tensor-memory columns, repeated in all four lane quarters.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
        "l"(desc), "r"(lead)
        : "memory");
}
// Descriptor of a 512-byte scale block: no swizzle, 8-row groups of 16-byte rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem_addr) {
    return (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | ((uint64_t)(128u >> 4) << 16) | ((uint64_t)(128u >> 4) << 32) |
           ((uint64_t)1u << 46);
}
// D (+)= A B with block scales: E2M1 operands, one E8M0 scale per 32 columns, 64 columns.
__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t accumulate, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 e, %7, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit_lead(uint64_t* bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}
__device__ __forceinline__ void expect_lead(uint64_t* bar, uint32_t bytes, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
        "r"(bytes), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void tma_lead(uint32_t smem_dst, const CUtensorMap* map, int x, int y, uint64_t* bar,
                                         uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];\n\t}" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)), "r"(lead)
        : "memory");
}
// Instruction descriptor of kind::mxf4: bits 4-5 scale bytes of B (0: bytes 0-1, 2: bytes 2-3 of the
// scale word), 7-9 and 10-11 operand types (1 = E2M1), 17-22 N / 8, 23 scale type (1 = E8M0),
// 24-28 M / 16, 29-30 scale bytes of A.
__device__ __forceinline__ uint32_t idesc_mx4(int n, uint32_t sf) {
    return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(kTM >> 4) << 24) |
           (sf << 29);
}

// 32 scale bytes of one row (1024 columns) from byte b on, zeros behind the row's end (nk = K / 32
// bytes): 16-byte loads where rows keep that alignment, narrower ones where not.
__device__ __forceinline__ void load_scales(uint32_t (&v)[8], const uint8_t* row, int b, int nk, int align) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0u;
    if (align == 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (b + 16 * i < nk) {
                const uint4 q = *reinterpret_cast<const uint4*>(row + b + 16 * i);
                v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
            }
    } else if (align == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (b + 4 * i < nk) v[i] = *reinterpret_cast<const uint32_t*>(row + b + 4 * i);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (b + i < nk) v[i / 4] |= (uint32_t)row[b + i] << (8 * (i & 3));
    }
}

template <typename T, int TN>
__global__ void __launch_bounds__(kThreadsMm, 1) mx4_matmul_kernel(Mx4MatmulArgs a, const __grid_constant__ CUtensorMap tm_w,
                                                                   const __grid_constant__ CUtensorMap tm_x) {
    using C = MmCfg<TN>;
    constexpr int kRing = C::kRing;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kRing], empty[kRing], sffull[kSfRing], sfempty[kSfRing], dfull[2], dempty[2], drain;
    __shared__ int ustart[257], seg[256], len[256], wsum[8];
    __shared__ Unit first_unit;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    uint8_t* ring = smem_raw + (1024u - (smem_u32(smem_raw) & 1023u) & 1023u);
    uint8_t* out = ring + C::kOutAt;
    volatile int* abort_flag = &abort_word;
    uint32_t* status = g_ops_status;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = lane_id();

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kSfRing; ++i) {
            mbar_init(&sffull[i], 4);    // the scale warps
            mbar_init(&sfempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], 8);
        }
        mbar_init(&drain, 1);
        abort_word = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_w);
        prefetch_tmap(&tm_x);
    }
    if (warp == 2) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    griddep_wait();
    griddep_launch_dependents();
    // the unit list: row tiles per expert, first unit of each.  Expert e's segment runs from the largest of
    // offsets[0..e] to the largest of offsets[0..e+1], held to [0, R]: the offsets themselves if they are sound,
    // and disjoint segments whatever they are.
    const int MT = (a.N + kTM - 1) / kTM;
    int mine = 0, inc = 0, low = 0, high = 0, o0 = 0, o1 = 0;
    if (tid < 256) {
        if (tid < a.E) {
            o0 = a.offsets[tid];
            o1 = a.offsets[tid + 1];
        }
        low = min(max(o0, 0), a.R);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, low, off);
            if (lane >= off) low = max(low, o);
        }
        if (lane == 31) wsum[warp] = low;
    }
    __syncthreads();
    if (tid < 256) {
        for (int w = 0; w < warp; ++w) low = max(low, wsum[w]);
        if (tid < a.E) {
            high = max(low, min(o1, a.R));
            if (blockIdx.x == 0 && (low != o0 || high != o1)) set_status(status, MOE_STATUS_BOUNDS);
            seg[tid] = low;
            len[tid] = high - low;
            mine = (high - low + TN - 1) / TN * MT;
        }
        inc = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += o;
        }
    }
    __syncthreads();   // (wsum is read)
    if (tid < 256 && lane == 31) wsum[warp] = inc;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid < 256) {
        for (int w = 0; w < warp; ++w) inc += wsum[w];
        if (tid < a.E) ustart[tid] = inc - mine;
        if (tid == a.E - 1) ustart[a.E] = inc;
        if (inc - mine <= (int)blockIdx.x && (int)blockIdx.x < inc)
            first_unit = UnitWalk<TN>::unit_of(tid, blockIdx.x - (inc - mine), low, high - low, MT);
    }
    __syncthreads();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);   // (uniform, to the compiler too)
    UnitWalk<TN> walk{ustart, seg, len, &first_unit, a.E, MT, ustart[a.E], (int)gridDim.x, (int)blockIdx.x};
    const int KS = (a.K + kStep - 1) / kStep;

    if (warp == 0) {
        // ------------------------------------------------------------------ TMA producer
        const uint32_t lead = elect_lane();
        uint32_t it = 0;
        while (walk.more()) {
            const Unit un = walk.next();
            const int boxes = (un.rows + kMx4BoxRows - 1) / kMx4BoxRows, wrow = un.e * a.N + un.mt * kTM;
            for (int ks = 0; ks < KS; ++ks, ++it) {
                const int s = it % kRing;
                const bool ok = mbar_wait(&empty[s], ((it / kRing) & 1u) ^ 1u, abort_flag, status);
                if (!__all_sync(0xffffffffu, ok)) goto producer_done;
                const uint32_t st = smem_u32(ring) + s * C::kStageBytes;
                expect_lead(&full[s], C::kABytes + boxes * kMx4BoxRows * 128, lead);
                tma_lead(st, &tm_w, ks * 128, wrow, &full[s], lead);
                for (int b = 0; b < boxes; ++b)
                    tma_lead(st + C::kABytes + b * kMx4BoxRows * 128, &tm_x, ks * 128, un.row0 + b * kMx4BoxRows, &full[s], lead);
            }
        }
    producer_done:
        // every copy issued must land before the CTA may exit
        for (uint32_t i = it > (uint32_t)kRing ? it - kRing : 0u; i < it; ++i)
            mbar_drain(&full[i % kRing], (i / kRing) & 1u);
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issuer
        const uint32_t lead = elect_lane();
        uint32_t it = 0, sfi = 0, tl = 0;
        bool issued = false;
        for (; walk.more(); ++tl) {
            const Unit un = walk.next();
            const int n = (un.rows + 15) / 16 * 16;
            const uint32_t ab = tl & 1u;
            bool ok = mbar_wait(&dempty[ab], ((tl >> 1) & 1u) ^ 1u, abort_flag, status);
            if (!__all_sync(0xffffffffu, ok)) goto mma_done;
            tc_fence_after();
            const uint32_t d = tmem + ab * TN;
            const uint32_t i0 = idesc_mx4(n, 0), i2 = idesc_mx4(n, 2);
            for (int ks = 0; ks < KS; ++ks, ++it) {
                const int s = it % kRing, j = ks % kSfSteps, c4 = sfi % kSfRing;
                if (j == 0) {
                    ok = mbar_wait(&sffull[c4], (sfi / kSfRing) & 1u, abort_flag, status);
                    if (!__all_sync(0xffffffffu, ok)) goto mma_done;
                }
                ok = mbar_wait(&full[s], (it / kRing) & 1u, abort_flag, status);
                if (!__all_sync(0xffffffffu, ok)) goto mma_done;
                tc_fence_after();
                const uint32_t st = smem_u32(ring) + s * C::kStageBytes;
                const uint32_t sf = smem_u32(ring) + C::kSfAt + (c4 * kSfSteps + j) * kSfBytes;
                const uint32_t tsf = tmem + kTmemSf + (it & 1u) * 32;
                const int kmma = min(4, (a.K - ks * kStep + 63) / 64);
                for (int c = 0; c < (kmma + 1) / 2; ++c) {
                    tmem_cp_scales(tsf + c * 4, scale_desc(sf + c * 512), lead);
                    tmem_cp_scales(tsf + 8 + c * 8, scale_desc(sf + 1024 + c * 1024), lead);
                    if (TN > 128 && n > 128) tmem_cp_scales(tsf + 12 + c * 8, scale_desc(sf + 1024 + c * 1024 + 512), lead);
                }
                const uint64_t ad = sdesc_sw128(st), bd = sdesc_sw128(st + C::kABytes);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    if (kk < kmma)
                        mma_mx4(d, ad + 2 * kk, bd + 2 * kk, (kk & 1) ? i2 : i0, tsf + (kk >> 1) * 4,
                                tsf + 8 + (kk >> 1) * 8, (ks | kk) != 0 ? 1u : 0u, lead);
                issued = true;
                commit_lead(&empty[s], lead);
                if (j == kSfSteps - 1 || ks == KS - 1) {
                    commit_lead(&sfempty[c4], lead);
                    ++sfi;
                }
            }
            commit_lead(&dfull[ab], lead);
        }
    mma_done:
        if (*abort_flag && issued) {
            commit_lead(&drain, lead);
            mbar_drain(&drain, 0);
        }
    } else if (warp >= 8 && warp < 12) {
        // ------------------------------------------------------------------ scales
        // Thread r has weight row r and token rows r and r + 128 of the unit.  It loads a row's scales
        // a sector (1024 columns, four steps) at a time, the next sector before it hands out this one.
        const int r = tid - 256, nk = a.K / 32;
        const int align = nk % 16 == 0 ? 16 : nk % 4 == 0 ? 4 : 1;
        uint32_t nxt[3][8] = {};
        int ks0 = 0;
        Unit un = {0, 0, 0, 0};
        auto fetch = [&]() {
            const int f = un.mt * kTM + r;
            load_scales(nxt[0], a.w_scales + ((size_t)un.e * a.N + f) * nk, ks0 * 8, f < a.N ? nk : 0, align);
#pragma unroll
            for (int i = 0; i < (TN > 128 ? 2 : 1); ++i) {
                const int row = r + 128 * i;
                load_scales(nxt[1 + i], a.scales + (size_t)(un.row0 + row) * nk, ks0 * 8, row < un.rows ? nk : 0, align);
            }
        };
        const uint32_t at = (uint32_t)((r & 31) * 16 + (r >> 5) * 4);
        uint32_t sfi = 0;
        int steps = 0;   // of the sector at hand (none yet)
        bool more = walk.more();
        if (more) un = walk.next();
        while (more || steps > 0) {
            uint32_t cur[3][8];
            const int now = steps;
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) cur[i][j] = nxt[i][j];
            steps = 0;
            if (more) {
                fetch();
                steps = min(kSfSteps, KS - ks0);
                ks0 += kSfSteps;
                if (ks0 >= KS) {
                    ks0 = 0;
                    more = walk.more();
                    if (more) un = walk.next();
                }
            }
            if (now == 0) continue;
            const int c = sfi % kSfRing;
            const bool ok = mbar_wait(&sfempty[c], ((sfi / kSfRing) & 1u) ^ 1u, abort_flag, status);
            if (!__all_sync(0xffffffffu, ok)) goto scales_done;
            uint8_t* sf = ring + C::kSfAt + c * kSfSteps * kSfBytes + at;
#pragma unroll
            for (int j = 0; j < kSfSteps; ++j) {
                if (j >= now) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    *reinterpret_cast<uint32_t*>(sf + j * kSfBytes + h * 512) = cur[0][2 * j + h];
                    *reinterpret_cast<uint32_t*>(sf + j * kSfBytes + 1024 + h * 1024) = cur[1][2 * j + h];
                    if (TN > 128) *reinterpret_cast<uint32_t*>(sf + j * kSfBytes + 1536 + h * 1024) = cur[2][2 * j + h];
                }
            }
            fence_proxy_async_smem();   // generic-proxy stores -> visible to tcgen05.cp
            __syncwarp();
            if (lane == 0) mbar_arrive(&sffull[c]);
            ++sfi;
        }
    scales_done:;
    } else if (warp >= 4) {
        // ------------------------------------------------------------------ epilogue
        // Two groups of four warps take the unit's chunks of 32 rows in turn.  A thread holds one feature
        // of the chunk's rows.  In bf16, the lanes of a pair swap halves so that each has two
        // neighbouring features of every other row, and the chunk goes through shared memory to
        // stores of whole 256-byte row pieces; the pair's two rows are 4 apart and the pitch is 272
        // bytes, so a warp's 4-byte stores fall into different banks.  (The pair's values stored
        // directly, 64 bytes a row: 162 us for 32768 x 2048 outputs of 512 columns, 108 us this way.)
        const int q = warp & 3, grp = warp >= 12 ? 1 : 0, gt = tid & 127;
        uint32_t tl = 0;
        for (; walk.more(); ++tl) {
            const Unit un = walk.next();
            const uint32_t ab = tl & 1u;
            const bool ok = mbar_wait(&dfull[ab], (tl >> 1) & 1u, abort_flag, status);
            if (named_bar_or(1 + grp, 128, !ok)) break;   // the group leaves together
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + ab * TN;
            const int f0 = un.mt * kTM, f = f0 + 32 * q + lane;
            T* y = static_cast<T*>(a.y) + (size_t)un.row0 * a.N;
            for (int c0 = 32 * grp; c0 < un.rows; c0 += 64) {
                uint32_t v[32];
                tmem_ld32(taddr + c0, v);
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int r = 0; r < 32; ++r)
                        if (c0 + r < un.rows && f < a.N) y[(size_t)(c0 + r) * a.N + f] = __uint_as_float(v[r]);
                } else {
                    const bool odd = lane & 1;
                    uint8_t* st = out + grp * kOutBytes;
                    uint8_t* at = st + (odd ? 4 * kOutPitch : 0) + (32 * q + (lane & ~1)) * 2;
#pragma unroll
                    for (int r8 = 0; r8 < 32; r8 += 8)
#pragma unroll
                        for (int r = r8; r < r8 + 4; ++r) {   // even lane: row r, odd lane: row r + 4
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[r] : v[r + 4], 1);
                            const float lo = __uint_as_float(odd ? got : v[r]), hi = __uint_as_float(odd ? v[r + 4] : got);
                            *reinterpret_cast<__nv_bfloat162*>(at + r * kOutPitch) = __floats2bfloat162_rn(lo, hi);
                        }
                    named_bar(3 + grp, 128);
                    uint4 o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[i] = *reinterpret_cast<const uint4*>(st + (i * 8 + (gt >> 4)) * kOutPitch + (gt & 15) * 16);
                    named_bar(3 + grp, 128);   // read: the next chunk may have the buffer
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = c0 + i * 8 + (gt >> 4), c = (gt & 15) * 8;
                        if (r < un.rows && f0 + c < a.N) *reinterpret_cast<uint4*>(y + (size_t)r * a.N + f0 + c) = o[i];
                    }
                }
            }
            tc_fence_before();   // the accumulator is read: the MMAs of the unit after the next may have it
            __syncwarp();
            if (lane == 0) mbar_arrive(&dempty[ab]);
        }
    }

    __syncthreads();
    if (warp == 2) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4QuantArgs& a, int dtype, cudaStream_t st) {
    const uint32_t items = (uint32_t)((size_t)a.T * (a.K / 16)), per = 256 * quant_items(a.pos);
    const dim3 grid((items + per - 1) / per);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        auto kernel = a.swiglu ? (a.pos ? mx4_quantize_kernel<T, true, true> : mx4_quantize_kernel<T, true, false>)
                               : (a.pos ? mx4_quantize_kernel<T, false, true> : mx4_quantize_kernel<T, false, false>);
        return launch_pdl(kernel, grid, dim3(256), 0, st, a, items);
    });
}

cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, long long rows, int K, void* out,
                                  int dtype, int num_sms, cudaStream_t st) {
    const size_t pieces = (size_t)rows * (K / 8), want = (pieces + 255) / 256, most = (size_t)num_sms * 32;
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return launch_pdl(mx4_dequantize_kernel<T>, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st,
                          reinterpret_cast<const uint32_t*>(codes), scales, pieces, static_cast<T*>(out));
    });
}

template <typename T, int TN>
static cudaError_t launch_matmul(const Mx4MatmulArgs& a, const CUtensorMap& tm_w, const CUtensorMap& tm_x, int num_sms,
                                 cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(mx4_matmul_kernel<T, TN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               MmCfg<TN>::kSmem);
    if (e != cudaSuccess) return e;
    // at most one row tile per TN rows and one more per expert that has rows
    const long long tiles = (long long)a.R / TN + (a.E < a.R ? a.E : a.R);
    const long long units = tiles * ((a.N + kTM - 1) / kTM);
    return launch_pdl(mx4_matmul_kernel<T, TN>, dim3((unsigned)(units < num_sms ? units : num_sms)), dim3(kThreadsMm),
                      MmCfg<TN>::kSmem, st, a, tm_w, tm_x);
}

cudaError_t launch_mx4_matmul(const Mx4MatmulArgs& a, const CUtensorMap& tm_w, const CUtensorMap& tm_x, int dtype,
                              int num_sms, cudaStream_t st) {
    // Row tiles of 64 up to 32 rows per expert on average.  256 experts of 1024 x 2048, tiles of 64 / of 224, in us:
    // 1 row each 46.7 / 49.6, 8 rows 48.6 / 51.1, 32 rows 51.7 / 53.0 (in uneven segments 58.0 / 55.9), 64 rows
    // 56.8 / 56.6 (71.8 / 61.3), 96 rows 84.5 / 61.1.
    const bool few = a.R <= 32ll * a.E;
    if (dtype == MOE_DTYPE_BF16)
        return few ? launch_matmul<__nv_bfloat16, 64>(a, tm_w, tm_x, num_sms, st)
                   : launch_matmul<__nv_bfloat16, 224>(a, tm_w, tm_x, num_sms, st);
    if (dtype == MOE_DTYPE_FP32)
        return few ? launch_matmul<float, 64>(a, tm_w, tm_x, num_sms, st)
                   : launch_matmul<float, 224>(a, tm_w, tm_x, num_sms, st);
    return cudaErrorInvalidValue;
}

cudaError_t mx4_take_status(uint32_t* host, cudaStream_t st) { return take_status(host, st); }

}  // namespace moe
