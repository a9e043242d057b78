// 4-bit products for few rows (a decode step): the weight as a stream.
//
// The step is bound by reading the codes once (0.5 bytes a weight and 2 per
// group), and next to that by turning them into operands. The weight is the A
// operand of warp-level m16n8k16 MMAs, 16 weight rows (or, for the SwiGLU pair,
// 8 rows of Wg over the same 8 of Wu) against up to 8 activation rows as B, so one set of
// expanded codes serves every row and no MMA is padded along the weight.
//
// A lane of a quad loads words of 8 consecutive codes straight into registers:
// for a group of 32 V codes (V = 1, 2, 4), V words at k = t * 8 V of the group
// (t: lane of the quad), so every MMA's 16 k lie in one group, the codes are
// exact integers in the operand (code - zero), and the group's scale multiplies
// the fp32 sums of the group: no rounding of the weight at all. In a word, code i
// is paired with code i + 4 (a mask and an OR put both into the mantissas of
// 128 or 1024, one subtraction leaves the integers); the activation rows are
// stored in shared memory in the same order, one 16-byte vector per word.
//
// Measured in graphs: 1 x 4096 x 4096 4.9 us, 1 x 11008 x 4096 8.5 us (2.7 TB/s), SwiGLU FFN
// 4096 x 11008 of 3 rows 24.3 us (2.9 TB/s). A CTA's start (rows of x to shared
// memory, their norm, the first codes: 2.3 us at 1 x 1024 x 1024) is what keeps one
// product of a decode step from the rate of its stream. Loads land in L1 lines, so
// shared memory taken for more than the rows costs loads in flight: with the
// largest carve-out the FFN took 32 us.
//
// Loads run in blocks of 16 (V = 1: 8) words of each of the lane's two weight rows,
// double-buffered across units (16 or 8 + 8 weight rows); a CTA's 8 warps take
// 8 slices of K and add their sums through shared memory in warp order.
//
// x * gamma is rounded to the dtype, the one rounding before the output's (in fp16 times
// a power of two where a row's products leave the type's range: lift_rows). For up
// to four rows half of the MMA's columns would be idle, and take what that rounding
// cuts off, if both copies of the rows leave room for a second CTA (kSmemPair: four rows up to
// K = 6592, one up to 26560): there is no rounding to speak of then (FFN of 3 rows
// 23.8 -> 24.3 us, 3 x 4096 x 4096 5.3 -> 5.6).
//
// More than eight rows are slabs of at most eight, side by side in the grid:
// they walk the weight at the same pace, so that it is read from HBM once and
// by the other slabs from L2. w4_few_rows says up to where that beats the
// tensor-core tile kernel, which expands each code once for all rows.
#include "fl_common.cuh"
#include "fl_host.h"
#include "fl_quant.cuh"
#include "fl_w4.h"

namespace fl {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
// words of one weight row in a register block (groups of 32 also hold four times the scales)
__host__ __device__ constexpr int block_words(int V) { return V == 1 ? 8 : 16; }
constexpr uint32_t kLeast16 = 0x2800u;  // 2^-5 in fp16 (lift_rows)
constexpr int kSmemMax = 200 * 1024;
constexpr int kSmemPair = 104 * 1024;  // two CTAs to an SM

// Row stride of the activation rows in 16-byte vectors: 4 mod 8, so that the
// 8 lanes of a quarter warp (two rows, four vectors each) hit different banks.
__host__ __device__ __forceinline__ int row_vecs(int K) { return (K / 8 + 7) / 8 * 8 + 4; }
// (64 bits: K may be any int)
__host__ __device__ __forceinline__ long long smem_bytes(int M, int K) { return (long long)M * row_vecs(K) * 16; }

template <int DT>
struct Mma;
template <>
struct Mma<DT_F16> {
    static constexpr uint32_t kMagic = 0x64006400u;  // 1024
    static __device__ __forceinline__ void run(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    // c = a b
    static __device__ __forceinline__ void first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    }
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
};
template <>
struct Mma<DT_BF16> {
    static constexpr uint32_t kMagic = 0x43004300u;  // 128
    static __device__ __forceinline__ void run(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    // c = a b
    static __device__ __forceinline__ void first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    }
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
};

// Codes of one weight row, V words, not kept in L1.
template <int V>
__device__ __forceinline__ void load_words(uint32_t (&w)[V], const uint8_t* p) {
    if constexpr (V == 4)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
            : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    else if constexpr (V == 2)
        asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    else
        asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
}

// One register block of the stream: U groups of the lane's two weight rows, and
// the scales and zero points of groups t, t + 4, .. of them (lane t of the quad).
template <int V>
struct Block {
    static constexpr int U = block_words(V) / V, S = U / 4;
    uint32_t w[2][U][V];
    uint16_t s[2][S];
    uint8_t z[2][S];
};

// The weight rows of a lane in unit u, first and second half of the MMA's 16.
struct Rows {
    const uint8_t* q[2];
    const uint16_t* s[2];
    const uint8_t* z[2];
};

template <bool DUAL>
__device__ __forceinline__ Rows rows_of(const W4Params& p, int u, int g, int groups) {
    Rows r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = DUAL ? h : 0;
        // (rows past N, in the last unit when N is 8 mod 16, repeat row N - 1)
        const size_t n = DUAL ? (size_t)u * 8 + g : (size_t)min(u * 16 + h * 8 + g, p.N - 1);
        r.q[h] = p.q[j] + n * (p.K / 2);
        r.s[h] = p.scales[j] + n * groups;
        r.z[h] = p.zeros[j] == nullptr ? nullptr : p.zeros[j] + n * groups;
    }
    return r;
}

// Issues the loads of groups c0 .. c0 + U - 1 (below c1).
template <int V, bool Z>
__device__ __forceinline__ void load_block(Block<V>& B, const Rows& r, int c0, int c1, int t) {
#pragma unroll
    for (int i = 0; i < Block<V>::U; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (c0 + i < c1) {
                load_words<V>(B.w[h][i], r.q[h] + ((size_t)(c0 + i) * 4 + t) * (4 * V));
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) B.w[h][i][j] = 0u;
            }
        }
#pragma unroll
    for (int i = 0; i < Block<V>::S; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = c0 + 4 * i + t;
            B.s[h][i] = c < c1 ? __ldg(r.s[h] + c) : (uint16_t)0;
            if (Z) B.z[h][i] = c < c1 ? __ldg(r.z[h] + c) : (uint8_t)0;
        }
}

// acc += the block's groups times the activation rows (xrow: this lane's row of
// them, offset to the quad's lane).
template <int DT, int V, bool Z>
__device__ __forceinline__ void mma_block(const Block<V>& B, const uint4* xrow, int c0, int c1, int t, float (&acc)[4]) {
    using O = Mma<DT>;
#pragma unroll
    for (int i = 0; i < Block<V>::U; ++i) {
        if (c0 + i >= c1) break;  // (warp-uniform)
        // the group's scale and zero point of both rows, from lane i % 4 of the quad
        const uint32_t mine = (uint32_t)B.s[0][i / 4] | ((uint32_t)B.s[1][i / 4] << 16);
        const uint32_t both = __shfl_sync(0xffffffffu, mine, i & 3, 4);
        uint32_t z0 = O::kMagic + 0x00080008u, z1 = z0;
        if (Z) {
            const uint32_t zm = (uint32_t)B.z[0][i / 4] | ((uint32_t)B.z[1][i / 4] << 8);
            const uint32_t zb = __shfl_sync(0xffffffffu, zm, i & 3, 4);
            z0 = O::kMagic + (zb & 15u) * 0x10001u, z1 = O::kMagic + ((zb >> 8) & 15u) * 0x10001u;
        }
        float c[4];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint4 x = xrow[((c0 + i) * V + j) * 4];
            const uint32_t w0 = B.w[0][i][j], w1 = B.w[1][i][j];
            uint32_t e[2][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                e[0][k] = O::sub(and_or(w0 >> (4 * k), 0x000f000fu, O::kMagic), z0);
                e[1][k] = O::sub(and_or(w1 >> (4 * k), 0x000f000fu, O::kMagic), z1);
            }
            const uint32_t a0[4] = {e[0][0], e[1][0], e[0][1], e[1][1]}, a1[4] = {e[0][2], e[1][2], e[0][3], e[1][3]};
            if (j == 0) O::first(c, a0, x.x, x.y);
            else O::run(c, a0, x.x, x.y);
            O::run(c, a1, x.z, x.w);
        }
        const float2 s = DTypeOps<DT>::unpack(both);
        acc[0] = fmaf(s.x, c[0], acc[0]);
        acc[1] = fmaf(s.x, c[1], acc[1]);
        acc[2] = fmaf(s.y, c[2], acc[2]);
        acc[3] = fmaf(s.y, c[3], acc[3]);
    }
}

// A 16-byte vector of 8 activations as (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ uint4 pair_up(const uint4& v) {
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                      __byte_perm(v.y, v.w, 0x7632));
}

// x * g - p of packed pairs, p being x * g rounded: the difference fits the dtype to
// its own precision.
template <int DT>
__device__ __forceinline__ uint32_t rest(uint32_t x, uint32_t g, uint32_t p) {
    const float2 a = DTypeOps<DT>::unpack(x), b = DTypeOps<DT>::unpack(g), c = DTypeOps<DT>::unpack(p);
    return DTypeOps<DT>::pack(fmaf(a.x, b.x, -c.x), fmaf(a.y, b.y, -c.y));
}

// The activation rows in shared memory: x, or x * gamma rounded once (and what
// that leaves in rows of their own behind, p.halves) with the
// RMS row scale in rscale. Vector v of a row (8 k) goes to the place where the
// quad reads it: group v / 4V, word v % V of lane v / V % 4. R: a bound on M.
// Returns (fp16) whether a warp saw products outside the type's range: lift_rows then looks at every row.
template <int DT, bool NORM, int R, int V, typename Pre>
__device__ bool build_rows(const W4Params& p, const uint16_t* x, int M, uint4* xs, float* rscale, Pre pre) {
    using Ops = DTypeOps<DT>;
    const int vecs = p.K / 8, ld = row_vecs(p.K);
    constexpr bool kRange = NORM && DT == DT_F16;
    __shared__ float part[kWarps][R];
    float sq[R];
    [[maybe_unused]] uint32_t big[R];  // the row's largest |x * gamma|, in pairs
#pragma unroll
    for (int m = 0; m < R; ++m) sq[m] = 0.f, big[m] = 0u;
    bool first = true;
    constexpr int C = R <= 4 ? 2 : 1;  // vectors of a row in flight per thread
    for (int c0 = threadIdx.x; c0 < vecs || first; c0 += C * kThreads) {
        uint4 v[C][R], gv[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = c0 + j * kThreads;
            if (c < vecs) {
                if (NORM) gv[j] = ldg_v4(p.gamma + (size_t)c * 8);
#pragma unroll
                for (int m = 0; m < R; ++m)
                    if (m < M) v[j][m] = ldg_v4(x + (size_t)m * p.K + (size_t)c * 8);
            }
        }
        if (first) pre();
        first = false;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = c0 + j * kThreads;
            if (c >= vecs) continue;
            const int to = c / (4 * V) * (4 * V) + c % V * 4 + c / V % 4;
#pragma unroll
            for (int m = 0; m < R; ++m) {
                if (m >= M) continue;
                uint4 o = v[j][m];
                if (NORM) {
                    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = Ops::unpack(w[e]);
                        sq[m] = fmaf(f.x, f.x, fmaf(f.y, f.y, sq[m]));
                    }
                    const uint4 g = gv[j], x1 = o;
                    o = make_uint4(Ops::mul2(o.x, g.x), Ops::mul2(o.y, g.y), Ops::mul2(o.z, g.z), Ops::mul2(o.w, g.w));
                    if constexpr (kRange) big[m] = absmax2<DT>(big[m], absmax8<DT>(o));
                    if (R <= 4 && p.halves)
                        xs[(M + m) * ld + to] = pair_up(make_uint4(rest<DT>(x1.x, g.x, o.x), rest<DT>(x1.y, g.y, o.y),
                                                                   rest<DT>(x1.z, g.z, o.z), rest<DT>(x1.w, g.w, o.w)));
                }
                xs[m * ld + to] = pair_up(o);
            }
        }
    }
    int again = 0;
    if (NORM) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if constexpr (kRange) {
            // of each row: whether a product is 2^-5 or more, and whether x is not all zeros; whether a product is infinite
            uint32_t s = 0u, top = 0u;
#pragma unroll
            for (int m = 0; m < R; ++m) {
                const uint32_t b = absmax_halves<DT>(big[m]);
                s |= (b >= kLeast16 ? 1u << m : 0u) | (sq[m] > 0.f ? 0x100u << m : 0u);
                top = max(top, b);
            }
            if (top >= Bits16<DT>::kInf) s |= 0x10000u;
            s = __reduce_or_sync(0xffffffffu, s);
            again = ((s >> 8) & ~s & 0xffu) != 0u || s >= 0x10000u;
        }
#pragma unroll
        for (int m = 0; m < R; ++m) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sq[m] += __shfl_xor_sync(0xffffffffu, sq[m], o);
            if (lane == 0) part[warp][m] = sq[m];
        }
        if constexpr (kRange) again = __syncthreads_or(again);
        else __syncthreads();
        if (threadIdx.x < R) {
            float a = 0.f;
            for (int w = 0; w < kWarps; ++w) a += part[w][threadIdx.x];
            rscale[threadIdx.x] = rsqrtf(a / (float)p.K + p.eps);
        }
    }
    __syncthreads();
    return again != 0;
}

// fp16 rows whose products x * gamma leave the type's range: above 65504, or all
// below 2^-5, where its smallest values would cost them bits (2^-25 of error next to
// a largest product of 2^-5 is 2^-20 of it, far below a rounding's 2^-12). The
// norm makes the answer the same size whatever the row's, so they are formed
// again times the power of two that puts the largest one into 2^13 .. 2^14, and
// rscale takes its inverse: exact, and other rows keep their bits. Seldom needed, so
// x is read again and nothing here is unrolled. Finding such rows costs every fp16
// call 0.04 to 0.2 us (1 x 4096 x 4096 4.77 -> 4.83, 4 rows 5.79 -> 6.00, 8 rows 6.23 -> 6.26).
template <int DT, int V>
__device__ void lift_rows(const W4Params& p, const uint16_t* x, int M, uint4* xs, float* rscale) {
    using Ops = DTypeOps<DT>;
    const int vecs = p.K / 8, ld = row_vecs(p.K);
    __shared__ float most[kWarps];
#pragma unroll 1
    for (int m = 0; m < M; ++m) {
        const uint16_t* row = x + (size_t)m * p.K;
        float a = 0.f;
#pragma unroll 1
        for (int i = threadIdx.x; i < vecs * 4; i += kThreads) {
            const float2 f = Ops::unpack(__ldg(reinterpret_cast<const uint32_t*>(row) + i));
            const float2 g = Ops::unpack(__ldg(reinterpret_cast<const uint32_t*>(p.gamma) + i));
            a = fmaxf(a, fmaxf(fabsf(f.x * g.x), fabsf(f.y * g.y)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = a;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) a = fmaxf(a, most[w]);
        // (a product of two fp16 values is 0, or 2^-48 to 2^32, or not finite: then the row is as it is.
        // From 65520 on it would round to infinity.)
        const int e = (int)(__float_as_uint(a) >> 23) - 127;
        if (a > 0.f && e < 128 && (a < 0x1p-5f || a >= 65520.f)) {
            const float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
#pragma unroll 1
            for (int c = threadIdx.x; c < vecs; c += kThreads) {
                const uint4 v = ldg_v4(row + (size_t)c * 8), g = ldg_v4(p.gamma + (size_t)c * 8);
                const uint32_t vw[4] = {v.x, v.y, v.z, v.w}, gw[4] = {g.x, g.y, g.z, g.w};
                uint32_t o[4], r[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = Ops::unpack(vw[j]), h = Ops::unpack(gw[j]);
                    const float2 t = make_float2(f.x * h.x * up, f.y * h.y * up);
                    o[j] = Ops::pack(t.x, t.y);
                    const float2 q = Ops::unpack(o[j]);
                    r[j] = Ops::pack(t.x - q.x, t.y - q.y);
                }
                const int to = c / (4 * V) * (4 * V) + c % V * 4 + c / V % 4;
                xs[m * ld + to] = pair_up(make_uint4(o[0], o[1], o[2], o[3]));
                if (p.halves) xs[(M + m) * ld + to] = pair_up(make_uint4(r[0], r[1], r[2], r[3]));
            }
            if (threadIdx.x == 0) rscale[m] *= __uint_as_float((uint32_t)(127 - 13 + e) << 23);
        }
        __syncthreads();  // (`most` is the next row's, and the rows are read next)
    }
}

template <int DT, bool DUAL, int V, bool Z>
__global__ void __launch_bounds__(kThreads, 2) fl_w4_rows_kernel(const __grid_constant__ W4Params p) {
    using Ops = DTypeOps<DT>;
    extern __shared__ __align__(16) uint8_t smem[];
    uint4* xs = reinterpret_cast<uint4*>(smem);
    __shared__ float rscale[8];
    __shared__ float4 red[2][kWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // this slab's rows
    const int m0 = blockIdx.y * p.slab, M = min(p.slab, p.M - m0);
    const uint16_t* x = p.x + (size_t)m0 * p.K;
    const int groups = p.K / (32 * V), units = DUAL ? p.N / 8 : (p.N + 15) / 16;
    const int per = (groups + kWarps - 1) / kWarps, s0 = min(groups, warp * per), s1 = min(groups, s0 + per);
    constexpr int U = Block<V>::U;
    const int blocks = (per + U - 1) / U;  // (the same for every warp: the block loop holds barriers)
    Rows rows = rows_of<DUAL>(p, blockIdx.x, g, groups);
    // L2 prefetch of the rows of x (each line by one CTA of the grid) and of this
    // warp's first codes: L2 is the point of coherence, so a prefetch before the
    // dependency wait cannot bring in stale data
    {
        const int xl = (M * p.K * 2 + 127) / 128;
        for (int i = (int)(threadIdx.x * gridDim.x + blockIdx.x); i < xl; i += kThreads * gridDim.x)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(x) + (size_t)i * 128));
        // 128-byte lines of the slice: 256 codes each
        for (int c = s0 * 16 * V + t * 128; c < s1 * 16 * V && c < s0 * 16 * V + 512; c += 512) {
            asm volatile("prefetch.global.L2 [%0];" ::"l"(rows.q[0] + c));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(rows.q[1] + c));
        }
    }
    griddep_wait();
    Block<V> A, B;
    auto pre = [&] { load_block<V, Z>(A, rows, s0, s1, t); };
    if (p.gamma != nullptr) {
        bool again;
        if (M <= 2) again = build_rows<DT, true, 2, V>(p, x, M, xs, rscale, pre);
        else if (M <= 4) again = build_rows<DT, true, 4, V>(p, x, M, xs, rscale, pre);
        else again = build_rows<DT, true, 8, V>(p, x, M, xs, rscale, pre);
        if (DT == DT_F16 && again) lift_rows<DT, V>(p, x, M, xs, rscale);  // (the same for every thread)
    } else {
        if (threadIdx.x < 8) rscale[threadIdx.x] = 1.f;
        if (M <= 4) build_rows<DT, false, 4, V>(p, x, M, xs, rscale, pre);
        else build_rows<DT, false, 8, V>(p, x, M, xs, rscale, pre);
    }
    griddep_launch_dependents();
    // columns 0 to 3, and 4 to 7 with p.halves: a row and what its rounding left
    // (a column past the last row is not used: any row will do)
    const int row = p.halves && g >= 4 ? (g - 4 < M ? M + g - 4 : 0) : g < M ? g : 0;
    const uint4* xrow = xs + row * row_vecs(p.K) + t;

    int q = 0, buf = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, buf ^= 1) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int b = 0; b < blocks; ++b, ++q) {
            const bool last = b == blocks - 1, more = !last || u + (int)gridDim.x < units;
            const int nb = last ? 0 : b + 1;
            if (last && more) rows = rows_of<DUAL>(p, u + gridDim.x, g, groups);
            if ((q & 1) == 0) {
                if (more) load_block<V, Z>(B, rows, s0 + nb * U, s1, t);
                mma_block<DT, V, Z>(A, xrow, s0 + b * U, s1, t, acc);
            } else {
                if (more) load_block<V, Z>(A, rows, s0 + nb * U, s1, t);
                mma_block<DT, V, Z>(B, xrow, s0 + b * U, s1, t, acc);
            }
        }
        red[buf][warp][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        __syncthreads();
        // One thread per output: lane (g, t) of the sums holds weight rows g and
        // g + 8 (gate and up) and activation rows 2 t and 2 t + 1.
        if (threadIdx.x < (DUAL ? 8 : 16) * M) {
            const int m = threadIdx.x / (DUAL ? 8 : 16), r = threadIdx.x % (DUAL ? 8 : 16);
            const float* src = &red[buf][0][(r & 7) * 4 + (m >> 1)].x + (m & 1) + (r >> 3) * 2;
            const float rs = rscale[m];
            float y = src[0], up = DUAL ? src[2] : 0.f;
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                y += src[w * 128];
                if (DUAL) up += src[w * 128 + 2];
            }
            if (p.halves) {  // (columns 4 on: two lanes further)
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    y += src[w * 128 + 8];
                    if (DUAL) up += src[w * 128 + 10];
                }
            }
            const int n = DUAL ? u * 8 + r : u * 16 + r;
            const size_t at = (size_t)(m0 + m) * p.N + n;
            if constexpr (DUAL) {
                p.out[at] = (uint16_t)(Ops::pack(w4_act(ACT_SILU, y * rs) * (up * rs), 0.f) & 0xffffu);
            } else if (n < p.N) {
                y *= rs;
                if (p.bias != nullptr) y += Ops::unpack(p.bias[n]).x;
                y = w4_act(p.act, y);
                if (p.residual != nullptr) y += Ops::unpack(p.residual[at]).x;
                p.out[at] = (uint16_t)(Ops::pack(y, 0.f) & 0xffffu);
            }
        }
        // (red is double-buffered: the next unit writes the other half, and the
        // one after that only follows the next __syncthreads)
    }
}

int slabs_of(int M) { return (M + 7) / 8; }
int slab_rows(int M) { return (M + slabs_of(M) - 1) / slabs_of(M); }

template <int DT, bool DUAL, int V, bool Z>
cudaError_t launch_rows(const W4Params& p, const host::LaunchContext& ctx, cudaStream_t stream) {
    auto kern = fl_w4_rows_kernel<DT, DUAL, V, Z>;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t attr = host::allow_smem(kern, kSmemMax, ctx.device, done);
    if (attr != cudaSuccess) return attr;
    const int slabs = slabs_of(p.M), smem = (int)smem_bytes(p.halves ? 2 * p.slab : p.slab, p.K), units = DUAL ? p.N / 8 : (p.N + 15) / 16;
    int most = ctx.sms * (smem <= kSmemPair ? 2 : 1) / slabs;  // resident CTAs of a slab
    if (most < 1) most = 1;
    return host::launch(kern, dim3((unsigned)(units < most ? units : most), (unsigned)slabs), kThreads, (size_t)smem, ctx.pdl,
                        stream, p);
}

// The choice between this kernel and the tile kernel, by rows and weights,
// measured side by side in graphs (us, this kernel / the tile kernel; with gamma but for
// the 4096 x 11008):
//   1024 x 1024: 64 rows 4.3 / 8.2, 128 rows 6.3 / 8.2
//   2048 x 2048: 64 rows 8.3 / 9.7; 4096 x 1024: 64 rows 9.3 / 8.7, 96 rows 13.3 / 9.3
//   4096 x 4096: 24 rows 10.5 / 15.6, 32 rows 12.5 / 15.6, 64 rows 18.7 / 16.4; without gamma
//   32 rows 11.8 / 10.8
//   11008 x 4096: 32 rows 24.5 / 33.4; 4096 x 11008: 16 rows 17.7 / 18.7, 24 rows 23.6 / 19.1,
//   32 rows 26.8 / 19.1
//   FFN 4096 x 11008: 16 rows 45 / 62, 24 rows 60 / 63, 32 rows 72 / 63, 64 rows 132 / 64
//   (with its gate and up product here and the other there: 70 with 24 rows, so
//   that long rows, for which 24 is late, keep to the limit of large weights)
int rows_limit(long long weights, int K) {
    return weights <= (1ll << 20) ? 128 : weights <= (4ll << 20) ? 64 : weights <= (64ll << 20) && K <= 8192 ? 32 : 24;
}

}  // namespace

bool w4_few_rows(int M, int N, int K, bool dual) {
    return M <= rows_limit((long long)N * K * (dual ? 2 : 1), K) && smem_bytes(slab_rows(M), K) <= kSmemMax;
}
bool w4_always_few(int M, int K) { return M <= 24 && smem_bytes(slab_rows(M), K) <= kSmemMax; }

fl_status w4_rows(int dt, bool dual, const W4Params& params, const host::LaunchContext& ctx, cudaStream_t stream) {
    W4Params p = params;
    p.slab = slab_rows(p.M);
    // Up to four rows leave half of the MMA's columns idle: there go the parts of
    // x * gamma that rounding it cuts off, if they fit beside a second CTA.
    p.halves = p.gamma != nullptr && p.slab <= 4 && smem_bytes(2 * p.slab, p.K) <= kSmemPair;
    cudaError_t e = cudaErrorInvalidValue;
#define FL_CASE(DT, DUAL, V)                                             \
    if (dt == DT && dual == DUAL && p.group == 32 * V)                   \
        e = p.zeros[0] != nullptr ? launch_rows<DT, DUAL, V, true>(p, ctx, stream) \
                                  : launch_rows<DT, DUAL, V, false>(p, ctx, stream);
    FL_CASE(0, false, 1) FL_CASE(0, false, 2) FL_CASE(0, false, 4) FL_CASE(0, true, 1) FL_CASE(0, true, 2) FL_CASE(0, true, 4)
    FL_CASE(1, false, 1) FL_CASE(1, false, 2) FL_CASE(1, false, 4) FL_CASE(1, true, 1) FL_CASE(1, true, 2) FL_CASE(1, true, 4)
#undef FL_CASE
    return host::launched(e, "4-bit decode kernel");
}

}  // namespace fl
