// 4-bit products for more rows than the decode kernel takes, on the tensor cores.
//
// The weight is the M operand: a tile takes 128 weight rows (or, for the
// SwiGLU pair, 64 rows of Wg and the same rows of Wu) against up to 256 tokens,
// so that the 4-bit codes are expanded where the MMA reads them: in tensor
// memory. Each K step of 64 a dequantising thread owns one weight row: it reads
// 32 bytes of codes from shared memory, forms the weight in the dtype and writes
// its row of the A operand with tcgen05.st; the tokens are the B operand, staged
// by TMA. 16-bit weights exist nowhere else.
//
// Roundings: the weight is rounded once, scale * (code - zero), or with the
// RMSNorm prologue scale * gamma * (code - zero), so that the tokens are
// multiplied as they are: with the output's two roundings, the error 1.4 times
// that of an fp32 product rounded once (rounding x * gamma as well would be a
// third: 1.6 times). The row scale 1 / rms, from a kernel of its own
// that reads x once, is applied to the fp32 sums. (That kernel and the products with
// gamma: 64 x 4096 x 4096 16.4 us instead of 11.3, 333 rows 24.1 instead of 17.3, 2048
// rows 58.5 instead of 45.5.)
//
// What bounds it, per K step: with 256 tokens the MMA (514 cycles; 512 by the
// tensor rate), with fewer the expansion of the codes, which sets a step's
// least time whatever the tile's width: some 540 cycles, a tenth more where gamma
// is multiplied in. Measured in graphs: 4096^3 86 to 92 us from run to run (1490 to 1600 TFLOP/s),
// 2048 rows of the SwiGLU FFN 4096 x 11008 368 to 403 us (1375 to 1505 TFLOP/s),
// 333 x 6144 x 4096 30 to 32 us, 64 x 4096 x 4096 14.0 to 16.4 us. The warps fetch instructions
// as hard as they compute: a step's two halves as one loop of half the code took
// 6 % off every size, four quarters gave it back. A tile of two blocks of 128
// rows by 128 tokens moved fewer bytes per MMA but expanded every code for half
// as many tokens: 237 us at 4096^3, when this one took 149.
//
// Roles: warp 0 loads tokens (stages of 64 k) and codes (stages of 256 k) by
// TMA, warp 1 owns tensor memory and issues the MMAs, warps 2 and 3 load the
// scales, zero points and gamma of 1024 k at a time into shared memory
// (transposed: one row per thread there; the first of them is loaded by the
// dequantising warps, which have nothing else to do yet), warps 4-19 dequantise,
// four to a K step, and apply the epilogue. (20 warps: a 21st would leave each
// thread 80 registers instead of 96; eight dequantising warps, with twice the
// registers, took 163 us at 4096^3.) The producer loads codes whenever their ring
// has room, so that they, which come from HBM and are needed first, run ahead as
// far as it reaches; the fewer the tokens, the more of shared memory is the
// codes'. A stage of tokens and the A slot of the same step share one full and
// one empty barrier (the bytes and the four warps' arrivals on the one, the MMA's
// commit on the other), so that the issuing warp waits once a step. No role
// divides inside a step: the producer's tile arithmetic alone, done per step, once
// held a step at 750 cycles.
//
// Few tiles: the K range is split over a cluster of up to 8 CTAs whose fp32
// partials are added through distributed shared memory in rank order. Without
// a split the CTAs are persistent: every ring runs on into the next tile, and
// the dequantising warps expand the next tile's first steps before they apply
// the epilogue, which holds the MMAs up only while the accumulator is read.
// Tiles left over from whole waves of CTAs go to a second launch, split over
// clusters, whose CTAs start as those of the last wave end: FFN 4096 x 11008
// with 64 rows 84 -> 68 us, 333 x 11008 x 4096 68 -> 49 us. (Equal shares of the
// last tiles' K range to every CTA of one launch, with partials through global
// memory, cost 6 to 13 us for the exchange: 333 x 11008 x 4096 59 us.)
//
// Every mbarrier wait is bounded as in the other kernels.
#include <atomic>
#include <type_traits>

#include "fl_common.cuh"
#include "fl_host.h"
#include "fl_resident.h"
#include "fl_w4.h"

namespace fl {

namespace {

constexpr int kThreads = 640;
constexpr int kRows = 128;       // weight rows of a tile (TMEM lanes)
constexpr int kTok = 256;        // tokens of a tile at most
constexpr int kStep = 64;        // k per B stage and A slot
constexpr int kGroups = 4;       // dequantising warpgroups: K step kb goes to kb % 4
constexpr int kWk = kGroups * kStep;  // k per code stage: one step of each warpgroup
constexpr int kSIter = 4;        // code stages per scale stage
constexpr int kSk = kSIter * kWk;
constexpr int kStages = 2 * kGroups, kWStages = 8, kSStages = 2;  // (at most; stages of tokens: 4 to 8)
constexpr int kRing = 192 * 1024;                   // both rings
constexpr int kWBytes = kRows * kWk / 2;            // 16 KB
constexpr int kSPitch = 130;                        // 16-bit scales of one group: 128 rows, padded
constexpr int kZPitch = 132;                        // zero-point bytes of one group
constexpr int kSGroups = kSk / 32;
constexpr int kSBytes = kSGroups * kSPitch * 2;
constexpr int kZBytes = kSGroups * kZPitch;
constexpr int kGBytes = kSk * 2;                    // gamma

constexpr int kOffS = kRing;
constexpr int kOffZ = kOffS + kSStages * kSBytes;
constexpr int kOffG = (kOffZ + kSStages * kZBytes + 15) / 16 * 16;
constexpr int kOffBar = kOffG + kSStages * kGBytes;
constexpr int kBars = 2 * kStages + 2 * kWStages + 2 * kSStages + 3;
constexpr int kOffSlot = kOffBar + kBars * 8;
constexpr int kSmem = kOffSlot + 16 + 1024;         // + alignment slack
static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
static_assert(kRows * kTok * 4 <= kRing, "the partial sums fit in the rings");

constexpr int kACol = 256;  // first tensor-memory column of the A slots (the accumulator: 0 .. 255)

struct TileParams {
    CUtensorMap tm_x;     // x [M, K], box {64, BT}
    CUtensorMap tm_q[2];  // codes [N, K / 2] bytes, box {128, 128} (pair: {128, 64} each)
    W4Params w;
    const float* row_scale;  // [M] 1 / rms of the rows of x, over kLift (with gamma)
    int bt, splits, steps_per_split, steps;  // K steps of 64
    int row_tiles, tile0, tiles;             // tiles tile0 .. tiles - 1
    int tail;                                // the second launch of a product
    int stages, w_stages, b_bytes;           // rings: stages * b_bytes of tokens, then the code stages
    int* status;
    unsigned long long timeout_ns;
};

// scale * gamma * (code - zero) is formed times this, a power of two that puts
// weights of usual sizes in the middle of fp16's range, and the row scale times
// its inverse.
template <int DT>
constexpr float kLift = DT == DT_F16 ? 64.f : 1.f;

template <int DT>
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    if constexpr (DT == DT_F16)
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    else
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// a * b in fp32, of the halves of two 16-bit pairs (exact: at most 5 and 11 significant bits)
template <int DT>
__device__ __forceinline__ float2 widening_mul(uint32_t a, uint32_t b) {
    float2 r;
    if constexpr (DT == DT_F16)
        asm("{\n\t.reg .b16 al, ah, bl, bh;\n\tmov.b32 {al, ah}, %2;\n\tmov.b32 {bl, bh}, %3;\n\t"
            "fma.rn.f32.f16 %0, al, bl, 0f80000000;\n\tfma.rn.f32.f16 %1, ah, bh, 0f80000000;\n\t}"
            : "=f"(r.x), "=f"(r.y) : "r"(a), "r"(b));
    else
        asm("{\n\t.reg .b16 al, ah, bl, bh;\n\tmov.b32 {al, ah}, %2;\n\tmov.b32 {bl, bh}, %3;\n\t"
            "fma.rn.f32.bf16 %0, al, bl, 0f80000000;\n\tfma.rn.f32.bf16 %1, ah, bh, 0f80000000;\n\t}"
            : "=f"(r.x), "=f"(r.y) : "r"(a), "r"(b));
    return r;
}

// Two fp32 products in one instruction.
__device__ __forceinline__ float2 mul2_f32(float2 a, float b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b));
    return d;
}

// Eight codes of a word, in order, as four pairs of weights. The code goes into
// the mantissa of a power of two B (128 bf16, 1024 fp16): the even one as B + c,
// the odd one, taken from the word shifted by one, as B + 8 c, and one FMA with
// (1, 1/8) and (-(B + z), -(B/8 + z)) leaves c - z, exactly. The product with
// the scale (s: its 16 bits twice) is the one rounding; with NORM gamma
// (g: of the 8 k) is multiplied in first, in fp32 and exactly (s: its fp32 bits).
template <int DT, bool NORM>
__device__ __forceinline__ void dequant8(uint32_t w, uint32_t s, uint32_t zc, const uint4& g, uint32_t* out) {
    constexpr uint32_t kMagic = DT == DT_F16 ? 0x64006400u : 0x43004300u;
    constexpr uint32_t kUnit = DT == DT_F16 ? 0x30003c00u : 0x3e003f80u;  // (1, 1/8)
    const uint32_t v = w >> 1, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = __byte_perm(w, v, (uint32_t)(i * 0x1111 + 0x4400));  // bytes w.i, w.i, v.i, v.i
        const uint32_t code = hfma2<DT>(and_or(pair, 0x0078000fu, kMagic), kUnit, zc);
        if constexpr (NORM) {
            const float2 f = mul2_f32(widening_mul<DT>(code, gw[i]), __uint_as_float(s));
            out[i] = DTypeOps<DT>::pack(f.x, f.y);
        } else {
            out[i] = DTypeOps<DT>::mul2(code, s);
        }
    }
}

// (-(B + z), -(B/8 + z)) for the FMA above
template <int DT>
__device__ __forceinline__ uint32_t zero_const(uint32_t z) {
    return (DT == DT_F16 ? 0xd800e400u : 0xc180c300u) + z * 0x00080001u;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// One K step, by a whole converged warp: four MMAs (A in tensor memory, 8
// columns each; B 32 bytes further along its swizzled rows) and the commit that
// frees the step's stage, issued by one elected lane. Operands computed by the
// converged warp stay in uniform registers, where the instructions take them
// from; under a divergent `lane == 0` each MMA waits for its operands to be moved
// there (487 cycles a step at least, measured alone, against 200).
__device__ __forceinline__ void mma_step(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t acc,
                                         uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 r, a1, a2, a3, l1, l2, l3;\n\t.reg .b64 b0, b1, b2, b3;\n\t"
        "elect.sync r|p, 0xffffffff;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
        "add.u32 l1, %2, 2;\n\tadd.u32 l2, %2, 4;\n\tadd.u32 l3, %2, 6;\n\t"
        "mov.b64 b0, {%2, %3};\n\tmov.b64 b1, {l1, %3};\n\tmov.b64 b2, {l2, %3};\n\tmov.b64 b3, {l3, %3};\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b0, %4, q;\n\t"
        "setp.eq.u32 q, 0, 0;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %4, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %4, q;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void commit_elected(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 r;\n\telect.sync r|p, 0xffffffff;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// 1 / rms (over kLift) of the rows of x [M, K]: one warp per row, eight vectors in flight per lane.
template <int DT>
__global__ void __launch_bounds__(256) fl_w4_row_scale_kernel(const uint16_t* __restrict__ x, float* __restrict__ scale,
                                                              int M, int K, float eps) {
    using Ops = DTypeOps<DT>;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long m = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (m >= M) return;
    const uint16_t* row = x + m * K;
    float s0 = 0.f, s1 = 0.f;
    for (int k0 = lane * 8; k0 < K; k0 += 256 * 8) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = k0 + u * 256 < K ? ldg_v4(row + k0 + u * 256) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = Ops::unpack(w[e]);
                s0 = fmaf(f.x, f.x, s0);
                s1 = fmaf(f.y, f.y, s1);
            }
        }
    }
    float s = s0 + s1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) scale[m] = rsqrtf(s / (float)K + eps) * (1.f / kLift<DT>);
}

// RES: a residual is added.
template <int DT, bool DUAL, bool NORM, bool RES>
__global__ void __launch_bounds__(kThreads, 1) fl_w4_tile_kernel(const __grid_constant__ TileParams p) {
    using Ops = DTypeOps<DT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sbase - raw);
    const W4Params& w = p.w;

    const uint32_t bar0 = sbase + kOffBar;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto wfull = [&](int s) { return bar0 + 8u * (2 * kStages + s); };
    auto wempty = [&](int s) { return bar0 + 8u * (2 * kStages + kWStages + s); };
    auto sfull = [&](int s) { return bar0 + 8u * (2 * kStages + 2 * kWStages + s); };
    auto sempty = [&](int s) { return bar0 + 8u * (2 * kStages + 2 * kWStages + kSStages + s); };
    const uint32_t dfull = bar0 + 8u * (kBars - 3), dempty = bar0 + 8u * (kBars - 2), drain = bar0 + 8u * (kBars - 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first_tile = p.tile0 + blockIdx.x / p.splits, tile_step = gridDim.x / p.splits, rank = blockIdx.x % p.splits;
    const int k0 = rank * p.steps_per_split, k1 = min(p.steps, k0 + p.steps_per_split), nk = k1 - k0;
    const int its = (nk + kGroups - 1) / kGroups;        // code stages of a tile
    const int s_count = (its + kSIter - 1) / kSIter;     // scale stages of a tile
    const int nb = p.stages, nw = p.w_stages;
    const uint32_t wring = sbase + (uint32_t)(nb * p.b_bytes);
    // weight rows run fastest: the CTAs at work share a few tiles of tokens
    auto row0_of = [&](int tile) { return tile % p.row_tiles * (DUAL ? kRows / 2 : kRows); };
    auto token0_of = [&](int tile) { return tile / p.row_tiles * p.bt; };
    // weight and row of TMEM lane r: for the pair, each warp's lanes 0-15 are
    // rows of Wg and 16-31 the same rows of Wu
    auto weight_of = [&](int r) { return DUAL ? (r >> 4) & 1 : 0; };
    auto row_in_tile = [&](int r) { return DUAL ? (r >> 5) * 16 + (r & 15) : r; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1 + 4);
            mbar_init(empty(s), 1);
        }
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(wfull(s), 1);
            mbar_init(wempty(s), 4 * kGroups);
        }
        for (int s = 0; s < kSStages; ++s) {
            mbar_init(sfull(s), 2);
            mbar_init(sempty(s), 4 * kGroups);
        }
        mbar_init(dfull, 1);
        mbar_init(dempty, 4 * kGroups);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&p.tm_x);
        tma_prefetch_desc(&p.tm_q[0]);
        if (DUAL) tma_prefetch_desc(&p.tm_q[1]);
    }
    if (warp == 1) {
        tmem_alloc(sbase + kOffSlot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kOffSlot);
    // the first codes towards L2 (the point of coherence) while the previous kernel finishes
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < nw && i < its; ++i)
            for (int j = 0; j <= (DUAL ? 1 : 0); ++j)
                tma_prefetch_2d(&p.tm_q[j], k0 * (kStep / 2) + i * (kWk / 2), row0_of(first_tile));
    }
    // The tail of a product need not wait for the launch before it, which waited
    // itself for what both read before it let this one in; it waits before it
    // ends, so that what follows finds both done.
    if (!p.tail) griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();

    // Scales, zero points and gamma of scale stage i of a tile into stage slot s
    // of shared memory, by `count` threads: neighbouring threads take
    // neighbouring groups of a row.
    auto load_scales = [&](int tile, int i, int s, int tid, int count) {
        const int per_row = w.K / w.group, ng = kSk / w.group, sh = 31 - __clz(ng);  // groups of a row; of a stage (8, 16, 32)
        const int g0 = (k0 * kStep + i * kSk) / w.group, g_end = min(per_row, (k1 * kStep + w.group - 1) / w.group);
        const int n0 = row0_of(tile);
        uint16_t* ds = reinterpret_cast<uint16_t*>(smem + kOffS + s * kSBytes);
        uint8_t* dz = smem + kOffZ + s * kZBytes;
        const bool zeros = w.zeros[0] != nullptr;
        if (NORM) {
            // (past K zeros: the tokens are zero there too)
            uint4* dg = reinterpret_cast<uint4*>(smem + kOffG + s * kGBytes);
            for (int e = tid; e < kSk / 8; e += count) {
                const int k = k0 * kStep + i * kSk + e * 8;
                dg[e] = k < w.K ? ldg_v4(w.gamma + k) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        constexpr int U = 8;  // loads in flight per thread
        for (int b = tid; b < kRows << sh; b += count * U) {
            uint16_t v[U];
            uint8_t z[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = b + count * u, r = e >> sh, g = g0 + (e & (ng - 1)), n = n0 + row_in_tile(r);
                const bool in = r < kRows && n < w.N && g < g_end;
                const size_t at = in ? (size_t)n * per_row + g : 0;  // (0: a valid address whose value is not used)
                v[u] = __ldg((weight_of(r) ? w.scales[1] : w.scales[0]) + at);
                if (zeros) z[u] = __ldg((weight_of(r) ? w.zeros[1] : w.zeros[0]) + at);
                if (!in) v[u] = 0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = b + count * u, r = e >> sh, g = e & (ng - 1);
                if (r < kRows) {
                    ds[g * kSPitch + r] = v[u];
                    dz[g * kZPitch + r] = zeros ? (uint8_t)(z[u] & 15) : (uint8_t)8;
                }
            }
        }
    };

    // ---------------------------------------------------------------- epilogue of the dequantising warps
    const int grp = (warp - 4) >> 2, r = (threadIdx.x - 128) & 127;
    const uint32_t dcol = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    // Outputs of tokens [t0, t0 + 4 T) of a tile, from this lane's accumulators of
    // them (t0 and m0 multiples of 4). Lane pairs exchange, so that each stores two
    // neighbouring outputs of a token at once.
    auto emit = [&](auto T, int n0, int m0, int t0, const float* v) {
        const int n = n0 + row_in_tile(r), nn = n & ~1;
        const bool odd = lane & 1, up = lane & 16;
        // this lane's first token: for the pair, gate lanes take tokens 0 and 2 of four, up lanes 1 and 3
        const int mine = m0 + t0 + (DUAL ? (up ? 1 : 0) + (odd ? 2 : 0) : (odd ? 1 : 0));
        const int end = nn < w.N ? min(w.M, m0 + p.bt) : 0;  // tokens below it are stored
        uint16_t* out = w.out + (size_t)mine * w.N + nn;
        // (all of the residual is requested before any of it is used)
        [[maybe_unused]] uint32_t res[2 * decltype(T)::value];
        if constexpr (RES) {
            const uint16_t* src = w.residual + (size_t)mine * w.N + nn;
#pragma unroll
            for (int e = 0; e < 2 * decltype(T)::value; ++e)
                res[e] = mine + 2 * e < end ? *reinterpret_cast<const uint32_t*>(src + 2 * e * (size_t)w.N) : 0u;
        }
        [[maybe_unused]] const float bias = !DUAL && w.bias != nullptr && n < w.N ? Ops::unpack(w.bias[n]).x : 0.f;
        // of two values, the one for the even lane stays there, the other goes over
        auto exchange = [&](float v0, float v1) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
            return make_float2(odd ? got : v0, odd ? v1 : got);
        };
        auto store = [&](float2 y, int t, size_t at) {
            if (mine + t >= end) return;
            if constexpr (RES) {
                const float2 x = Ops::unpack(res[t / 2]);
                y.x += x.x;
                y.y += x.y;
            }
            *reinterpret_cast<uint32_t*>(out + at) = Ops::pack(y.x, y.y);
        };
        auto all = [&](auto act) {
            size_t at = 0;
#pragma unroll
            for (int e = 0; e < 4 * decltype(T)::value; e += 4, at += 4 * (size_t)w.N) {
                float a[4] = {v[e], v[e + 1], v[e + 2], v[e + 3]};
                if (NORM) {
                    const float4 rs = __ldg(reinterpret_cast<const float4*>(p.row_scale + m0 + t0 + e));
                    a[0] *= rs.x;
                    a[1] *= rs.y;
                    a[2] *= rs.z;
                    a[3] *= rs.w;
                }
                if constexpr (DUAL) {
                    // lanes 16 apart hold the gate and the up value of a row
                    const float o0 = __shfl_xor_sync(0xffffffffu, up ? a[0] : a[1], 16);
                    const float o1 = __shfl_xor_sync(0xffffffffu, up ? a[2] : a[3], 16);
                    store(exchange(w4_act(ACT_SILU, up ? o0 : a[0]) * (up ? a[1] : o0),
                                   w4_act(ACT_SILU, up ? o1 : a[2]) * (up ? a[3] : o1)),
                          e, at);
                } else {
                    store(exchange(act(a[0] + bias), act(a[1] + bias)), e, at);
                    store(exchange(act(a[2] + bias), act(a[3] + bias)), e + 2, at + 2 * (size_t)w.N);
                }
            }
        };
        // (the activation is chosen once, not per value)
        if (DUAL || w.act == ACT_NONE) all([](float y) { return y; });
        else all([&](float y) { return w4_act(w.act, y); });
    };
    // Epilogue of the i-th tile of this CTA. false: the MMAs did not finish.
    auto epilogue = [&](int tile, int i) {
        if (!__all_sync(0xffffffffu, wait_bar(dfull, (uint32_t)(i & 1), p.status, p.timeout_ns, 28))) return false;
        tc_fence_after();
        const int n0 = row0_of(tile), m0 = token0_of(tile), chunks = (p.bt + 31) / 32;
        auto release = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dempty);
        };
        if (grp >= chunks) release();
        for (int c = grp; c < chunks; c += kGroups) {
            float v[32];
            tmem_ld_32x32b_x32(dcol + 32u * c, reinterpret_cast<uint32_t(&)[32]>(v));
            tmem_ld_wait();
            if (p.splits == 1) {
                if (c + kGroups >= chunks) release();
                emit(std::integral_constant<int, 8>(), n0, m0, 32 * c, v);
            } else {
                // partial sums into this CTA's shared memory: [token][row]
                float* part = reinterpret_cast<float*>(smem);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (32 * c + e < p.bt) part[(32 * c + e) * kRows + r] = v[e];
            }
        }
        return true;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer of tokens and codes
        if (lane == 0) {
            // Codes: the next stage's tile, index in it, ring slot and phase. They
            // are loaded as soon as their ring has room, looked for once per step of
            // tokens, and waited for only where that step needs them (so tokens never
            // run ahead of codes, and the wait cannot be for itself).
            int c_tile = first_tile, c_at = 0, c_s = 0, c_issued = 0, c_row = row0_of(first_tile);
            uint32_t c_ph = 0;
            auto load_codes = [&] {
                mbar_arrive_expect_tx(wfull(c_s), kWBytes);
                const uint32_t dst = wring + c_s * kWBytes;
                const int x = (k0 + c_at * kGroups) * (kStep / 2);
                tma_load_2d(dst, &p.tm_q[0], wfull(c_s), x, c_row);
                if (DUAL) tma_load_2d(dst + kWBytes / 2, &p.tm_q[1], wfull(c_s), x, c_row);
                ++c_issued;
                if (++c_s == nw) c_s = 0, c_ph ^= 1u;
                if (++c_at == its) c_at = 0, c_tile += tile_step, c_row = row0_of(c_tile);
            };
            int issued = 0, s = 0, stages = 0;  // token loads, their slot, code stages before this tile
            uint32_t ph = 0;
            bool ok = true;
            for (int tile = first_tile; ok && tile < p.tiles; tile += tile_step, stages += its) {
                const int t0 = token0_of(tile);
                for (int kb = 0; kb < nk; ++kb) {
                    if (c_issued <= stages + kb / kGroups) {
                        if (!(ok = wait_bar(wempty(c_s), c_ph ^ 1u, p.status, p.timeout_ns, 20))) break;
                        load_codes();
                    } else if (c_tile < p.tiles && mbar_try_wait_cluster(wempty(c_s), c_ph ^ 1u)) {
                        load_codes();
                    }
                    if (!(ok = wait_bar(empty(s), ph ^ 1u, p.status, p.timeout_ns, 21))) break;
                    mbar_arrive_expect_tx(full(s), (uint32_t)p.b_bytes);
                    tma_load_2d(sbase + s * p.b_bytes, &p.tm_x, full(s), (k0 + kb) * kStep, t0);
                    ++issued;
                    if (++s == nb) s = 0, ph ^= 1u;
                }
            }
            // every load this thread issued lands before the CTA may exit
            for (int i = 1; i <= nb && i <= issued; ++i)
                wait_bar_drain(full((issued - i) % nb), (uint32_t)(((issued - i) / nb) & 1), 20000000ull);
            for (int i = 1; i <= nw && i <= c_issued; ++i)
                wait_bar_drain(wfull((c_issued - i) % nw), (uint32_t)(((c_issued - i) / nw) & 1), 20000000ull);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (the whole warp, converged)
        // The next step's barrier is tested while this step's MMAs are issued, and
        // tensor memory's base is taken as what it is when all 512 columns are
        // allocated: 0, so that no operand comes from a register of the warp.
        const uint32_t idesc = umma_idesc_f16(Ops::kFormat, 128, (uint32_t)p.bt);
        const uint64_t desc = sw128_kmajor_desc(sbase);
        const uint32_t lo0 = (uint32_t)desc, hi = (uint32_t)(desc >> 32), lo_step = (uint32_t)p.b_bytes >> 4;
        bool ok = true;
        uint32_t ph = 0, lo = lo0, slot = 0, ready = 0;
        for (int tile = first_tile, i = 0; ok && tile < p.tiles; tile += tile_step, ++i) {
            // the previous tile's accumulator has been read
            if (i > 0) ok = __all_sync(0xffffffffu, wait_bar(dempty, (uint32_t)((i - 1) & 1), p.status, p.timeout_ns, 29));
            for (int kb = 0; ok && kb < nk; ++kb) {
                if (!__all_sync(0xffffffffu, ready) &&
                    !(ok = __all_sync(0xffffffffu, wait_bar(full(slot), ph, p.status, p.timeout_ns, 22))))
                    break;
                tc_fence_after();
                const uint32_t now = slot, now_lo = lo;
                ++slot;
                lo += lo_step;
                if (slot == (uint32_t)nb) slot = 0, lo = lo0, ph ^= 1u;
                ready = mbar_try_wait_cluster(full(slot), ph);
                mma_step(0u, kACol + 32u * now, now_lo, hi, idesc, (uint32_t)kb, empty(now));
            }
            if (ok) commit_elected(dfull);
        }
        // all MMAs issued by this warp complete before tensor memory is released
        commit_elected(drain);
        wait_bar_drain(drain, 0, 20000000ull);
    } else if (warp < 4) {
        // ------------------------------------------------------------ scales and zero points of the stages after the first
        int g = 0;  // scale stages so far
        bool ok = true;
        for (int tile = first_tile; ok && tile < p.tiles; tile += tile_step)
            for (int i = 0; i < s_count; ++i, ++g) {
                if (g == 0) continue;
                const int s = g % kSStages;
                if (!(ok = __all_sync(0xffffffffu, wait_bar(sempty(s), (uint32_t)((g / kSStages) & 1) ^ 1u, p.status, p.timeout_ns, 24))))
                    break;
                load_scales(tile, i, s, threadIdx.x - 64, 64);
                __syncwarp();
                if (lane == 0) mbar_arrive(sfull(s));
            }
    } else {
        // ------------------------------------------------------------ dequantise, one row per thread
        const int gsh = 31 - __clz(w.group);
        // this row's codes of the warpgroup's K step in a code stage
        const int srow = weight_of(r) * (kRows / 2) + row_in_tile(r);
        const uint32_t src0 = wring + srow * 128 + (((2 * grp) ^ (srow & 7)) << 4);
        const uint32_t src1 = wring + srow * 128 + (((2 * grp + 1) ^ (srow & 7)) << 4);
        load_scales(first_tile, 0, 0, threadIdx.x - 128, 512);
        named_bar_sync(1, 512);
        bool ok = true;
        int ws = 0, g = 0, done = 0, last = -1;  // scale stages and tiles so far
        int base = 0;                            // A slot of the tile's first step, and its phase
        uint32_t wph = 0, base_ph = 0;
        for (int tile = first_tile; ok && tile < p.tiles; tile += tile_step) {
            int a = base + grp;
            uint32_t aph = base_ph;
            if (a >= nb) a -= nb, aph ^= 1u;
            for (int it = 0; ok && it < its; ++it) {
                const int ss = g % kSStages, kb = it * kGroups + grp;
                ok = wait_bar(wfull(ws), wph, p.status, p.timeout_ns, 25);
                if (ok && it % kSIter == 0 && g > 0) {
                    // (the barrier of slot 0 saw no phase for the very first stage)
                    const int phases = g / kSStages - (ss == 0 ? 1 : 0);
                    ok = wait_bar(sfull(ss), (uint32_t)(phases & 1), p.status, p.timeout_ns, 26);
                }
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                if (kb < nk) {
                    ok = __all_sync(0xffffffffu, wait_bar(empty(a), aph ^ 1u, p.status, p.timeout_ns, 27));
                    if (!ok) break;
                    tc_fence_after();
                    const uint16_t* ds = reinterpret_cast<const uint16_t*>(smem + kOffS + ss * kSBytes) + r;
                    const uint8_t* dz = smem + kOffZ + ss * kZBytes + r;
                    const int kin = (it % kSIter) * kWk + grp * kStep;
                    const uint32_t sg = sbase + kOffG + ss * kGBytes + kin * 2;
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        const uint4 c = ld_shared_v4((h ? src1 : src0) + ws * kWBytes);
                        const int g1 = (kin + 32 * h) >> gsh;
                        uint32_t sc = ds[g1 * kSPitch];
                        sc = NORM ? __float_as_uint(Ops::unpack(sc).x * kLift<DT>) : sc * 0x10001u;
                        const uint32_t zc = zero_const<DT>(dz[g1 * kZPitch]);
                        const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint4 gv = NORM ? ld_shared_v4(sg + 64 * h + 16 * e) : make_uint4(0u, 0u, 0u, 0u);
                            dequant8<DT, NORM>(cw[e], sc, zc, gv, o + 4 * e);
                        }
                        tmem_st_32x32b_x16(dcol + kACol + 32u * a + 16u * h, o);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) {
                    if (kb < nk) mbar_arrive(full(a));
                    mbar_arrive(wempty(ws));
                }
                if (kb < nk && (a += kGroups) >= nb) a -= nb, aph ^= 1u;
                if (++ws == nw) ws = 0, wph ^= 1u;
                if (it % kSIter == kSIter - 1 || it == its - 1) {
                    if (lane == 0) mbar_arrive(sempty(ss));
                    ++g;
                }
                // the tile before this one: its last MMAs ran while this tile's first steps were expanded
                if (it == 0 && last >= 0) {
                    ok = epilogue(last, done++);
                    last = -1;
                }
            }
            last = tile;
            base += nk;
            base_ph ^= (uint32_t)(base / nb) & 1u;
            base %= nb;
        }
        if (ok && last >= 0) epilogue(last, done);
    }

    if (p.splits > 1) {
        __syncwarp();
        cluster_barrier_sync();
        // each rank finishes its range of tokens of the cluster's one tile
        if (warp >= 4) {
            const int n0 = row0_of(first_tile), m0 = token0_of(first_tile);
            const int per = ((p.bt + p.splits - 1) / p.splits + 3) & ~3;
            const int t1 = min(p.bt, (rank + 1) * per);
            for (int t = rank * per + 4 * grp; t < t1; t += 4 * kGroups) {
                float v[8][4];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (i >= p.splits) break;
                    const uint32_t a = mapa_cluster(sbase + (uint32_t)(t * kRows + r) * 4u, (uint32_t)i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[i][e] = ld_cluster_f32(a + e * kRows * 4);
                }
#pragma unroll
                for (int i = 1; i < 8; ++i)
                    if (i < p.splits)
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[0][e] += v[i][e];
                emit(std::integral_constant<int, 1>(), n0, m0, t, v[0]);
            }
        }
        __syncwarp();
        cluster_barrier_sync();  // no CTA leaves while another reads its sums
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (p.tail) griddep_wait();
}

template <int DT, bool DUAL, bool NORM, bool RES>
struct Kern {
    static cudaError_t configure(int device) {
        static std::atomic<unsigned long long> done{0};
        return host::allow_smem(fl_w4_tile_kernel<DT, DUAL, NORM, RES>, kSmem, device, done);
    }
    static void config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* a, dim3 grid, int splits, int pdl, cudaStream_t s) {
        cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = kSmem;
        cfg.stream = s;
        a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        a[0].val.programmaticStreamSerializationAllowed = pdl;
        a[1].id = cudaLaunchAttributeClusterDimension;
        a[1].val.clusterDim.x = (unsigned)splits;
        a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
        cfg.attrs = a;
        cfg.numAttrs = 2;
    }
    static cudaError_t launch(const TileParams& p, dim3 grid, const host::LaunchContext& ctx, cudaStream_t s) {
        cudaError_t e = configure(ctx.device);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute a[2];
        config(cfg, a, grid, p.splits, ctx.pdl, s);
        return cudaLaunchKernelEx(&cfg, fl_w4_tile_kernel<DT, DUAL, NORM, RES>, p);
    }
    // clusters of `splits` CTAs that are resident at once
    static cudaError_t resident(int splits, int device, int* n) {
        cudaError_t e = configure(device);
        if (e == cudaSuccess) {
            cudaLaunchConfig_t cfg;
            cudaLaunchAttribute a[2];
            config(cfg, a, dim3((unsigned)splits), splits, 0, nullptr);
            e = cudaOccupancyMaxActiveClusters(n, fl_w4_tile_kernel<DT, DUAL, NORM, RES>, &cfg);
        }
        if (e != cudaSuccess) cudaGetLastError();  // (reported here: not the next launch's)
        return e;
    }
};

}  // namespace

size_t w4_tile_workspace(int M, bool norm) { return norm ? ((size_t)M + kTok + 32) * sizeof(float) : 0; }

fl_status w4_tile(int dt, bool dual, const W4Params& w, void* workspace, const host::LaunchContext& ctx, cudaStream_t stream) {
    TileParams p;
    const bool norm = w.gamma != nullptr;
    p.row_scale = nullptr;
    if (norm) {
        float* scale = static_cast<float*>(workspace);
        p.row_scale = scale;
        const dim3 grid((unsigned)((w.M + 7) / 8));
        // Its CTAs begin only when the kernel before it is done if they have much to read: let in
        // early they crowd into the few multiprocessors that are idle in its last wave
        // (us of a product, early / not: 64 x 4096^2 16.6 / 16.9, 333 24.1 / 24.8, 1024 33.7 / 34.0,
        // 2048 65.7 / 59.1; 333 x 6144 x 4096 33.8 / 31.8, 333 x 11008 x 4096 44.9 / 45.3).
        const int early = (long long)w.M * w.K < (1ll << 21) ? ctx.pdl : 0;
        auto kern = dt == FL_F16 ? fl_w4_row_scale_kernel<DT_F16> : fl_w4_row_scale_kernel<DT_BF16>;
        const fl_status st = host::launched(host::launch(kern, grid, 256, 0, early, stream, w.x, scale, w.M, w.K, w.eps),
                                            "row scale kernel");
        if (st != FL_OK) return st;
    }
    p.steps = (w.K + kStep - 1) / kStep;
    const int rows = dual ? kRows / 2 : kRows, row_tiles = (w.N + rows - 1) / rows;
    // Tokens of a tile and K split: the least time of whole waves of resident
    // CTAs or clusters, in cycles as measured. A K step costs the MMA (2.2 a
    // token) or, below some 260 tokens, what its warps need to expand the codes and
    // to issue it (570; 690 with gamma, which is multiplied in in fp32); a wave
    // its epilogue, a split the exchange of the partial sums. Tiles left over from
    // whole waves may be split in a launch of their own (the tail), which fills
    // the multiprocessors as they fall idle. Ranges of a split are multiples of
    // 128 k, the largest group.
    static Resident<host::kMaxDevices, 8> resident;
    double least = 0;
    const int tt0 = (w.M + kTok - 1) / kTok;
    int token_tiles = 0, tail_splits = 1;
    auto split_steps = [&](int s) { return ((p.steps + 1) / 2 + s - 1) / s * 2; };
    auto can_split = [&](int s) {
        const int per = split_steps(s);
        return per >= 4 && (p.steps + per - 1) / per == s;
    };
    auto clusters = [&](int s, int* n) {  // resident at once
        return (cudaError_t)resident.get(
            ctx.device, s, [&](int* got) { return (int)Kern<DT_BF16, false, false, false>::resident(s, ctx.device, got); }, n);
    };
    int n1 = 0;
    const cudaError_t asked = clusters(1, &n1);
    if (asked != cudaSuccess)
        return host::fail(FL_ERR_CUDA, "4-bit tile kernel: occupancy query: %s", cudaGetErrorString(asked));
    if (n1 == 0) return host::fail(FL_ERR_CUDA, "4-bit tile kernel: no resident CTA");
    for (int tt = tt0; tt <= 3 * tt0 && tt <= tt0 + 64; ++tt) {
        const int bt = ((w.M + tt - 1) / tt + 15) / 16 * 16;
        if (tt > tt0 && bt < 64) break;
        // (rounded up to 16 tokens, fewer tiles may do; none starts at or past M)
        const int count = (w.M + bt - 1) / bt;
        const long long tiles = (long long)row_tiles * count;
        const double least_step = norm ? 690.0 : 570.0, step = 2.2 * bt > least_step ? 2.2 * bt : least_step;
        const double round = step * p.steps + 6000.0;
        auto consider = [&](double cost, int splits, int tail) {
            if (token_tiles != 0 && cost >= least) return;
            least = cost;
            token_tiles = count;
            p.bt = bt;
            p.splits = splits;
            tail_splits = tail;
        };
        consider(5000.0 + (double)((tiles + n1 - 1) / n1) * round, 1, 1);
        for (int s = 2; s <= 8; ++s) {
            // (a size whose query fails is left out of this choice)
            int n = 0;
            if (!can_split(s) || clusters(s, &n) != cudaSuccess || n == 0) continue;
            const double one = step * split_steps(s) + 11000.0 + 12.0 * bt;
            consider((double)((tiles + n - 1) / n) * one, s, 1);
            if (tiles > n1 && tiles % n1 != 0)
                consider(5000.0 + (double)(tiles / n1) * round + 3000.0 + (double)((tiles % n1 + n - 1) / n) * one, 1, s);
        }
    }
    const long long tiles = (long long)row_tiles * token_tiles;
    if (tiles * p.splits > 0x7fffffffll) return host::fail(FL_ERR_UNSUPPORTED, "4-bit tile kernel: too many tiles");
    p.row_tiles = row_tiles;
    const int all = (int)tiles, plain = tail_splits > 1 ? all / n1 * n1 : all;
    // rings: as many stages of tokens as leave the codes two stages, eight at most; the rest to the codes
    p.b_bytes = p.bt * kStep * 2;
    p.stages = (kRing - 2 * kWBytes) / p.b_bytes;
    if (p.stages > kStages) p.stages = kStages;
    p.w_stages = (kRing - p.stages * p.b_bytes) / kWBytes;
    if (p.w_stages > kWStages) p.w_stages = kWStages;
    fl_status st;
    if ((st = host::encode_matrix(&p.tm_x, dt, 2, w.x, w.K, w.M, kStep, p.bt)) != FL_OK) return st;
    if ((st = host::encode_matrix(&p.tm_q[0], dt, 1, w.q[0], w.K / 2, w.N, kWk / 2, rows)) != FL_OK) return st;
    if (dual && (st = host::encode_matrix(&p.tm_q[1], dt, 1, w.q[1], w.K / 2, w.N, kWk / 2, rows)) != FL_OK) return st;
    if (!dual) p.tm_q[1] = p.tm_q[0];
    p.w = w;
    p.status = ctx.status;
    p.timeout_ns = ctx.timeout_ns;
    if (dual && !norm) return host::fail(FL_ERR_UNSUPPORTED, "4-bit tile kernel: the pair needs gamma");
    // tiles [t0, t1) with K split over clusters of `splits`
    auto launch_tiles = [&](int t0, int t1, int splits) {
        p.tile0 = t0, p.tiles = t1, p.tail = t0 > 0;
        p.splits = splits, p.steps_per_split = split_steps(splits);
        const int n = t1 - t0;
        const bool res = w.residual != nullptr;
        const dim3 grid((unsigned)(splits > 1 ? n * splits : n < n1 ? n : n1));
        cudaError_t e;
#define FL_LAUNCH(DT)                                                                                \
    e = dual ? Kern<DT, true, true, false>::launch(p, grid, ctx, stream)                             \
        : norm ? (res ? Kern<DT, false, true, true>::launch(p, grid, ctx, stream)                    \
                      : Kern<DT, false, true, false>::launch(p, grid, ctx, stream))                  \
               : (res ? Kern<DT, false, false, true>::launch(p, grid, ctx, stream)                   \
                      : Kern<DT, false, false, false>::launch(p, grid, ctx, stream))
        if (dt == FL_F16)
            FL_LAUNCH(DT_F16);
        else
            FL_LAUNCH(DT_BF16);
#undef FL_LAUNCH
        return host::launched(e, "4-bit tile kernel");
    };
    if ((st = launch_tiles(0, plain, p.splits)) != FL_OK || plain == all) return st;
    return launch_tiles(plain, all, tail_splits);
}

}  // namespace fl
