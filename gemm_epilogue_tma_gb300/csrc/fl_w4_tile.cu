// 4-bit products for nine rows and more, on the tensor cores.
//
// The weight is the M operand: a tile takes 128 weight rows (or, for the
// SwiGLU pair, 64 rows of Wg and the same rows of Wu) against up to 256 tokens,
// so that the 4-bit codes are expanded where the MMA reads them: in tensor
// memory. Each K step of 64 a dequantising thread owns one weight row: it reads
// 32 bytes of codes from shared memory, forms scale * (code - zero) in the
// dtype (one rounding) and writes its row of the A operand with tcgen05.st; the
// tokens are the B operand, staged by TMA. 16-bit weights exist nowhere else.
//
// What bounds it: with many tokens the shared-memory traffic of the B operand
// (per K step 256 * 128 bytes written by TMA and read by the MMA, against 590
// cycles of MMA); with few the weight stream, for which the K range is split over a
// cluster of up to 8 CTAs whose fp32 partials are added through distributed
// shared memory in rank order. A tile of two blocks of 128 rows by 128 tokens
// moved fewer bytes per MMA but expanded every code for half as many tokens, and the
// expansion (about 440 instructions a warp and step) set its pace: 237 us at
// 4096^3.
//
// Roles: warp 0 loads the tokens by TMA (stages of 64 k), warp 1 owns tensor
// memory and issues the MMAs, warps 2 and 3 load the scales and zero points of
// 1024 k at a time into shared memory (transposed: one row per thread there; the
// first of them is loaded by the dequantising warps, which have nothing else to
// do yet), warps 4-19 dequantise, four to a K step, and when the MMAs are done
// apply the epilogue, warp 20 loads the codes by TMA (stages of 256 k). Codes
// and tokens have producers of their own, so that the codes, which come from
// HBM and are needed first, run ahead as far as their ring reaches; the fewer
// the tokens, the more of shared memory is the codes'. A stage of tokens and the A
// slot of the same step share one full and one empty barrier (the bytes and
// the four warps' arrivals on the one, the MMA's commit on the other): the single
// issuing thread competes with four dequantising warps for its scheduler, and a
// step with two waits and two commits took it 680 to 850 cycles whatever the
// tile's width.
//
// Every mbarrier wait is bounded as in the other kernels.
#include <atomic>

#include "fl_common.cuh"
#include "fl_host.h"
#include "fl_w4.h"

namespace fl {

namespace {

constexpr int kThreads = 672;
constexpr int kRows = 128;       // weight rows of a tile (TMEM lanes)
constexpr int kTok = 256;        // tokens of a tile at most
constexpr int kStep = 64;        // k per B stage and A slot
constexpr int kGroups = 4;       // dequantising warpgroups: K step kb goes to kb % 4
constexpr int kWk = kGroups * kStep;  // k per code stage: one step of each warpgroup
constexpr int kSIter = 4;        // code stages per scale stage
constexpr int kSk = kSIter * kWk;
constexpr int kStages = 2 * kGroups, kWStages = 8, kSStages = 2;  // (at most; stages of tokens: 4 or 8)
constexpr int kRing = 192 * 1024;                   // both rings
constexpr int kWBytes = kRows * kWk / 2;            // 16 KB
constexpr int kSPitch = 130;                        // 16-bit scales of one group: 128 rows, padded
constexpr int kZPitch = 132;                        // zero-point bytes of one group
constexpr int kSGroups = kSk / 32;
constexpr int kSBytes = kSGroups * kSPitch * 2;
constexpr int kZBytes = kSGroups * kZPitch;

constexpr int kOffS = kRing;
constexpr int kOffZ = kOffS + kSStages * kSBytes;
constexpr int kOffBar = (kOffZ + kSStages * kZBytes + 7) / 8 * 8;
constexpr int kBars = 2 * kStages + 2 * kWStages + 2 * kSStages + 2;
constexpr int kOffSlot = kOffBar + kBars * 8;
constexpr int kSmem = kOffSlot + 16 + 1024;         // + alignment slack
static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
static_assert(kRows * kTok * 4 <= kRing, "the partial sums fit in the rings");

constexpr int kACol = 256;  // first tensor-memory column of the A slots (the accumulator: 0 .. 255)

struct TileParams {
    CUtensorMap tm_x;     // x [M, K], box {64, BT}
    CUtensorMap tm_q[2];  // codes [N, K / 2] bytes, box {128, 128} (pair: {128, 64} each)
    W4Params w;
    int bt, splits, steps_per_split, steps;  // K steps of 64
    int stages, w_stages, b_bytes;           // rings: stages * b_bytes of tokens, then the code stages
    int* status;
    unsigned long long timeout_ns;
};

template <int DT>
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    if constexpr (DT == DT_F16)
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    else
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// Eight codes of a word, in order, as four pairs scale * (code - zero). The
// code goes into the mantissa of a power of two B (128 bf16, 1024 fp16): the
// even one as B + c, the odd one, taken from the word shifted by one, as
// B + 8 c, and one FMA with (1, 1/8) and (-(B + z), -(B/8 + z)) leaves c - z,
// exactly. The product with the scale is the one rounding.
template <int DT>
__device__ __forceinline__ void dequant8(uint32_t w, uint32_t s2, uint32_t zc, uint32_t* out) {
    constexpr uint32_t kMagic = DT == DT_F16 ? 0x64006400u : 0x43004300u;
    constexpr uint32_t kUnit = DT == DT_F16 ? 0x30003c00u : 0x3e003f80u;  // (1, 1/8)
    const uint32_t v = w >> 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = __byte_perm(w, v, (uint32_t)(i * 0x1111 + 0x4400));  // bytes w.i, w.i, v.i, v.i
        out[i] = DTypeOps<DT>::mul2(hfma2<DT>(and_or(pair, 0x0078000fu, kMagic), kUnit, zc), s2);
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
// from; under a divergent `lane == 0` each MMA waits for its operands to be moved there.
__device__ __forceinline__ void mma_step(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 r, a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
        "elect.sync r|p, 0xffffffff;\n\t"
        "setp.ne.b32 q, %4, 0;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
        "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t"
        "setp.eq.u32 q, 0, 0;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, q;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void commit_elected(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 r;\n\telect.sync r|p, 0xffffffff;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

template <int DT, bool DUAL>
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
    const uint32_t dfull = bar0 + 8u * (kBars - 2), drain = bar0 + 8u * (kBars - 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / p.splits, rank = blockIdx.x % p.splits;
    const int m0 = blockIdx.y * p.bt;
    const int n0 = tile * (DUAL ? kRows / 2 : kRows);  // first weight row (of each weight of the pair)
    const int k0 = rank * p.steps_per_split, k1 = min(p.steps, k0 + p.steps_per_split), nk = k1 - k0;
    const int nb = p.stages, nw = p.w_stages;
    const uint32_t wring = sbase + (uint32_t)(nb * p.b_bytes);
    // weight and row of TMEM lane r: for the pair, each warp's lanes 0-15 are
    // rows of Wg and 16-31 the same rows of Wu
    auto weight_of = [&](int r) { return DUAL ? (r >> 4) & 1 : 0; };
    auto row_of = [&](int r) { return n0 + (DUAL ? (r >> 5) * 16 + (r & 15) : r); };

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
    if (warp == 20 && lane == 0) {
        for (int i = 0; i < nw && i * kGroups < nk; ++i)
            for (int j = 0; j <= (DUAL ? 1 : 0); ++j)
                tma_prefetch_2d(&p.tm_q[j], k0 * (kStep / 2) + i * (kWk / 2), n0);
    }
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();

    // Scales and zero points of scale stage i into shared memory, by `count`
    // threads: neighbouring threads take neighbouring groups of a row.
    const int s_count = (nk * kStep + kSk - 1) / kSk;
    auto load_scales = [&](int i, int tid, int count) {
        const int per_row = w.K / w.group, ng = kSk / w.group, sh = 31 - __clz(ng);  // groups of a row; of a stage (8, 16, 32)
        const int g0 = (k0 * kStep + i * kSk) / w.group, g_end = min(per_row, (k1 * kStep + w.group - 1) / w.group);
        uint16_t* ds = reinterpret_cast<uint16_t*>(smem + kOffS + (i % kSStages) * kSBytes);
        uint8_t* dz = smem + kOffZ + (i % kSStages) * kZBytes;
        const bool zeros = w.zeros[0] != nullptr;
        constexpr int U = 8;  // loads in flight per thread
        for (int b = tid; b < kRows << sh; b += count * U) {
            uint16_t v[U];
            uint8_t z[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = b + count * u, r = e >> sh, g = g0 + (e & (ng - 1)), n = row_of(r);
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

    bool ready = false;  // epilogue warps: the accumulator is complete
    if (warp == 0) {
        // ------------------------------------------------------------ tokens
        if (lane == 0) {
            int issued = 0, s = 0;
            uint32_t ph = 0;
            for (int kb = 0; kb < nk; ++kb) {
                if (!wait_bar(empty(s), ph ^ 1u, p.status, p.timeout_ns, 21)) break;
                mbar_arrive_expect_tx(full(s), (uint32_t)p.b_bytes);
                tma_load_2d(sbase + s * p.b_bytes, &p.tm_x, full(s), (k0 + kb) * kStep, m0);
                ++issued;
                if (++s == nb) s = 0, ph ^= 1u;
            }
            // every load this thread issued lands before the CTA may exit
            for (int i = 1; i <= nb && i <= issued; ++i)
                wait_bar_drain(full((issued - i) % nb), (uint32_t)(((issued - i) / nb) & 1), 20000000ull);
        }
    } else if (warp == 20) {
        // ------------------------------------------------------------ codes
        if (lane == 0) {
            int issued = 0, s = 0;
            uint32_t ph = 0;
            for (int kb = 0; kb < nk; kb += kGroups) {
                if (!wait_bar(wempty(s), ph ^ 1u, p.status, p.timeout_ns, 20)) break;
                mbar_arrive_expect_tx(wfull(s), kWBytes);
                const uint32_t dst = wring + s * kWBytes;
                const int x = (k0 + kb) * (kStep / 2);
                tma_load_2d(dst, &p.tm_q[0], wfull(s), x, n0);
                if (DUAL) tma_load_2d(dst + kWBytes / 2, &p.tm_q[1], wfull(s), x, n0);
                ++issued;
                if (++s == nw) s = 0, ph ^= 1u;
            }
            for (int i = 1; i <= nw && i <= issued; ++i)
                wait_bar_drain(wfull((issued - i) % nw), (uint32_t)(((issued - i) / nw) & 1), 20000000ull);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (the whole warp, converged)
        const uint32_t idesc = umma_idesc_f16(Ops::kFormat, 128, (uint32_t)p.bt);
        bool ok = true;
        uint32_t ph = 0;
        for (int kb = 0, s = 0; kb < nk; ++kb) {
            ok = __all_sync(0xffffffffu, wait_bar(full(s), ph, p.status, p.timeout_ns, 22));
            if (!ok) break;
            tc_fence_after();
            mma_step(tmem, tmem + kACol + 32u * s, sw128_kmajor_desc(sbase + s * p.b_bytes), idesc, kb, empty(s));
            if (++s == nb) s = 0, ph ^= 1u;
        }
        if (ok) commit_elected(dfull);
        // all MMAs issued by this warp complete before tensor memory is released
        commit_elected(drain);
        wait_bar_drain(drain, 0, 20000000ull);
    } else if (warp < 4) {
        // ------------------------------------------------------------ scales and zero points of the later stages
        for (int i = 1; i < s_count; ++i) {
            const int s = i % kSStages;
            if (!wait_bar(sempty(s), (uint32_t)((i / kSStages) & 1) ^ 1u, p.status, p.timeout_ns, 24)) break;
            load_scales(i, threadIdx.x - 64, 64);
            __syncwarp();
            if (lane == 0) mbar_arrive(sfull(s));
        }
    } else {
        // ------------------------------------------------------------ dequantise, one row per thread
        const int grp = (warp - 4) >> 2, r = (threadIdx.x - 128) & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int gsh = 31 - __clz(w.group);
        // this row's codes of the warpgroup's K step in a code stage
        const int srow = DUAL ? weight_of(r) * (kRows / 2) + (r >> 5) * 16 + (r & 15) : r;
        const uint32_t src0 = wring + srow * 128 + (((2 * grp) ^ (srow & 7)) << 4);
        const uint32_t src1 = wring + srow * 128 + (((2 * grp + 1) ^ (srow & 7)) << 4);
        load_scales(0, threadIdx.x - 128, 512);
        named_bar_sync(1, 512);
        bool ok = true;
        int ws = 0, a = grp;
        uint32_t wph = 0, ph = 0;
        for (int it = 0, kb = grp; kb < nk; ++it, kb += kGroups) {
            const int ss = it / kSIter % kSStages;
            ok = wait_bar(wfull(ws), wph, p.status, p.timeout_ns, 25);
            if (ok && it % kSIter == 0 && it > 0) {
                // (stage 0's barrier has seen no phase for the first 1024 k)
                const int i = it / kSIter, phases = i / kSStages - (ss == 0 ? 1 : 0);
                ok = wait_bar(sfull(ss), (uint32_t)(phases & 1), p.status, p.timeout_ns, 26);
            }
            if (!ok) break;
            const uint4 c0 = ld_shared_v4(src0 + ws * kWBytes), c1 = ld_shared_v4(src1 + ws * kWBytes);
            const uint16_t* ds = reinterpret_cast<const uint16_t*>(smem + kOffS + ss * kSBytes);
            const uint8_t* dz = smem + kOffZ + ss * kZBytes;
            const int kin = (it % kSIter) * kWk + grp * kStep;
            const int ga = kin >> gsh, gb = (kin + 32) >> gsh;
            const uint32_t sa = (uint32_t)ds[ga * kSPitch + r] * 0x10001u, sb = (uint32_t)ds[gb * kSPitch + r] * 0x10001u;
            const uint32_t za = zero_const<DT>(dz[ga * kZPitch + r]), zb = zero_const<DT>(dz[gb * kZPitch + r]);
            uint32_t o[32];
            dequant8<DT>(c0.x, sa, za, o);
            dequant8<DT>(c0.y, sa, za, o + 4);
            dequant8<DT>(c0.z, sa, za, o + 8);
            dequant8<DT>(c0.w, sa, za, o + 12);
            dequant8<DT>(c1.x, sb, zb, o + 16);
            dequant8<DT>(c1.y, sb, zb, o + 20);
            dequant8<DT>(c1.z, sb, zb, o + 24);
            dequant8<DT>(c1.w, sb, zb, o + 28);
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(wempty(ws));
                if (it % kSIter == kSIter - 1) mbar_arrive(sempty(ss));
            }
            if (++ws == nw) ws = 0, wph ^= 1u;
            ok = wait_bar(empty(a), ph ^ 1u, p.status, p.timeout_ns, 27);
            if (!ok) break;
            tc_fence_after();
            tmem_st_32x32b_x32(tmem + lanes + kACol + 32u * a, o);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(full(a));
            if ((a += kGroups) >= nb) a = grp, ph ^= 1u;
        }
        ready = ok && wait_bar(dfull, 0, p.status, p.timeout_ns, 28);
        tc_fence_after();
    }

    // ---------------------------------------------------------------- epilogue
    const bool epi = warp >= 4 && warp < 20;
    const int grp = (warp - 4) >> 2, r = (threadIdx.x - 128) & 127;
    const uint32_t dcol = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int n = row_of(r), nn = n & ~1;
    const float bias = epi && !DUAL && w.bias != nullptr && n < w.N ? Ops::unpack(w.bias[n]).x : 0.f;
    // two neighbouring outputs of token m
    auto store = [&](int m, float a, float b) {
        if (m >= w.M || m >= m0 + p.bt || nn >= w.N) return;
        const size_t at = (size_t)m * w.N + nn;
        if (!DUAL && w.residual != nullptr) {
            const float2 x = Ops::unpack(*reinterpret_cast<const uint32_t*>(w.residual + at));
            a += x.x;
            b += x.y;
        }
        *reinterpret_cast<uint32_t*>(w.out + at) = Ops::pack(a, b);
    };
    // of two values, the one for the even lane stays there, the other goes over: lane pairs then hold
    // neighbouring outputs, of the first value's token in the even lane and the second's in the odd one
    auto pair = [&](float v0, float v1, float& a, float& b) {
        const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v0 : v1, 1);
        a = (lane & 1) ? got : v0;
        b = (lane & 1) ? v1 : got;
    };
    // accumulators of tokens m .. m + 3 at this lane's row
    auto emit4 = [&](int m, float v0, float v1, float v2, float v3) {
        float a, b;
        if constexpr (DUAL) {
            // lanes 16 apart hold the gate and the up value: the gate's lane takes tokens m and m + 2, the up's m + 1 and m + 3
            const bool up = lane & 16;
            const float o0 = __shfl_xor_sync(0xffffffffu, up ? v0 : v1, 16), o1 = __shfl_xor_sync(0xffffffffu, up ? v2 : v3, 16);
            const float h0 = act_apply(ACT_SILU, up ? o0 : v0) * (up ? v1 : o0);
            const float h1 = act_apply(ACT_SILU, up ? o1 : v2) * (up ? v3 : o1);
            pair(h0, h1, a, b);
            store(m + (up ? 1 : 0) + ((lane & 1) ? 2 : 0), a, b);
        } else {
            pair(act_apply(w.act, v0 + bias), act_apply(w.act, v1 + bias), a, b);
            store(m + (lane & 1), a, b);
            pair(act_apply(w.act, v2 + bias), act_apply(w.act, v3 + bias), a, b);
            store(m + 2 + (lane & 1), a, b);
        }
    };
    if (p.splits == 1) {
        if (epi && __all_sync(0xffffffffu, ready)) {
            for (int c = grp; c < (p.bt + 31) / 32; c += kGroups) {
                uint32_t g[32];
                tmem_ld_32x32b_x32(dcol + 32u * c, g);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    emit4(m0 + 32 * c + e, __uint_as_float(g[e]), __uint_as_float(g[e + 1]), __uint_as_float(g[e + 2]),
                          __uint_as_float(g[e + 3]));
            }
        }
    } else {
        // partial sums into this CTA's shared memory: [token][row]
        float* part = reinterpret_cast<float*>(smem);
        if (epi && __all_sync(0xffffffffu, ready)) {
            for (int c = grp; c < (p.bt + 31) / 32; c += kGroups) {
                uint32_t g[32];
                tmem_ld_32x32b_x32(dcol + 32u * c, g);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (32 * c + e < p.bt) part[(32 * c + e) * kRows + r] = __uint_as_float(g[e]);
            }
        }
        __syncwarp();
        cluster_barrier_sync();
        // each rank finishes its range of tokens
        if (epi) {
            const int per = ((p.bt + p.splits - 1) / p.splits + 3) & ~3;
            const int t1 = min(p.bt, (rank + 1) * per);
            for (int t = rank * per + 4 * grp; t < t1; t += 4 * kGroups) {
                float v[4][8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (i >= p.splits) break;
                    const uint32_t a = mapa_cluster(sbase + (uint32_t)(t * kRows + r) * 4u, (uint32_t)i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e][i] = ld_cluster_f32(a + e * kRows * 4);
                }
#pragma unroll
                for (int i = 1; i < 8; ++i)
                    if (i < p.splits)
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e][0] += v[e][i];
                emit4(m0 + t, v[0][0], v[1][0], v[2][0], v[3][0]);
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
}

template <int DT, bool DUAL>
struct Kern {
    static cudaError_t configure() {
        static const cudaError_t e = [] {
            auto k = fl_w4_tile_kernel<DT, DUAL>;
            cudaError_t r = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
            return r;
        }();
        return e;
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
    static cudaError_t launch(const TileParams& p, dim3 grid, int pdl, cudaStream_t s) {
        cudaError_t e = configure();
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute a[2];
        config(cfg, a, grid, p.splits, pdl, s);
        return cudaLaunchKernelEx(&cfg, fl_w4_tile_kernel<DT, DUAL>, p);
    }
    // clusters of `splits` CTAs that are resident at once
    static int resident(int splits) {
        if (configure() != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute a[2];
        config(cfg, a, dim3((unsigned)splits), splits, 0, nullptr);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, fl_w4_tile_kernel<DT, DUAL>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        return n;
    }
};

}  // namespace

fl_status w4_tile(int dt, bool dual, const W4Params& w, const host::LaunchContext& ctx, cudaStream_t stream) {
    TileParams p;
    p.steps = (w.K + kStep - 1) / kStep;
    const int rows = dual ? kRows / 2 : kRows, row_tiles = (w.N + rows - 1) / rows;
    // Tokens of a tile and K split: the least time of whole waves of resident
    // clusters. A K step costs the MMA and its shared-memory traffic (2.7
    // cycles a token) or the expansion of its codes (about 300), whichever is
    // more; a split adds the exchange of the partial sums. Ranges of a split
    // are multiples of 128 k, the largest group.
    static std::atomic<int> resident[9];
    double least = 0;
    const int tt0 = (w.M + kTok - 1) / kTok;
    int token_tiles = 0;
    for (int tt = tt0; tt <= tt0 + 2 && tt <= w.M; ++tt) {
        const int bt = ((w.M + tt - 1) / tt + 15) / 16 * 16;
        for (int s = 1; s <= 8; ++s) {
            const int per = ((p.steps + 1) / 2 + s - 1) / s * 2;
            if (s > 1 && (per < 4 || (p.steps + per - 1) / per != s)) continue;
            int n = resident[s].load();
            if (n == 0) {
                n = Kern<DT_BF16, false>::resident(s);
                if (n <= 0) n = -1;
                resident[s] = n;
            }
            if (n < 0) continue;
            const long long waves = ((long long)row_tiles * tt + n - 1) / n;
            const double step = 2.7 * bt > 300.0 ? 2.7 * bt : 300.0;
            const double cost = (double)waves * (step * per + 4000.0 + (s > 1 ? 1500.0 + 12.0 * bt : 0.0));
            if (token_tiles == 0 || cost < least) {
                least = cost;
                token_tiles = tt;
                p.bt = bt;
                p.splits = s;
                p.steps_per_split = per;
            }
        }
    }
    if (token_tiles == 0) return host::fail(FL_ERR_CUDA, "4-bit tile kernel: no resident CTA");
    // rings: eight stages of tokens where they leave half of shared memory to the codes, else four
    p.b_bytes = p.bt * kStep * 2;
    p.stages = 2 * kGroups * p.b_bytes <= kRing / 2 ? 2 * kGroups : kGroups;
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
    const dim3 grid((unsigned)(row_tiles * p.splits), (unsigned)token_tiles);
    cudaError_t e;
    if (dt == FL_F16)
        e = dual ? Kern<DT_F16, true>::launch(p, grid, ctx.pdl, stream) : Kern<DT_F16, false>::launch(p, grid, ctx.pdl, stream);
    else
        e = dual ? Kern<DT_BF16, true>::launch(p, grid, ctx.pdl, stream) : Kern<DT_BF16, false>::launch(p, grid, ctx.pdl, stream);
    return host::launched(e, "4-bit tile kernel");
}

}  // namespace fl
