// 4-bit products for nine rows and more, on the tensor cores.
//
// The weight is the M operand: a tile takes 128 rows of each of two weight
// blocks (rows n .. n + 255 of one weight, or, for the SwiGLU pair, rows
// n .. n + 127 of Wg and of Wu) against up to 128 tokens, so that the 4-bit
// codes are expanded where the MMA reads them: in tensor memory. Each K step
// of 64 a dequantising thread owns one weight row: it reads 32 bytes of codes
// from shared memory, forms scale * (code - zero) in the dtype (one rounding)
// and writes its row of the A operand with tcgen05.st; the tokens are the B
// operand, staged by TMA. 16-bit weights exist nowhere else.
//
// Per K step and SM the two MMAs (128 x BT x 64 each) read 2 * BT * 128 bytes
// of shared memory and TMA writes BT * 128 bytes and 8 KB of codes. With few
// tokens the tile is a weight stream: the K range is then split over a cluster
// of up to 8 CTAs, whose fp32 partials are added through distributed shared
// memory in rank order.
//
// Roles: warp 0 TMA producer (codes in stages of 256 k, tokens in stages of
// 64 k), warp 1 tensor memory and MMA issue, warps 2 and 3 load the scales and
// zero points of 1024 k at a time into shared memory (transposed: one row per
// thread there), warps 4-7 and 8-11 dequantise block 0 and block 1 and, when
// the MMAs are done, apply the epilogue.
//
// Every mbarrier wait is bounded as in the other kernels.
#include <atomic>

#include "fl_common.cuh"
#include "fl_host.h"
#include "fl_w4.h"

namespace fl {

namespace {

constexpr int kThreads = 384;
constexpr int kRows = 128;       // weight rows of one block (TMEM lanes)
constexpr int kTok = 128;        // tokens of a tile at most
constexpr int kStep = 64;        // k per B stage and A slot
constexpr int kWk = 256;         // k per code stage
constexpr int kSk = 1024;        // k per scale stage
constexpr int kBStages = 6, kWStages = 2, kSStages = 2, kSlots = 4;
constexpr int kBBytes = kTok * kStep * 2;           // 16 KB
constexpr int kWBytes = kRows * kWk / 2;            // 16 KB, one block
constexpr int kSPitch = 130;                        // 16-bit scales of one group: 128 rows, padded
constexpr int kZPitch = 132;                        // zero-point bytes of one group
constexpr int kSGroups = kSk / 32;
constexpr int kSBytes = kSGroups * kSPitch * 2;     // scales of one block and stage
constexpr int kZBytes = kSGroups * kZPitch;

constexpr int kOffW = kBStages * kBBytes;
constexpr int kOffS = kOffW + kWStages * 2 * kWBytes;
constexpr int kOffZ = kOffS + kSStages * 2 * kSBytes;
constexpr int kOffBar = (kOffZ + kSStages * 2 * kZBytes + 7) / 8 * 8;
constexpr int kBars = 2 * kBStages + 2 * kWStages + 2 * kSlots + 2 * kSStages + 2;
constexpr int kOffSlot = kOffBar + kBars * 8;
constexpr int kSmem = kOffSlot + 16 + 1024;         // + alignment slack
static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
static_assert(kRows * 2 * kTok * 4 <= kOffS, "the partial sums fit in the rings");

constexpr int kACol = 256;  // first tensor-memory column of the A slots (the accumulators: 0 and 128)

struct TileParams {
    CUtensorMap tm_x;     // x [M, K], box {64, BT}
    CUtensorMap tm_q[2];  // codes [N, K / 2] bytes, box {128, 128}
    W4Params w;
    int bt, splits, steps_per_split, steps;  // K steps of 64
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
        out[i] = DTypeOps<DT>::mul2(hfma2<DT>((pair & 0x0078000fu) | kMagic, kUnit, zc), s2);
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

template <int DT, bool DUAL>
__global__ void __launch_bounds__(kThreads, 1) fl_w4_tile_kernel(const __grid_constant__ TileParams p) {
    using Ops = DTypeOps<DT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sbase - raw);
    const W4Params& w = p.w;

    const uint32_t bar0 = sbase + kOffBar;
    auto bfull = [&](int s) { return bar0 + 8u * s; };
    auto bempty = [&](int s) { return bar0 + 8u * (kBStages + s); };
    auto wfull = [&](int s) { return bar0 + 8u * (2 * kBStages + s); };
    auto wempty = [&](int s) { return bar0 + 8u * (2 * kBStages + kWStages + s); };
    auto afull = [&](int s) { return bar0 + 8u * (2 * kBStages + 2 * kWStages + s); };
    auto aempty = [&](int s) { return bar0 + 8u * (2 * kBStages + 2 * kWStages + kSlots + s); };
    auto sfull = [&](int s) { return bar0 + 8u * (2 * kBStages + 2 * kWStages + 2 * kSlots + s); };
    auto sempty = [&](int s) { return bar0 + 8u * (2 * kBStages + 2 * kWStages + 2 * kSlots + kSStages + s); };
    const uint32_t dfull = bar0 + 8u * (kBars - 2), drain = bar0 + 8u * (kBars - 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / p.splits, rank = blockIdx.x % p.splits;
    const int m0 = blockIdx.y * p.bt;
    // first row of each weight block
    const int n0 = tile * (DUAL ? kRows : 2 * kRows);
    const int k0 = rank * p.steps_per_split, k1 = min(p.steps, k0 + p.steps_per_split), nk = k1 - k0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kBStages; ++s) {
            mbar_init(bfull(s), 1);
            mbar_init(bempty(s), 1);
        }
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(wfull(s), 1);
            mbar_init(wempty(s), 8);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(afull(s), 8);
            mbar_init(aempty(s), 1);
        }
        for (int s = 0; s < kSStages; ++s) {
            mbar_init(sfull(s), 2);
            mbar_init(sempty(s), 8);
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
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < kWStages && i * (kWk / kStep) < nk; ++i) {
            tma_prefetch_2d(&p.tm_q[0], k0 * (kStep / 2) + i * (kWk / 2), n0);
            tma_prefetch_2d(&p.tm_q[DUAL], k0 * (kStep / 2) + i * (kWk / 2), DUAL ? n0 : n0 + kRows);
        }
    }
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();

    bool ready = false;  // epilogue warps: the accumulators are complete
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            int bi = 0, wi = 0;  // loads issued
            for (int kb = 0; kb < nk; ++kb) {
                if (kb % (kWk / kStep) == 0) {
                    const int s = wi % kWStages;
                    if (!wait_bar(wempty(s), (uint32_t)((wi / kWStages) & 1) ^ 1u, p.status, p.timeout_ns, 20)) break;
                    mbar_arrive_expect_tx(wfull(s), 2 * kWBytes);
                    const uint32_t dst = sbase + kOffW + s * 2 * kWBytes;
                    const int x = (k0 + kb) * (kStep / 2);
                    tma_load_2d(dst, &p.tm_q[0], wfull(s), x, n0);
                    tma_load_2d(dst + kWBytes, &p.tm_q[DUAL], wfull(s), x, DUAL ? n0 : n0 + kRows);
                    ++wi;
                }
                const int s = bi % kBStages;
                if (!wait_bar(bempty(s), (uint32_t)((bi / kBStages) & 1) ^ 1u, p.status, p.timeout_ns, 21)) break;
                mbar_arrive_expect_tx(bfull(s), (uint32_t)p.bt * (kStep * 2));
                tma_load_2d(sbase + s * kBBytes, &p.tm_x, bfull(s), (k0 + kb) * kStep, m0);
                ++bi;
            }
            // every load this thread issued lands before the CTA may exit
            for (int i = 1; i <= kBStages && i <= bi; ++i)
                wait_bar_drain(bfull((bi - i) % kBStages), (uint32_t)(((bi - i) / kBStages) & 1), 20000000ull);
            for (int i = 1; i <= kWStages && i <= wi; ++i)
                wait_bar_drain(wfull((wi - i) % kWStages), (uint32_t)(((wi - i) / kWStages) & 1), 20000000ull);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_f16(Ops::kFormat, 128, (uint32_t)p.bt);
            bool ok = true;
            for (int kb = 0; kb < nk; ++kb) {
                const int s = kb % kBStages, a = kb % kSlots;
                ok = wait_bar(bfull(s), (uint32_t)((kb / kBStages) & 1), p.status, p.timeout_ns, 22) &&
                     wait_bar(afull(a), (uint32_t)((kb / kSlots) & 1), p.status, p.timeout_ns, 23);
                if (!ok) break;
                tc_fence_after();
                const uint64_t db = sw128_kmajor_desc(sbase + s * kBBytes);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int kk = 0; kk < kStep / 16; ++kk)
                        umma_f16_ts(tmem + 128u * j, tmem + kACol + 64u * a + 32u * j + 8u * kk, db + 2 * kk, idesc,
                                    (kb | kk) != 0);
                umma_commit(bempty(s));
                umma_commit(aempty(a));
            }
            if (ok) umma_commit(dfull);
            // all MMAs issued by this thread complete before tensor memory is released
            umma_commit(drain);
            wait_bar_drain(drain, 0, 20000000ull);
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------ scales and zero points of block j
        const int j = warp - 2, row0 = DUAL ? n0 : n0 + kRows * j;
        const uint16_t* sc = w.scales[DUAL ? j : 0];
        const uint8_t* zp = w.zeros[DUAL ? j : 0];
        const int per_row = w.K / w.group, ng = kSk / w.group;  // groups of a row; of a stage (8, 16 or 32)
        const int sh = 31 - __clz(ng);
        const int stages = (nk * kStep + kSk - 1) / kSk;
        for (int i = 0; i < stages; ++i) {
            const int s = i % kSStages;
            if (!wait_bar(sempty(s), (uint32_t)((i / kSStages) & 1) ^ 1u, p.status, p.timeout_ns, 24)) break;
            const int g0 = (k0 * kStep + i * kSk) / w.group;
            uint16_t* ds = reinterpret_cast<uint16_t*>(smem + kOffS + (s * 2 + j) * kSBytes);
            uint8_t* dz = smem + kOffZ + (s * 2 + j) * kZBytes;
            constexpr int U = 16;
            for (int b = lane; b < kRows << sh; b += 32 * U) {
                uint16_t v[U];
                uint8_t z[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int e = b + 32 * u, r = e >> sh, g = g0 + (e & (ng - 1));
                    const bool in = r < kRows && row0 + r < w.N && g < per_row;
                    v[u] = in ? __ldg(sc + (size_t)(row0 + r) * per_row + g) : (uint16_t)0;
                    z[u] = in && zp != nullptr ? (uint8_t)(__ldg(zp + (size_t)(row0 + r) * per_row + g) & 15) : (uint8_t)8;
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int e = b + 32 * u, r = e >> sh, g = e & (ng - 1);
                    if (r < kRows) {
                        ds[g * kSPitch + r] = v[u];
                        dz[g * kZPitch + r] = z[u];
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(sfull(s));
        }
    } else {
        // ------------------------------------------------------------ dequantise block j, one row per thread
        const int j = (warp - 4) >> 2, row = (threadIdx.x - 128) & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int gsh = 31 - __clz(w.group);
        bool ok = true;
        for (int kb = 0; kb < nk; ++kb) {
            const int wi = kb / (kWk / kStep), ws = wi % kWStages, q = kb % (kWk / kStep);
            const int si = kb / (kSk / kStep), ss = si % kSStages;
            if (q == 0) ok = wait_bar(wfull(ws), (uint32_t)((wi / kWStages) & 1), p.status, p.timeout_ns, 25);
            if (ok && kb % (kSk / kStep) == 0)
                ok = wait_bar(sfull(ss), (uint32_t)((si / kSStages) & 1), p.status, p.timeout_ns, 26);
            if (!ok) break;
            const uint32_t src = sbase + kOffW + (ws * 2 + j) * kWBytes + row * 128;
            const uint4 c0 = ld_shared_v4(src + (((2 * q) ^ (row & 7)) << 4));
            const uint4 c1 = ld_shared_v4(src + (((2 * q + 1) ^ (row & 7)) << 4));
            const uint16_t* ds = reinterpret_cast<const uint16_t*>(smem + kOffS + (ss * 2 + j) * kSBytes);
            const uint8_t* dz = smem + kOffZ + (ss * 2 + j) * kZBytes;
            const int kin = (kb % (kSk / kStep)) * kStep;
            const int ga = kin >> gsh, gb = (kin + 32) >> gsh;
            const uint32_t sa = (uint32_t)ds[ga * kSPitch + row] * 0x10001u, sb = (uint32_t)ds[gb * kSPitch + row] * 0x10001u;
            const uint32_t za = zero_const<DT>(dz[ga * kZPitch + row]), zb = zero_const<DT>(dz[gb * kZPitch + row]);
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
                // the last reads of a stage of codes and of scales
                if (q == kWk / kStep - 1 || kb == nk - 1) mbar_arrive(wempty(ws));
                if (kb % (kSk / kStep) == kSk / kStep - 1 || kb == nk - 1) mbar_arrive(sempty(ss));
            }
            const int a = kb % kSlots;
            ok = wait_bar(aempty(a), (uint32_t)((kb / kSlots) & 1) ^ 1u, p.status, p.timeout_ns, 27);
            if (!ok) break;
            tc_fence_after();
            tmem_st_32x32b_x32(tmem + lanes + kACol + 64u * a + 32u * j, o);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(afull(a));
        }
        ready = ok && wait_bar(dfull, 0, p.status, p.timeout_ns, 28);
        tc_fence_after();
    }

    // ---------------------------------------------------------------- epilogue
    const int jb = (warp - 4) >> 2;  // weight block of an epilogue warp
    const int lrow = (threadIdx.x - 128) & 127;
    const int n = n0 + lrow + (DUAL ? 0 : kRows * jb);
    const uint32_t dcol = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    // out[m][n] of two tokens: lanes n and n + 1 exchange, so that the even
    // lane stores both rows' values of token m, the odd lane those of m + 1
    const float bias = warp >= 4 && !DUAL && w.bias != nullptr && n < w.N ? Ops::unpack(w.bias[n]).x : 0.f;
    auto store2 = [&](int m, float v0, float v1) {
        if constexpr (!DUAL) {
            v0 = act_apply(w.act, v0 + bias);
            v1 = act_apply(w.act, v1 + bias);
        }
        const float give = (lane & 1) ? v0 : v1, got = __shfl_xor_sync(0xffffffffu, give, 1);
        float a = (lane & 1) ? got : v0, b = (lane & 1) ? v1 : got;
        const int mm = m + (lane & 1), nn = n & ~1;
        if (mm >= w.M || mm >= m0 + p.bt || nn >= w.N) return;
        const size_t at = (size_t)mm * w.N + nn;
        if (!DUAL && w.residual != nullptr) {
            const float2 r = Ops::unpack(*reinterpret_cast<const uint32_t*>(w.residual + at));
            a += r.x;
            b += r.y;
        }
        *reinterpret_cast<uint32_t*>(w.out + at) = Ops::pack(a, b);
    };
    if (p.splits == 1) {
        // (the pair's epilogue is shared by token halves: both blocks' accumulators are at the same lanes)
        if (warp >= 4 && __all_sync(0xffffffffu, ready)) {
            const int chunks = (p.bt + 31) / 32;
            for (int c = DUAL ? jb : 0; c < chunks; c += DUAL ? 2 : 1) {
                uint32_t g[32];
                tmem_ld_32x32b_x32(dcol + (DUAL ? 0u : 128u * jb) + 32u * c, g);
                if constexpr (DUAL) {
                    uint32_t u[32];
                    tmem_ld_32x32b_x32(dcol + 128u + 32u * c, u);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        g[e] = __float_as_uint(act_apply(ACT_SILU, __uint_as_float(g[e])) * __uint_as_float(u[e]));
                } else {
                    tmem_ld_wait();
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    store2(m0 + 32 * c + e, __uint_as_float(g[e]), __uint_as_float(g[e + 1]));
            }
        }
    } else {
        // partial sums into this CTA's shared memory: [block][token][row]
        float* part = reinterpret_cast<float*>(smem);
        if (warp >= 4 && __all_sync(0xffffffffu, ready)) {
            for (int c = 0; c < (p.bt + 31) / 32; ++c) {
                uint32_t g[32];
                tmem_ld_32x32b_x32(dcol + 128u * jb + 32u * c, g);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (32 * c + e < p.bt) part[(jb * p.bt + 32 * c + e) * kRows + lrow] = __uint_as_float(g[e]);
            }
        }
        __syncwarp();
        cluster_barrier_sync();
        // each rank finishes its range of tokens
        if (warp >= 4) {
            const int per = ((p.bt + p.splits - 1) / p.splits + 1) & ~1;
            const int t1 = min(p.bt, (rank + 1) * per);
            auto sum = [&](int j, int t) {
                const uint32_t a = sbase + (uint32_t)((j * p.bt + t) * kRows + lrow) * 4u;
                float v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < p.splits) v[r] = ld_cluster_f32(mapa_cluster(a, (uint32_t)r));
                float s = v[0];
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < p.splits) s += v[r];
                return s;
            };
            for (int t = rank * per + (DUAL ? 2 * jb : 0); t < t1; t += DUAL ? 4 : 2) {
                const int tb = t + 1 < p.bt ? t + 1 : t;
                float v0 = sum(DUAL ? 0 : jb, t), v1 = sum(DUAL ? 0 : jb, tb);
                if constexpr (DUAL) {
                    v0 = act_apply(ACT_SILU, v0) * sum(1, t);
                    v1 = act_apply(ACT_SILU, v1) * sum(1, tb);
                }
                store2(m0 + t, v0, v1);
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
    const int token_tiles = (w.M + kTok - 1) / kTok;
    p.bt = ((w.M + token_tiles - 1) / token_tiles + 15) / 16 * 16;
    const int row_tiles = dual ? (w.N + kRows - 1) / kRows : (w.N + 2 * kRows - 1) / (2 * kRows);
    const long long tiles = (long long)row_tiles * token_tiles;
    p.steps = (w.K + kStep - 1) / kStep;
    // K split over a cluster when the tiles leave SMs idle: the least time, in
    // units of one unsplit tile, of whole waves of resident clusters. Ranges
    // are whole multiples of 128 k, the largest group.
    static std::atomic<int> resident[9];
    int best = 1;
    double least = 0;
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
        const double cost = (double)((tiles + n - 1) / n) * (per / (double)p.steps + (s > 1 ? 0.02 : 0.0));
        if (s == 1 || cost < least) best = s, least = cost;
    }
    p.splits = best;
    p.steps_per_split = ((p.steps + 1) / 2 + best - 1) / best * 2;
    fl_status st;
    if ((st = host::encode_matrix(&p.tm_x, dt, 2, w.x, w.K, w.M, kStep, p.bt)) != FL_OK) return st;
    if ((st = host::encode_matrix(&p.tm_q[0], dt, 1, w.q[0], w.K / 2, w.N, kWk / 2, kRows)) != FL_OK) return st;
    if (dual && (st = host::encode_matrix(&p.tm_q[1], dt, 1, w.q[1], w.K / 2, w.N, kWk / 2, kRows)) != FL_OK) return st;
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
