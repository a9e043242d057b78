// Attention of a prompt's rows over 16-bit keys and values (fl_attention).
//
//   out[i, h] = sum_j p_j v[j] / sum_j p_j,  p_j = 2^(c s_j - m),  s_j = q[i, h] . k[j],  c = scale log2(e)
//
// over the keys j that row i of its sequence sees, all of them or, causal, those up
// to i + len_k - len_q. One pass over the keys with a running maximum m and sum;
// scores and p never leave the multiprocessor.
//
// A CTA takes 256 rows of one sequence and head, as two tiles of 128 rows, over all
// keys in blocks of 128. Both products are tcgen05 MMAs: S = Q K^T from shared
// memory into tensor memory; p replaces S there, in 16 bits, and is the A
// operand of O += P V, whose B operand is the value block as it lies in memory
// (keys along its rows: an MN-major operand, so nothing is transposed). Tensor memory
// holds S and O of both tiles, all 512 columns. Two softmax warpgroups, one per tile and one
// thread per row, work while the tensor core has the other tile's products.
//
// The maximum is moved only when a score passes it by 2^8, since only then is O
// multiplied, in tensor memory, by the softmax warps themselves: p is at most
// 2^8 otherwise, which fp32 sums and 16-bit p do not mind. Rounded are p (to the dtype)
// and the output.
//
// Blocks that some row does not see as a whole are masked score by score. A value
// that a row may not see must not reach it times zero (0 inf, 0 NaN): two warps
// zero the rows behind the last key in such blocks, take what is not finite out
// of the others and note the first key of each channel where it stood, and the
// epilogue adds it to the rows that see that key. (Blocks that every row sees are taken as they are: an infinity
// times a weight that rounds to 0 is a NaN there.)
//
// What bounds it: the products. A block of both tiles takes 1.4 to 1.5 us, the products
// alone 1.36 at the dense rate that was measured for a large library product. 32 and 8 heads of 128,
// bf16, across boxes: one causal sequence of 8192 rows 353 to 376 us (1460 to 1557 TFLOP/s), 4096 106
// (1290); 16384 rows of 16 heads 653 to 657 (1674 to 1685). Heads of 64 channels have half the
// products for the same softmax: 8192 rows 290 us (949). A
// CTA's start (its rows found, the first loads and scores: 2.9 us) and end (output: 2.5)
// are not hidden, since a multiprocessor holds one, so that short
// sequences fare worse (eight of 512 rows: 41.9 us, 411 TFLOP/s; five chunks of 330 to
// 490 rows over 480 to 1930 keys: 53 us, 724). (CTAs that stay and take the next
// rows while the last are finished were no faster: the softmax warps store the output.) Two tiles to a CTA, not one,
// so that each block of keys is read for 256 rows.
//
// Few rows over many keys: a cluster of up to 8 CTAs takes the same rows, each a run of
// the blocks, and adds the parts through distributed shared memory, in order, each CTA
// for its share of the rows (one row over 4096 keys 44 -> 17 us, 16 over 30000 291 -> 80).
//
// Every mbarrier wait is bounded as in the other kernels.
#include <algorithm>
#include <climits>

#include <type_traits>

#include "fl_attn_mma.cuh"
#include "fl_host.h"
#include "fl_quant.cuh"

namespace fl {

namespace {

constexpr int kRows = 128;               // rows of a tile, keys of a block
constexpr int kThreads = 384;            // 8 softmax warps, MMA, TMA, 2 for values
constexpr int kWarpMma = 8, kWarpTma = 9, kWarpFix = 10;
constexpr float kLazy = 8.f, kLarge = 0x1p20f;
constexpr unsigned long long kBlockNs = 20000;  // that a block of keys takes at most where others use the GPU too
constexpr int kOCol = 256;               // tensor-memory columns: S of tile i at 128 i, O at 256 + 128 i

struct AttnParams {
    CUtensorMap tm_q, tm_k, tm_v;
    uint16_t* out;
    long long o_row, o_head;
    const int* cu_q;
    const int* cu_k;
    int rows_q, rows_k, heads_q, group, head_dim, n_seqs, causal;
    int splits;  // CTAs of a cluster
    float c;  // scale * log2(e)
    int* status;
    unsigned long long timeout_ns;
};

template <int DP>
struct Layout {
    static constexpr int kBlock = kRows * DP * 2;   // a tile of q, a block of k or v
    static constexpr int kSlots = DP == 128 ? 4 : 8;  // blocks of k and v in turn
    static constexpr int kOffRing = 2 * kBlock;
    static constexpr int kOffNote = kOffRing + kSlots * kBlock;  // [3][DP] first keys of NaN, inf, -inf; [1] whether any
    static constexpr int kOffBar = kOffNote + (3 * DP + 4) * 4;
    static constexpr int kBars = 2 + 4 * kSlots + 2 + 2 + 2 + 2;
    static constexpr int kOffSlot = kOffBar + kBars * 8;
    static constexpr int kSmem = kOffSlot + 16 + 1024;
    // parts of a cluster, in place of q, k and v: [256][kPitch] sums, [256] maxima and sums of weights
    static constexpr int kPitch = DP + 4;
    static constexpr int kOffMl = 2 * kRows * kPitch * 4;
    static_assert(kOffMl + 2 * kRows * 8 <= kOffNote, "parts");
};

// Takes what is not finite out of eight values at addr, channels ch .. of a key, and
// notes the first key of each channel: NaN, inf and -inf apart.
template <int DT, int DP>
__device__ __forceinline__ void take_out(uint32_t addr, int ch, int key, int* note) {
    constexpr uint32_t kInf = Bits16<DT>::kInf;
    const uint4 x = ld_shared_v4(addr);
    if (absmax_halves<DT>(absmax8<DT>(x)) < kInf) return;
    note[3 * DP] = 1;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr + 2 * i) : "memory");
        if ((v & kInf) != kInf) continue;
        atomicMin(&note[((v & 0x7fffu) != kInf ? 0 : v >> 15 ? 2 : 1) * DP + ch + i], key);
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr + 2 * i), "h"((uint16_t)0) : "memory");
    }
}
// What was taken out, back to a row that sees keys up to `last`: channels ch .. of its output.
template <int DT, int DP>
__device__ __forceinline__ uint4 put_back(const uint4& v, int ch, int last, const int* note) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const float inf = __int_as_float(0x7f800000);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f = DTypeOps<DT>::unpack(w[i]);
        float* const y[2] = {&f.x, &f.y};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = ch + 2 * i + e;
            if (note[c] <= last) *y[e] += __int_as_float(0x7fffffff);
            if (note[DP + c] <= last) *y[e] += inf;
            if (note[2 * DP + c] <= last) *y[e] -= inf;
        }
        w[i] = DTypeOps<DT>::pack(f.x, f.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// DP: head_dim rounded up to 64 or 128.
template <int DT, int DP>
__global__ void __launch_bounds__(kThreads, 1) fl_attention_kernel(const __grid_constant__ AttnParams p) {
    using Ops = DTypeOps<DT>;
    using Lay = Layout<DP>;
    constexpr int NS = Lay::kSlots, CH = DP / 64;  // CH: 64-channel chunks of a block
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sbase - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar0 = sbase + Lay::kOffBar;
    auto q_full = [&](int i) { return bar0 + 8u * i; };
    auto full = [&](int s) { return bar0 + 8u * (2 + s); };
    auto empty = [&](int s) { return bar0 + 8u * (2 + NS + s); };
    auto s_full = [&](int i) { return bar0 + 8u * (2 + 2 * NS + i); };
    auto p_full = [&](int i) { return bar0 + 8u * (4 + 2 * NS + i); };
    auto o_full = [&](int i) { return bar0 + 8u * (6 + 2 * NS + i); };
    auto v_ready = [&](int s) { return bar0 + 8u * (8 + 2 * NS + s); };
    auto v_raw = [&](int s) { return bar0 + 8u * (8 + 3 * NS + s); };
    const uint32_t fixed = bar0 + 8u * (8 + 4 * NS), drain = fixed + 8u;
    int* const note = reinterpret_cast<int*>(smem + Lay::kOffNote);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full(i), 1);
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), 4);
            mbar_init(o_full(i), 1);
        }
        for (int s = 0; s < NS; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
            mbar_init(v_ready(s), 2);
            mbar_init(v_raw(s), 1);
        }
        mbar_init(fixed, 2);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 3 * DP + 1; i += kThreads) note[i] = i < 3 * DP ? INT_MAX : 0;
    if (warp == kWarpMma) {
        tmem_alloc(sbase + Lay::kOffSlot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    auto release = [&] {
        if (warp == kWarpMma) tmem_dealloc(0u, 512);
    };

    // ------------------------------------------------------------ the CTA's rows
    // (tiles counted from the last: causal rows that see the most keys come first)
    const int rank = p.splits > 1 ? (int)cluster_rank() : 0, work = blockIdx.x / p.splits;
    const int head = work % p.heads_q, index = work / p.heads_q;
    int q0 = 0, lq = p.rows_q, k0 = 0, lk = p.rows_k, row0;  // the sequence; this CTA's first row in it
    if (p.cu_q == nullptr) {
        row0 = ((lq + 2 * kRows - 1) / (2 * kRows) - 1 - index) * (2 * kRows);
        if (row0 < 0) return release();
    } else {
        // every warp finds it for itself, 32 sequences at a time from the last
        int left = index, found = -1, n = 0, first = 0;
        for (int e = p.n_seqs; e > 0 && found < 0; e -= 32) {
            const int b = e - 1 - lane;
            int a = 0, z = 0, ka = 0, kz = 0;
            if (b >= 0) {
                a = max(0, min(__ldg(p.cu_q + b), p.rows_q));
                z = max(a, min(__ldg(p.cu_q + b + 1), p.rows_q));
                ka = max(0, min(__ldg(p.cu_k + b), p.rows_k));
                kz = max(ka, min(__ldg(p.cu_k + b + 1), p.rows_k));
            }
            const int tiles = (z - a + 2 * kRows - 1) / (2 * kRows);
            int up = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up += x;
            }
            const uint32_t m = __ballot_sync(0xffffffffu, left < up);
            if (m != 0) {
                const int l = __ffs(m) - 1;
                found = e - 1 - l;
                q0 = __shfl_sync(0xffffffffu, a, l);
                lq = __shfl_sync(0xffffffffu, z, l) - q0;
                k0 = __shfl_sync(0xffffffffu, ka, l);
                lk = __shfl_sync(0xffffffffu, kz, l) - k0;
                n = __shfl_sync(0xffffffffu, tiles, l);
                first = __shfl_sync(0xffffffffu, up, l) - n;
            } else {
                left -= __shfl_sync(0xffffffffu, up, 31);
            }
        }
        if (found < 0) return release();
        row0 = (n - 1 - (left - first)) * (2 * kRows);
    }
    // row r of the sequence sees keys 0 .. r + shift, and lk - 1 at most
    const int shift = p.causal ? lk - lq : lk;
    auto blocks_of = [&](int i) {
        const int first = row0 + i * kRows, last = min(lq, first + kRows) - 1;
        if (first >= lq) return 0;
        const long long end = min((long long)lk, (long long)last + shift + 1);
        return end <= 0 ? 0 : (int)((end + kRows - 1) / kRows);
    };
    // this CTA's blocks, of all of them: from j0 on, n0 and n1 for the two tiles, counted from there
    const int all = max(blocks_of(0), blocks_of(1));
    const int j0 = (int)((long long)all * rank / p.splits), nb = (int)((long long)all * (rank + 1) / p.splits) - j0;
    const int n0 = max(0, min(blocks_of(0) - j0, nb)), n1 = max(0, min(blocks_of(1) - j0, nb));
    // from this block on some row does not see every key of it, or it is not whole
    const int edge = max(0, (int)(max(0ll, min((long long)lk, (long long)row0 + shift + 1)) / kRows) - j0);
    const int kv_head = head / p.group;
    // Load number `load` of k and v in turn (k of block j is 2 j, v 2 j + 1) is full
    // on full(slot), or for values of blocks from `edge` on, which are mended before
    // they are used, on v_raw(slot) and then v_ready(slot); those barriers see nothing
    // before. (Values use every other slot.)
    auto mended = [&](int load) { return (load & 1) != 0 && load >= 2 * edge; };
    auto parity = [&](int load) { return (uint32_t)((mended(load) ? (load / 2 - edge) / (NS / 2) : load / NS) & 1); };

    // (all 512 columns: the base is 0)
    // 384 threads are launched with 168 registers: the softmax warps take 216, the others 72 (256 * 216 + 128 * 72 = 384 * 168)
    if (warp >= kWarpMma) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kWarpTma) {
            if (lane == 0) {
                auto load = [&](const CUtensorMap* m, uint32_t dst, uint32_t bar, int h, int row) {
                    mbar_arrive_expect_tx(bar, Lay::kBlock);
                    for (int c = 0; c < CH; ++c) tma_load_3d(dst + c * (kRows * 128), m, bar, 64 * c, h, row);
                };
                bool ok = true;
                int issued = 0;
                auto next = [&](const CUtensorMap* m, int block) {
                    const int s = issued % NS;
                    if (!(ok = wait_here(empty(s), (uint32_t)((issued / NS) & 1) ^ 1u, p.status, p.timeout_ns, 40))) return;
                    load(m, sbase + Lay::kOffRing + s * Lay::kBlock, mended(issued) ? v_raw(s) : full(s), kv_head, k0 + (j0 + block) * kRows);
                    ++issued;
                };
                if (nb > 0) {
                    if (n0 > 0) load(&p.tm_q, sbase, q_full(0), head, q0 + row0);
                    next(&p.tm_k, 0);
                    if (n1 > 0) load(&p.tm_q, sbase + Lay::kBlock, q_full(1), head, q0 + row0 + kRows);
                    for (int j = 0; ok && j < nb; ++j) {
                        next(&p.tm_v, j);
                        if (ok && j + 1 < nb) next(&p.tm_k, j + 1);
                    }
                    // every load this thread issued lands before the CTA may exit
                    if (n0 > 0) drain_here(q_full(0), 0);
                    if (n1 > 0) drain_here(q_full(1), 0);
                    for (int i = issued - 1; i >= 0 && i >= issued - NS; --i)
                        drain_here(mended(i) ? v_raw(i % NS) : full(i % NS), parity(i));
                }
            }
        } else if (warp == kWarpMma) {
            const uint32_t qk = umma_idesc_f16(Ops::kFormat, kRows, kRows), pv = umma_idesc_f16(Ops::kFormat, kRows, DP) | kBMajorN;
            const uint64_t kd = sw128_kmajor_desc(sbase), vd = sw128_mnmajor_desc(sbase, kRows * 128);
            const uint32_t k_hi = (uint32_t)(kd >> 32), v_hi = (uint32_t)(vd >> 32);
            auto wait = [&](uint32_t bar, uint32_t parity, int where) {
                const bool ok = __all_sync(0xffffffffu, wait_here(bar, parity, p.status, p.timeout_ns, where));
                tc_fence_after();
                return ok;
            };
            auto slot_lo = [&](uint64_t d, int load) { return (uint32_t)d + (uint32_t)((Lay::kOffRing + load % NS * Lay::kBlock) >> 4); };
            auto scores = [&](int i, int load) {
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    mma4_ss(128u * i, (uint32_t)kd + (uint32_t)((i * Lay::kBlock + c * kRows * 128) >> 4),
                            slot_lo(kd, load) + (uint32_t)(c * kRows * 128 >> 4), k_hi, qk, c);
                commit_elected(s_full(i));
            };
            bool ok = true;
            if (nb > 0) {
                ok = wait(full(0), 0, 41);
                for (int i = 0; ok && i < 2; ++i)
                    if (0 < (i ? n1 : n0) && (ok = wait(q_full(i), 0, 42))) scores(i, 0);
                if (ok) commit_elected(empty(0));
            }
            for (int j = 0; ok && j < nb; ++j) {
                const int lv = 2 * j + 1, lkey = 2 * j + 2;
                if (!(ok = wait(mended(lv) ? v_ready(lv % NS) : full(lv % NS), parity(lv), 43))) break;
                if (j + 1 < nb && !(ok = wait(full(lkey % NS), parity(lkey), 45))) break;
                for (int i = 0; ok && i < 2; ++i) {
                    const int n = i ? n1 : n0;
                    if (j >= n) continue;
                    if (!(ok = wait(p_full(i), (uint32_t)(j & 1), 46))) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        mma4_ts(kOCol + 128u * i, 128u * i + 32u * h, slot_lo(vd, lv) + (uint32_t)(h * 64 * 128 >> 4), v_hi, pv,
                                (uint32_t)(j + h));
                    if (j + 1 < n) scores(i, lkey);
                    else commit_elected(o_full(i));
                }
                if (ok) {
                    commit_elected(empty(lv % NS));
                    if (j + 1 < nb) commit_elected(empty(lkey % NS));
                }
            }
            // all MMAs issued by this warp complete before tensor memory is released
            commit_elected(drain);
            drain_here(drain, 0);
        } else {
            // values of blocks that are not seen whole
            // (The first wait is for all blocks in front: 1.5 us each, over 2 s for some 1.4 million of them; every one adds to its limit.)
            const unsigned long long in_front = (unsigned long long)min(edge, nb) * kBlockNs;
            for (int j = edge; j < nb; ++j) {
                const int lv = 2 * j + 1, s = lv % NS;
                if (!__all_sync(0xffffffffu, wait_here(v_raw(s), parity(lv), p.status, p.timeout_ns + in_front, 47))) break;
                const int first_key = (j0 + j) * kRows, valid = min(kRows, lk - first_key);
                const uint32_t base = sbase + Lay::kOffRing + s * Lay::kBlock;
                constexpr int U = 8;  // vectors in flight (one at a time a block took 1.7 us longer than its products)
                for (int c = 0; c < CH; ++c)
                    for (int e = valid * 8 + (int)threadIdx.x - kWarpFix * 32; e < kRows * 8; e += 64)
                        st_shared_v4(base + c * (kRows * 128) + 16 * e, 0u, 0u, 0u, 0u);
#pragma unroll 1
                for (int e0 = threadIdx.x - kWarpFix * 32; e0 < kRows * CH * 8; e0 += 64 * U) {
                    // vector e: 64-channel chunk e / 1024, row e / 8 % 128, 16-byte place e % 8 in its row
                    uint32_t m = 0;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const uint4 x = ld_shared_v4(base + 16 * (e0 + 64 * u));
                        if ((e0 + 64 * u) / 8 % kRows < valid) m = absmax2<DT>(m, absmax8<DT>(x));
                    }
                    // (the rare cases in a loop of their own: the instructions of the common one are few and stay cached)
                    if (absmax_halves<DT>(m) < Bits16<DT>::kInf) continue;
#pragma unroll 1
                    for (int e = e0; e < e0 + 64 * U; e += 64) {
                        const int r = e / 8 % kRows;
                        if (r < valid)
                            take_out<DT, DP>(base + 16 * e, e / (8 * kRows) * 64 + (((e & 7) ^ (r & 7)) << 3), first_key + r, note);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(v_ready(s));
            }
            if (lane == 0) mbar_arrive(fixed);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ------------------------------------------------------------ softmax: a row per thread
        const int i = warp >> 2, n = i ? n1 : n0, r = row0 + (int)threadIdx.x;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, s_col = lanes + 128u * i, o_col = lanes + kOCol + 128u * i;
        const int last = (int)min((long long)lk - 1, (long long)r + shift);  // the last key that the row sees
        const int warp_last = (int)min((long long)lk - 1, (long long)(r - lane) + shift);
        const float kNone = __int_as_float(0xff800000);
        float m = kNone, neg = 0.f;  // the maximum, and minus it (0 where there is none yet)
        float2 l = make_float2(0.f, 0.f);
        bool any_large = false, ok = true;
        // c s - m is formed with one rounding. Once m is 2^20 in size its own rounding would show in that, as 2^4 and more from
        // 2^28 on, which p cannot hold: such a row's scores are rounded, as m was, before the difference. (Warps without such a row pass by;
        // the check and what stands behind it cost calls 0.1 to 1 us of a CTA's start, and 2 % at 64 channels.)
        auto weights_of_large = [&](int j) {
            const int seen = last - (j0 + j) * kRows;
            const bool large = fabsf(neg) >= kLarge;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                float x[32];
                uint32_t w[16];
                tmem_ld_32x32b_x32(s_col + 32u * c, reinterpret_cast<uint32_t(&)[32]>(x));
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float v[2];
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const float y = large ? __fadd_rn(__fmul_rn(x[e + f], p.c), neg) : fmaf(x[e + f], p.c, neg);
                        v[f] = 32 * c + e + f > seen ? 0.f : ex2(y);
                    }
                    l = add2(l, make_float2(v[0], v[1]));
                    w[e / 2] = Ops::pack(v[0], v[1]);
                }
                tmem_st_32x32b_x16(s_col + 16u * c, w);
            }
        };
        for (int j = 0; j < n; ++j) {
            if (!(ok = __all_sync(0xffffffffu, wait_here(s_full(i), (uint32_t)(j & 1), p.status, p.timeout_ns, 48)))) break;
            tc_fence_after();
            float s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(s_col + 32u * c, reinterpret_cast<uint32_t(&)[32]>(s[c]));
            tmem_ld_wait();
            if ((j0 + j) * kRows + kRows - 1 > warp_last) {
                const int seen = last - (j0 + j) * kRows;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * c + e > seen) s[c][e] = kNone;
            }
            float top = kNone, top1 = kNone;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    top = fmaxf(top, fmaxf(s[c][e], s[c][e + 1]));
                    top1 = fmaxf(top1, fmaxf(s[c][e + 2], s[c][e + 3]));
                }
            top = fmaxf(top, top1) * p.c;
            const bool over = top > m + kLazy;
            if (__any_sync(0xffffffffu, over)) {
                float f = 1.f;
                if (over) {
                    f = ex2(m - top);
                    m = top, neg = -top;
                }
                any_large = __any_sync(0xffffffffu, fabsf(neg) >= kLarge);
                if (j > 0) {
                    l.x *= f, l.y *= f;
#pragma unroll
                    for (int c = 0; c < DP / 32; ++c) {
                        float o[32];
                        tmem_ld_32x32b_x32(o_col + 32u * c, reinterpret_cast<uint32_t(&)[32]>(o));
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f;
                        tmem_st_32x32b_x32(o_col + 32u * c, reinterpret_cast<uint32_t(&)[32]>(o));
                    }
                }
            }
            if (__builtin_expect(any_large, 0)) {
                weights_of_large(j);
            } else {
                const float2 cc = make_float2(p.c, p.c), nn = make_float2(neg, neg);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float* x = &s[2 * h + e / 16][2 * (e % 16)];
                        const float2 y = ffma2(make_float2(x[0], x[1]), cc, nn);
                        const float2 v = make_float2(ex2(y.x), ex2(y.y));
                        l = add2(l, v);
                        w[e] = Ops::pack(v.x, v.y);
                    }
                    tmem_st_32x32b_x32(s_col + 32u * h, w);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(i));
        }
        if (ok && n > 0) {
            ok = __all_sync(0xffffffffu, wait_here(o_full(i), 0, p.status, p.timeout_ns, 49));
            tc_fence_after();
            if (ok) ok = __all_sync(0xffffffffu, wait_here(fixed, 0, p.status, p.timeout_ns, 50));
        }
        if (p.splits > 1) {
            // this CTA's part: sums as they are, in fp32, once no product reads shared memory any more
            named_bar_sync(1, 2 * kRows);
            const uint32_t part = sbase + threadIdx.x * (Lay::kPitch * 4);
#pragma unroll 1
            for (int c = 0; c < DP / 32; ++c) {
                float o[32];
                if (n > 0) {
                    tmem_ld_32x32b_x32(o_col + 32u * c, reinterpret_cast<uint32_t(&)[32]>(o));
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    st_shared_v4(part + (32 * c + e) * 4, __float_as_uint(o[e]), __float_as_uint(o[e + 1]), __float_as_uint(o[e + 2]),
                                 __float_as_uint(o[e + 3]));
            }
            if (n > 0 && *reinterpret_cast<volatile int*>(note + 3 * DP) != 0) {
#pragma unroll 1
                for (int ch = 0; ch < DP; ++ch) {
                    float y = ld_shared_f32(part + 4 * ch);
                    if (note[ch] <= last) y += __int_as_float(0x7fffffff);
                    if (note[DP + ch] <= last) y -= kNone;
                    if (note[2 * DP + ch] <= last) y += kNone;
                    st_shared_f32(part + 4 * ch, y);
                }
            }
            *reinterpret_cast<float2*>(smem + Lay::kOffMl + threadIdx.x * 8) = make_float2(m, l.x + l.y);
        } else if (ok && row0 + i * kRows < lq) {
            const bool any = n > 0 && *reinterpret_cast<volatile int*>(note + 3 * DP) != 0;
            const float f = last >= 0 ? 1.f / (l.x + l.y) : 0.f;
            // A warp's rows go through its part of its tile of q, which no product reads any more, so that
            // neighbouring lanes store neighbouring 16 bytes (a row per lane: 5 us instead of 1).
            const uint32_t stage = sbase + i * Lay::kBlock + (warp & 3) * 32 * (DP * 2);
#pragma unroll 1
            for (int c = 0; c < DP / 32; ++c) {
                float o[32];
                if (n > 0) {
                    tmem_ld_32x32b_x32(o_col + 32u * c, reinterpret_cast<uint32_t(&)[32]>(o));
                    tmem_ld_wait();
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint4 v = make_uint4(Ops::pack(o[e] * f, o[e + 1] * f), Ops::pack(o[e + 2] * f, o[e + 3] * f),
                                         Ops::pack(o[e + 4] * f, o[e + 5] * f), Ops::pack(o[e + 6] * f, o[e + 7] * f));
                    if (last < 0) v = make_uint4(0u, 0u, 0u, 0u);
                    const int chunk = 4 * c + e / 8;
                    st_shared_v4(stage + lane * (DP * 2) + ((chunk ^ (lane & 7)) << 4), v.x, v.y, v.z, v.w);
                }
            }
            __syncwarp();
            uint16_t* out = p.out + (long long)head * p.o_head;
            constexpr int C = DP / 8, R = 32 / C;  // chunks of a row, rows of a store
            const int chunk = lane % C, first = r - lane;
            if (!any) {
                // (eight rows' loads before the first store: one after another 16 stores took 1.6 us)
#pragma unroll
                for (int k0 = 0; k0 < 32; k0 += 8 * R) {
                    uint4 v[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int row = k0 + u * R + lane / C;
                        v[u] = ld_shared_v4(stage + row * (DP * 2) + ((chunk ^ (row & 7)) << 4));
                    }
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int row = k0 + u * R + lane / C;
                        if (first + row < lq && chunk * 8 < p.head_dim)
                            *reinterpret_cast<uint4*>(out + (long long)(q0 + first + row) * p.o_row + chunk * 8) = v[u];
                    }
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < 32; k += R) {
                    const int row = k + lane / C;
                    const int sees = __shfl_sync(0xffffffffu, last, row);
                    const uint4 v = put_back<DT, DP>(ld_shared_v4(stage + row * (DP * 2) + ((chunk ^ (row & 7)) << 4)), chunk * 8, sees, note);
                    if (first + row < lq && chunk * 8 < p.head_dim)
                        *reinterpret_cast<uint4*>(out + (long long)(q0 + first + row) * p.o_row + chunk * 8) = v;
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    release();
    if (p.splits > 1) {
        cluster_barrier_sync();
        // each CTA finishes its share of the rows: a row to a warp, DP / 32 channels to a lane
        constexpr int C = DP / 32, kMost = 8;
        const int rows = min(2 * kRows, lq - row0);
        const float kNone = __int_as_float(0xff800000);
        for (int r = rows * rank / p.splits + warp; r < rows * (rank + 1) / p.splits; r += kThreads / 32) {
            float ml[2] = {kNone, 0.f};
            if (lane < p.splits)
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(ml[0]), "=f"(ml[1]) : "r"(mapa_cluster(sbase + Lay::kOffMl + r * 8, lane)) : "memory");
            float o[kMost][C];
#pragma unroll
            for (int c = 0; c < kMost; ++c) {
                if (c >= p.splits) continue;
                const uint32_t at = mapa_cluster(sbase + (r * Lay::kPitch + lane * C) * 4, c);
                if constexpr (C == 4)
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(o[c][0]), "=f"(o[c][1]), "=f"(o[c][2]), "=f"(o[c][3]) : "r"(at) : "memory");
                else
                    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(o[c][0]), "=f"(o[c][1]) : "r"(at) : "memory");
            }
            float top = ml[0];
#pragma unroll
            for (int w = 4; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            top = __shfl_sync(0xffffffffu, top, 0);
            const float weight = ml[0] == kNone ? 0.f : ex2(ml[0] - top);
            float sum = 0.f, y[C] = {};
#pragma unroll
            for (int c = 0; c < kMost; ++c) {
                if (c >= p.splits) continue;
                const float w = __shfl_sync(0xffffffffu, weight, c);
                sum = fmaf(__shfl_sync(0xffffffffu, ml[1], c), w, sum);
#pragma unroll
                for (int e = 0; e < C; ++e) y[e] = fmaf(o[c][e], w, y[e]);
            }
            const bool sees = min((long long)lk - 1, (long long)row0 + r + shift) >= 0;
            const float f = sees ? 1.f / sum : 0.f;
            uint16_t* out = p.out + (long long)(q0 + row0 + r) * p.o_row + (long long)head * p.o_head + lane * C;
            if (lane * C >= p.head_dim) continue;
            if constexpr (C == 4)
                *reinterpret_cast<uint2*>(out) = sees ? make_uint2(Ops::pack(y[0] * f, y[1] * f), Ops::pack(y[2] * f, y[3] * f)) : make_uint2(0u, 0u);
            else
                *reinterpret_cast<uint32_t*>(out) = sees ? Ops::pack(y[0] * f, y[1] * f) : 0u;
        }
        cluster_barrier_sync();  // (the others have read this CTA's part)
    }
}

}  // namespace

}  // namespace fl

extern "C" fl_status fl_attention(const fl_attention_desc* d, void* stream) {
    using namespace fl;
    using host::fail;
    const char* what = "fl_attention";
    if (d == nullptr) return fail(FL_ERR_INVALID_ARG, "%s: null description", what);
    if (!host::valid_dtype(d->dtype)) return fail(FL_ERR_INVALID_ARG, "%s: bad dtype %d", what, (int)d->dtype);
    if (d->rows_q < 0 || d->rows_k < 0 || d->heads_q < 1 || d->heads_k < 1 || d->head_dim < 1 || d->n_seqs < 1)
        return fail(FL_ERR_INVALID_ARG, "%s: sizes must be positive (rows may be 0)", what);
    if (d->heads_q % d->heads_k != 0)
        return fail(FL_ERR_INVALID_ARG, "%s: heads_q (%d) must be a multiple of heads_k (%d)", what, d->heads_q, d->heads_k);
    if (d->head_dim % 8 != 0) return fail(FL_ERR_ALIGNMENT, "%s: head_dim must be a multiple of 8 (%d)", what, d->head_dim);
    if (d->head_dim > 128) return fail(FL_ERR_UNSUPPORTED, "%s: head_dim above 128 (%d)", what, d->head_dim);
    if (!(d->scale > 0.f) || d->scale > 1e30f) return fail(FL_ERR_INVALID_ARG, "%s: scale must be positive and finite", what);
    if ((d->cu_q == nullptr) != (d->cu_k == nullptr))
        return fail(FL_ERR_INVALID_ARG, "%s: cu_q and cu_k must be given both or neither", what);
    if (d->cu_q == nullptr && d->n_seqs != 1) return fail(FL_ERR_INVALID_ARG, "%s: cu_q must be given for several sequences", what);
    if (d->n_seqs > 1 << 30) return fail(FL_ERR_UNSUPPORTED, "%s: more than 2^30 sequences", what);
    // 256-row tiles at most: every sequence with rows has one that may be short
    const long long seqs = d->rows_q < d->n_seqs ? d->rows_q : d->n_seqs;
    const long long tiles = d->cu_q == nullptr ? (d->rows_q + 2ll * kRows - 1) / (2 * kRows)
                                               : (d->rows_q + (2ll * kRows - 1) * seqs) / (2 * kRows);
    if (tiles * d->heads_q >= (1ll << 31) || d->rows_q > INT_MAX - 4 * kRows || d->rows_k > INT_MAX - 4 * kRows)
        return fail(FL_ERR_UNSUPPORTED, "%s: too many rows", what);
    if (d->rows_q == 0) return host::ok();
    fl_status st;
    if ((st = host::check_ptr("q", d->q, true)) != FL_OK) return st;
    if ((st = host::check_ptr("k", d->k, d->rows_k > 0)) != FL_OK) return st;
    if ((st = host::check_ptr("v", d->v, d->rows_k > 0)) != FL_OK) return st;
    if ((st = host::check_ptr("out", d->out, true)) != FL_OK) return st;
    if ((reinterpret_cast<uintptr_t>(d->cu_q) | reinterpret_cast<uintptr_t>(d->cu_k)) & 3u)
        return fail(FL_ERR_ALIGNMENT, "%s: cu_q and cu_k must be 4-byte aligned", what);
    struct Side {
        const char* name;
        const void* p;
        int rows, heads;
        long long row, head;
    };
    const Side sides[4] = {{"out", d->out, d->rows_q, d->heads_q, d->out_row, d->out_head},
                           {"q", d->q, d->rows_q, d->heads_q, d->q_row, d->q_head},
                           {"k", d->k, d->rows_k, d->heads_k, d->k_row, d->k_head},
                           {"v", d->v, d->rows_k, d->heads_k, d->v_row, d->v_head}};
    for (int i = 0; i < 4; ++i) {
        const Side& s = sides[i];
        if (s.rows == 0) continue;
        if ((st = host::check_heads(what, s.name, s.rows, s.heads, d->head_dim, s.row, s.head, i == 0)) != FL_OK) return st;
        // (a tensor map's strides are below 2^40 bytes)
        if (s.row >= 1ll << 39 || s.head >= 1ll << 39)
            return fail(FL_ERR_UNSUPPORTED, "%s: strides of %s above 2^39 elements", what, s.name);
        if ((s.rows > 1 && s.row == 0) || (s.heads > 1 && s.head == 0))
            return fail(FL_ERR_UNSUPPORTED, "%s: %s is expanded (a stride of 0)", what, s.name);
        if (i == 0) continue;
        if (host::apart(d->out, d->out_row, (d->heads_q - 1) * d->out_head + d->head_dim, s.p, s.row,
                        (s.heads - 1) * s.head + d->head_dim, 2))
            continue;
        if (host::overlap(d->out, host::span_heads(d->rows_q, d->heads_q, d->head_dim, d->out_row, d->out_head), s.p,
                          host::span_heads(s.rows, s.heads, d->head_dim, s.row, s.head)))
            return fail(FL_ERR_INVALID_ARG, "%s: out overlaps %s", what, s.name);
    }
    for (const int* cu : {d->cu_q, d->cu_k})
        if (cu != nullptr && host::overlap(d->out, host::span_heads(d->rows_q, d->heads_q, d->head_dim, d->out_row, d->out_head),
                                           cu, ((size_t)d->n_seqs + 1) * 4))
            return fail(FL_ERR_INVALID_ARG, "%s: out overlaps cu_q or cu_k", what);
    host::LaunchContext ctx;
    if ((st = host::launch_context(static_cast<cudaStream_t>(stream), &ctx)) != FL_OK) return st;
    AttnParams p = {};
    CUtensorMap* maps[3] = {&p.tm_q, &p.tm_k, &p.tm_v};
    for (int i = 0; i < 3; ++i) {
        Side s = sides[i + 1];
        if (s.rows == 0) s = sides[1];  // (no keys: never read)
        if ((st = host::encode_heads(maps[i], d->dtype, s.p, d->head_dim, s.heads, s.rows,
                                     s.heads > 1 ? s.head : d->head_dim, s.rows > 1 ? s.row : d->head_dim, kRows)) != FL_OK)
            return st;
    }
    p.out = static_cast<uint16_t*>(d->out), p.o_row = d->out_row, p.o_head = d->out_head;
    p.cu_q = d->cu_q, p.cu_k = d->cu_k, p.rows_q = d->rows_q, p.rows_k = d->rows_k, p.heads_q = d->heads_q;
    p.group = d->heads_q / d->heads_k, p.head_dim = d->head_dim, p.n_seqs = d->n_seqs, p.causal = d->causal != 0;
    p.c = d->scale * 1.44269504088896341f;
    p.status = ctx.status, p.timeout_ns = ctx.timeout_ns;
    // Fewer CTAs than half the multiprocessors: clusters, while each CTA keeps four blocks of keys
    // (of a sequence of average length).
    const long long blocks = (d->rows_k / d->n_seqs + kRows - 1) / kRows;
    p.splits = 1;
    while (p.splits < 8 && tiles * d->heads_q * p.splits * 2 <= ctx.sms && blocks >= 8 * p.splits) p.splits *= 2;
    auto go = [&](auto dt, auto dp) -> fl_status {
        constexpr int DT = decltype(dt)::value, DP = decltype(dp)::value;
        static std::atomic<unsigned long long> done{0};
        constexpr int bytes = Layout<DP>::kSmem;
        static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
        const cudaError_t e = host::allow_smem(fl_attention_kernel<DT, DP>, bytes, ctx.device, done);
        if (e != cudaSuccess) return host::fail(FL_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
        return host::launched(host::launch_cluster(fl_attention_kernel<DT, DP>, dim3((unsigned)(tiles * d->heads_q * p.splits)), kThreads,
                                                   bytes, ctx.pdl, p.splits, static_cast<cudaStream_t>(stream), p),
                              what);
    };
    using std::integral_constant;
    if (d->dtype == FL_F16)
        return d->head_dim <= 64 ? go(integral_constant<int, DT_F16>(), integral_constant<int, 64>())
                                 : go(integral_constant<int, DT_F16>(), integral_constant<int, 128>());
    return d->head_dim <= 64 ? go(integral_constant<int, DT_BF16>(), integral_constant<int, 64>())
                             : go(integral_constant<int, DT_BF16>(), integral_constant<int, 128>());
}
