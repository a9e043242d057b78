// Attention over the paged 8-bit cache for sequences of many rows: the
// verification of large trees, prompts behind a cache (fl_kv_attend; the
// formulas and the division of the work are those of fl_kv_attend.cu and .cuh).
//
// Up to 256 rows (a sequence's rows times a group's heads) are two tiles of 128 on
// the tensor cores, as in fl_attention.cu: S = Q K^T into tensor memory, weights
// in its place as the A operand of O += W V, values as an MN-major operand. The codes
// are widened to fp16, exactly, on their way: TMA brings them into shared memory as they
// are, six warps write them out as the 16-bit operands' swizzled blocks, and the
// scales go onto the scores and the weights as before, two per position. The
// warp-level kernel widens them again for every 32 rows: trees of 48 rows for a group of four
// heads over contexts of 1000 to 10600 positions, 23000 in all, 146 us there, 59 to 60 here.
//
// What bounds it: of those the start of a CTA (lengths and plan 4, rows of q 4)
// takes 10, its 9 to 11 blocks 2.8 to 3 each (of which 1.8 are the softmax of a tile and 0.9 the
// products and the barriers between, the other tile's the same), the end 3, the second launch 5.
//
// Roles: warps 0-7 softmax, one tile to four of them, a row to a thread; warp 8 the
// MMAs, warp 9 the loads, 10-15 widen. Blocks of 128 positions of k and v take
// turns in a ring of three for the codes and one of three for the operands. The scales of
// four blocks are kept: loads run at most three blocks ahead of the softmax.
//
// Every mbarrier wait is bounded as in the other kernels.
#include <algorithm>
#include <type_traits>

#include "fl_kv_attend.cuh"

namespace fl {

namespace {

using namespace attend;

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kRows = 128;
constexpr int kWarpMma = 8, kWarpTma = 9, kWarpWiden = 10, kWiden = kWarps - kWarpWiden;
constexpr int kRing = 3, kTabs = 4;
constexpr int kOCol = 256;  // tensor-memory columns: S of tile i at 128 i, O at 256 + 128 i

template <int DP, int TILES>
struct Layout {
    static constexpr int kBlock = kRows * DP * 2;  // a tile of q, a block of k or v
    static constexpr int kCodes = kRows * DP;
    static constexpr int kOffRing = TILES * kBlock;
    static constexpr int kOffRaw = kOffRing + kRing * kBlock;
    static constexpr int kOffTab = kOffRaw + kRing * kCodes;          // [kTabs][3][128]: scales of k, of v, the logarithm of the latter
    static constexpr int kOffBits = kOffTab + kTabs * 3 * kRows * 4;  // [kTabs][4]: which positions are there
    static constexpr int kOffC = kOffBits + kTabs * 16;
    static constexpr int kOffBar = kOffC + TILES * kRows * 4;
    static constexpr int kBars = 4 * kRing + 6 + kTabs + 2;
    static constexpr int kOffSlot = kOffBar + kBars * 8;
    static constexpr int kSmem = kOffSlot + 16 + 1024;
    // what the rows' threads leave, in place of q, k and v: [rows][kPitch] sums
    static constexpr int kPitch = DP + 4;
    static_assert(TILES * kRows * kPitch * 4 <= kOffTab, "sums");
};

// Sixteen codes as fp16 in order.
template <int FMT>
__device__ __forceinline__ void widen16(const uint4& x, uint32_t (&o)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (FMT == FL_KV_INT8) {
            // 1024 + 128 + code in the mantissa, less 1152
            const uint32_t u = w[i] ^ 0x80808080u;
            const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
            asm("sub.f16x2 %0, %1, %2;" : "=r"(o[2 * i]) : "r"(lo), "r"(0x64806480u));
            asm("sub.f16x2 %0, %1, %2;" : "=r"(o[2 * i + 1]) : "r"(hi), "r"(0x64806480u));
        } else {
            o[2 * i] = widen<FMT>(w[i]);
            o[2 * i + 1] = widen<FMT>(w[i] >> 16);
        }
    }
}

// DP: head_dim rounded up to 64 or 128. TILES: 1 or 2.
template <int DT, int FMT, int DP, int TILES>
__global__ void __launch_bounds__(kThreads, 1) fl_kv_attend_tile_kernel(const __grid_constant__ AttendParams p) {
    using Ops = DTypeOps<DT>;
    using Lay = Layout<DP, TILES>;
    constexpr int M = TILES * kRows, CH = DP / 64;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (sbase - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar0 = sbase + Lay::kOffBar;
    auto raw_full = [&](int x) { return bar0 + 8u * (x % kRing); };
    auto raw_empty = [&](int x) { return bar0 + 8u * (kRing + x % kRing); };
    auto full = [&](int x) { return bar0 + 8u * (2 * kRing + x % kRing); };
    auto empty = [&](int x) { return bar0 + 8u * (3 * kRing + x % kRing); };
    auto s_full = [&](int i) { return bar0 + 8u * (4 * kRing + i); };
    auto p_full = [&](int i) { return bar0 + 8u * (4 * kRing + 2 + i); };
    auto o_full = [&](int i) { return bar0 + 8u * (4 * kRing + 4 + i); };
    auto tab_full = [&](int j) { return bar0 + 8u * (4 * kRing + 6 + j % kTabs); };
    const uint32_t drain = bar0 + 8u * (4 * kRing + 6 + kTabs), q_full = drain + 8u;
    auto round = [&](int x) { return (uint32_t)(x / kRing & 1); };
    float* const tabs = reinterpret_cast<float*>(smem + Lay::kOffTab);
    float* const cs = reinterpret_cast<float*>(smem + Lay::kOffC);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kRing; ++s) {
            mbar_init(raw_full(s), 33);
            mbar_init(raw_empty(s), kWiden);
            mbar_init(full(s), kWiden);
            mbar_init(empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), 4);
            mbar_init(o_full(i), 1);
        }
        for (int j = 0; j < kTabs; ++j) mbar_init(tab_full(j), kWiden);
        mbar_init(drain, 1);
        mbar_init(q_full, kWarps - 1);
        fence_mbar_init();
    }
    if (warp == kWarpTma && lane < 2) tma_prefetch_desc(&p.tm[lane]);
    if (warp == kWarpMma) {
        tmem_alloc(sbase + Lay::kOffSlot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch_dependents();

    // ------------------------------------------------------------ the CTA's piece
    const Pieces<kWarps, kTileResident> pieces(p, M, false);
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.part != nullptr) units_of<kTileResident, M, DP>(p)->count = (int)pieces.units;
    Seq s;
    Piece piece;
    const bool mine = pieces.find(0, piece, s);
    if (!mine || piece.seq < 0) {
        if (warp == kWarpMma) tmem_dealloc(0u, 512);
        return;
    }
    const int r0 = piece.block * M, rows = min(M, s.n * p.group - r0);
    const int t0 = (int)((long long)s.tiles * piece.k / piece.pieces), t1 = (int)((long long)s.tiles * (piece.k + 1) / piece.pieces);
    const int k0 = t0 * kTile, k1 = min(s.keys, t1 * kTile), nb = t1 - t0;
    const int n0 = nb, n1 = rows > kRows ? nb : 0;
    if (piece.k == 0 && threadIdx.x == 0) {
        if (s.from + s.n > (long long)p.table_pages * p.page_size) atomicCAS(p.range, 0, s.row0 + 1);
        if (piece.pieces > 1)
            units_of<kTileResident, M, DP>(p)->unit[piece.units] = Unit{s.row0, s.n, r0, piece.head, piece.pieces, piece.slot, s.blocks * p.heads, 0};
    }

    // ------------------------------------------------------------ q as fp16, a row to sixteen lanes
    // (by all warps but the one that loads)
    if (warp != kWarpTma) {
        const int c = lane & 15, first = 2 * (warp < kWarpTma ? warp : warp - 1) + (lane >> 4);
        constexpr int kStride = 2 * (kWarps - 1);
        auto place = [&](int r) {
            return sbase + r / kRows * Lay::kBlock + (c >> 3) * (kRows * 128) + r % kRows * 128 + (((c & 7) ^ (r & 7)) << 4);
        };
        constexpr int Q = (M + kStride - 1) / kStride;
        uint4 q[Q];
        // (row of q and head from step to step without a division)
        const int i_step = kStride / p.group, h_step = kStride - i_step * p.group;
        int i = (r0 + first) / p.group, h = (r0 + first) - i * p.group;
#pragma unroll
        for (int u = 0; u < Q; ++u) {
            const int r = first + u * kStride;
            if (u > 0) {
                i += i_step, h += h_step;
                if (h >= p.group) ++i, h -= p.group;
            }
            q[u] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows && 8 * c < p.head_dim)
                q[u] = ldg_v4(p.q + (long long)(s.row0 + i) * p.q_row + (long long)(piece.head * p.group + h) * p.q_head + 8 * c);
        }
#pragma unroll
        for (int u = 0; u < Q; ++u) {
            const int r = first + u * kStride;
            uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
            float up = 1.f;
            if (DT == DT_BF16) {
                // 2^(14 - e) for a largest value of 2^e to 2^(e + 1); rows without a finite, not tiny one stay as they are
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int ex = (int)(top >> 7);
                if (ex > 0 && ex < 255) up = __uint_as_float((uint32_t)min(254, 127 + 14 + 127 - ex) << 23);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = Ops::unpack(w[e]);
                    w[e] = DTypeOps<DT_F16>::pack(f.x * up, f.y * up);
                }
            }
            if (r < M && 8 * c < DP) st_shared_v4(place(r), w[0], w[1], w[2], w[3]);
            if (r < M && c == 0) cs[r] = fmaxf(p.log2_scale / up, 0x1p-126f);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
    }

    // (all 512 columns of tensor memory: the base is 0)
    // 512 threads are launched with 128 registers: the softmax warps take 176, the others 80 (256 * 176 + 256 * 80 = 512 * 128)
    if (warp >= kWarpMma) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == kWarpMma) {
            const uint32_t qk = umma_idesc_f16(0, kRows, kRows), wv = umma_idesc_f16(0, kRows, DP) | kBMajorN;
            const uint64_t kd = sw128_kmajor_desc(sbase), vd = sw128_mnmajor_desc(sbase, kRows * 128);
            const uint32_t k_hi = (uint32_t)(kd >> 32), v_hi = (uint32_t)(vd >> 32);
            auto wait = [&](uint32_t bar, uint32_t parity, int where) {
                const bool ok = __all_sync(0xffffffffu, wait_here(bar, parity, p.status, p.timeout_ns, where));
                tc_fence_after();
                return ok;
            };
            auto slot_lo = [&](uint64_t d, int x) { return (uint32_t)d + (uint32_t)((Lay::kOffRing + x % kRing * Lay::kBlock) >> 4); };
            auto scores = [&](int i, int x) {
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    mma4_ss(128u * i, (uint32_t)kd + (uint32_t)((i * Lay::kBlock + c * kRows * 128) >> 4),
                            slot_lo(kd, x) + (uint32_t)(c * kRows * 128 >> 4), k_hi, qk, c);
                commit_elected(s_full(i));
            };
            bool ok = true;
            if (nb > 0) {
                ok = wait(q_full, 0, 60) && wait(full(0), 0, 61);
                for (int i = 0; ok && i < TILES; ++i)
                    if (0 < (i ? n1 : n0)) scores(i, 0);
                if (ok) commit_elected(empty(0));
            }
            for (int j = 0; ok && j < nb; ++j) {
                const int xv = 2 * j + 1, xk = 2 * j + 2;
                if (!(ok = wait(full(xv), round(xv), 62))) break;
                if (j + 1 < nb && !(ok = wait(full(xk), round(xk), 63))) break;
                for (int i = 0; ok && i < TILES; ++i) {
                    if (j >= (i ? n1 : n0)) continue;
                    if (!(ok = wait(p_full(i), (uint32_t)(j & 1), 64))) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        mma4_ts(kOCol + 128u * i, 128u * i + 32u * h, slot_lo(vd, xv) + (uint32_t)(h * 64 * 128 >> 4), v_hi, wv, (uint32_t)(j + h));
                    if (j + 1 < nb) scores(i, xk);
                    else commit_elected(o_full(i));
                }
                if (ok) {
                    commit_elected(empty(xv));
                    if (j + 1 < nb) commit_elected(empty(xk));
                }
            }
            // all MMAs issued by this warp complete before tensor memory is released
            commit_elected(drain);
            drain_here(drain, 0);
        } else if (warp == kWarpTma) {
            // positions lane + 32 u of a block: their table entries (one block ahead), boxes and scales
            const int* table = p.page_table + piece.seq * p.table_stride;
            int entry[4], row[4], next[4], next_row[4];
            auto look_up = [&](int j, int* e, int* in_page) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int pos = k0 + j * kRows + 32 * u + lane;
                    e[u] = -2, in_page[u] = 0;
                    if (j < nb && pos < k1) {
                        const int page = p.page_shift >= 0 ? pos >> p.page_shift : (int)((uint32_t)pos / (uint32_t)p.page_size);
                        in_page[u] = pos - page * p.page_size;
                        e[u] = __ldg(table + page);
                    }
                }
            };
            look_up(0, next, next_row);
            bool ok = true;
            int issued = 0;
            for (int x = 0; ok && x < 2 * nb; ++x) {
                const int j = x >> 1;
                if ((x & 1) == 0) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) entry[u] = next[u], row[u] = next_row[u];
                    look_up(j + 1, next, next_row);
                }
                if (!(ok = __all_sync(0xffffffffu, wait_here(raw_empty(x), round(x) ^ 1u, p.status, p.timeout_ns, 65)))) break;
                const uint32_t dst = sbase + Lay::kOffRaw + x % kRing * Lay::kCodes, tab = sbase + Lay::kOffTab + j % kTabs * (3 * kRows * 4);
                // (which positions are there, in front of the arrival that hands it on: the one behind the copies orders them alone)
                if ((x & 1) == 0) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t bits = __ballot_sync(0xffffffffu, entry[u] >= 0 && entry[u] < p.n_pages);
                        if (lane == 0)
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(sbase + Lay::kOffBits + j % kTabs * 16 + 4 * u), "r"(bits) : "memory");
                    }
                }
                if (lane == 0) mbar_arrive_expect_tx(raw_full(x), Lay::kCodes);
                __syncwarp();
                const CUtensorMap* map = &p.tm[x & 1];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool there = entry[u] >= 0 && entry[u] < p.n_pages;
                    const int at = 32 * u + lane;
                    // (a page that is not there: past the last, zeros)
                    if ((at & ((1 << p.box_log) - 1)) == 0)
                        tma_load_4d(dst + at * DP, map, raw_full(x), 0, piece.head, there ? row[u] : 0, there ? entry[u] : p.n_pages);
                    if ((x & 1) == 0) {
                        if (entry[u] != -2 && !there) atomicCAS(p.range, 0, s.row0 + 1);
                        if (there) {
                            const long long from = ((long long)entry[u] * p.page_size + row[u]) * p.heads + piece.head;
                            cp_async4(tab + at * 4, p.scale[0] + from);
                            cp_async4(tab + (kRows + at) * 4, p.scale[1] + from);
                        }
                    }
                }
                __syncwarp();
                cp_async_arrive(raw_full(x));
                ++issued;
            }
            // every load of this warp lands before the CTA may exit
            for (int x = issued - 1; x >= 0 && x >= issued - kRing; --x) drain_here(raw_full(x), round(x));
        } else {
            const int tid = (int)threadIdx.x - kWarpWiden * 32;
            bool ok = true;
            for (int x = 0; ok && x < 2 * nb; ++x) {
                const int j = x >> 1;
                ok = wait_here(raw_full(x), round(x), p.status, p.timeout_ns, 66) && wait_here(empty(x), round(x) ^ 1u, p.status, p.timeout_ns, 67);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const uint32_t src = sbase + Lay::kOffRaw + x % kRing * Lay::kCodes, dst = sbase + Lay::kOffRing + x % kRing * Lay::kBlock;
                float* const tab = tabs + j % kTabs * (3 * kRows);
                if ((x & 1) == 0 && tid < kRows) tab[2 * kRows + tid] = lg2(tab[kRows + tid]);
                const uint4 bits = ld_shared_v4(sbase + Lay::kOffBits + j % kTabs * 16);
                const bool gaps = (bits.x & bits.y & bits.z & bits.w) != 0xffffffffu;
                constexpr int V = kRows * DP / 16, U = (V + 32 * kWiden - 1) / (32 * kWiden);  // vectors of 16 codes, in flight
#pragma unroll 1
                for (int e0 = tid; e0 < V; e0 += 32 * kWiden * U) {
                    uint4 v[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int e = e0 + 32 * kWiden * u;
                        if (e < V) v[u] = ld_shared_v4(src + 16 * e);
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int e = e0 + 32 * kWiden * u, r = e / (DP / 16), c = e % (DP / 16);
                        if (e >= V) continue;
                        if ((x & 1) && gaps) {
                            // (a value that is not there may be none, and would not vanish times zero)
                            const uint32_t word = r < 64 ? (r < 32 ? bits.x : bits.y) : (r < 96 ? bits.z : bits.w);
                            if (!(word >> (r & 31) & 1)) v[u] = make_uint4(0u, 0u, 0u, 0u);
                        }
                        uint32_t o[8];
                        widen16<FMT>(v[u], o);
                        const uint32_t at = dst + (c >> 2) * (kRows * 128) + r * 128;
                        const uint32_t k = (uint32_t)(2 * (c & 3)) ^ (r & 7);
                        st_shared_v4(at + (k << 4), o[0], o[1], o[2], o[3]);
                        st_shared_v4(at + ((k ^ 1u) << 4), o[4], o[5], o[6], o[7]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if ((x & 1) == 0) mbar_arrive(tab_full(j));
                    mbar_arrive(full(x));
                    mbar_arrive(raw_empty(x));
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        // ------------------------------------------------------------ softmax: a row per thread
        const int i = warp >> 2, n = i ? n1 : n0, r = (int)threadIdx.x;  // (one tile: warps 4-7 have nothing to do)
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, s_col = lanes + 128u * i, o_col = lanes + kOCol + 128u * i;
        const float kNone = __int_as_float(0xff800000), kNoMaxYet = __int_as_float(0x7f800000);
        wait_here(q_full, 0, p.status, p.timeout_ns, 59);
        const float c = r < M ? cs[r] : 0.f;
        const int qi = min(r0 + r, s.n * p.group - 1) / p.group;  // the row of q among the sequence's
        const int q_first = __shfl_sync(0xffffffffu, qi, 0), q_last = __shfl_sync(0xffffffffu, qi, 31);  // of the warp
        float mx = kNone, nx = 0.f, mb = kNone;  // the maximum of x, minus it (0 where there is none yet); that of x + log2 vs, less it
        float2 l = make_float2(0.f, 0.f);
        bool seen = false, ok = true;
        const bool idle = r - lane >= rows;  // (a warp without rows: what its lines of the products hold is not read)
        for (int j = 0; j < n; ++j) {
            // Drafts that the row sees, found while the scores are on their way. (A row of the tree per load, eight at
            // once: a draft per load and thread, one after another, took 13 us in the last block of a tree of 48.)
            const int pos0 = k0 + j * kRows;
            uint32_t sees[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
            if (pos0 + kRows > s.from && !idle) {
#pragma unroll 1
                for (int w = 0; w < 4; ++w) {
                    const long long first = pos0 + 32 * w - s.from;  // the draft at the word's bit 0
                    if (first + 31 < 0) continue;
                    uint32_t m = 0;
                    if (p.tree == nullptr) {
                        const long long d = qi - first;
                        m = d >= 31 ? 0xffffffffu : d < 0 ? 0u : (2u << (int)d) - 1u;
                    } else {
                        const long long d = first + lane;
                        const bool in = d >= 0 && d < p.tree_cols;
                        constexpr int U = 8;
#pragma unroll 1
                        for (int q = q_first; q <= q_last; q += U) {
                            const uint8_t* at = p.tree + (s.row0 + q) * p.tree_stride + d;
                            uint32_t is[U];
#pragma unroll
                            for (int u = 0; u < U; ++u) {
                                is[u] = in && q + u <= q_last ? __ldg(at) : d < 0;
                                at += p.tree_stride;
                            }
#pragma unroll
                            for (int u = 0; u < U; ++u) {
                                const uint32_t word = __ballot_sync(0xffffffffu, is[u] != 0);
                                if (qi == q + u) m = word;
                            }
                        }
                    }
                    if (w == 0) sees[0] = m;
                    if (w == 1) sees[1] = m;
                    if (w == 2) sees[2] = m;
                    if (w == 3) sees[3] = m;
                }
            }
            ok = wait_here(tab_full(j), (uint32_t)(j / kTabs & 1), p.status, p.timeout_ns, 68) && wait_here(s_full(i), (uint32_t)(j & 1), p.status, p.timeout_ns, 69);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            if (idle) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(i));
                continue;
            }
            const uint32_t tab = sbase + Lay::kOffTab + j % kTabs * (3 * kRows * 4);
            const uint4 there = ld_shared_v4(sbase + Lay::kOffBits + j % kTabs * 16);
            sees[0] &= there.x, sees[1] &= there.y, sees[2] &= there.z, sees[3] &= there.w;
            const bool all = (sees[0] & sees[1] & sees[2] & sees[3]) == 0xffffffffu;
            seen |= (sees[0] | sees[1] | sees[2] | sees[3]) != 0;
            // Weights of the values: 2^(x + log2 vs - mx - mb) = 2^(x - mx) vs 2^-mb. Once there are maxima, and where every
            // position is seen, they are formed in one pass with those: good unless a weight passes 2^8 (or the
            // sum fp32's range), which is rare. Otherwise, and for maxima of kLarge or more in size, the maxima are found first.
            uint32_t w[4][16];
            bool done = false;
            const float2 cc = make_float2(c, c);
            if (__all_sync(0xffffffffu, all) && __any_sync(0xffffffffu, mx == kNone || mb == kNone)) {
                // (the first maxima: those of a quarter, which mostly will do)
                float x[32], ta = kNone, tb = kNone;
                tmem_ld_32x32b_x32(s_col, reinterpret_cast<uint32_t(&)[32]>(x));
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float y = x[e] * ld_shared_f32(tab + e * 4) * c;
                    ta = fmaxf(ta, y), tb = fmaxf(tb, y + ld_shared_f32(tab + (2 * kRows + e) * 4));
                }
                if (mx == kNone && ta > kNone && fabsf(ta) < kLarge) mx = ta, nx = -ta;
                if (mb == kNone && tb > kNone && mx > kNone && fabsf(nx) < kLarge) mb = tb + nx;
            }
            if (__all_sync(0xffffffffu, all && mx > kNone && mb > kNone && fabsf(nx) < kLarge)) {
                const float to = ex2(-mb);
                const float2 nn = make_float2(nx, nx), tt = make_float2(to, to);
                float2 sum = l;
                uint32_t most = 0;
                float x2[2][32];  // (the next 32 scores on their way)
                tmem_ld_32x32b_x32(s_col, reinterpret_cast<uint32_t(&)[32]>(x2[0]));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    tmem_ld_wait();
                    if (q < 3) tmem_ld_32x32b_x32(s_col + 32u * (q + 1), reinterpret_cast<uint32_t(&)[32]>(x2[(q + 1) & 1]));
                    const float (&x)[32] = x2[q & 1];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const uint4 k4 = ld_shared_v4(tab + (32 * q + e) * 4), v4 = ld_shared_v4(tab + (kRows + 32 * q + e) * 4);
                        const float2 y0 = ffma2(mul2(make_float2(x[e], x[e + 1]), make_float2(__uint_as_float(k4.x), __uint_as_float(k4.y))), cc, nn);
                        const float2 y1 = ffma2(mul2(make_float2(x[e + 2], x[e + 3]), make_float2(__uint_as_float(k4.z), __uint_as_float(k4.w))), cc, nn);
                        const float2 a0 = make_float2(ex2(y0.x), ex2(y0.y)), a1 = make_float2(ex2(y1.x), ex2(y1.y));
                        const float2 b0 = mul2(mul2(a0, make_float2(__uint_as_float(v4.x), __uint_as_float(v4.y))), tt);
                        const float2 b1 = mul2(mul2(a1, make_float2(__uint_as_float(v4.z), __uint_as_float(v4.w))), tt);
                        sum = add2(sum, add2(a0, a1));
                        w[q][e / 2] = DTypeOps<DT_F16>::pack(b0.x, b0.y), w[q][e / 2 + 1] = DTypeOps<DT_F16>::pack(b1.x, b1.y);
                        asm("max.f16x2 %0, %0, %1;" : "+r"(most) : "r"(w[q][e / 2]));
                        asm("max.f16x2 %0, %0, %1;" : "+r"(most) : "r"(w[q][e / 2 + 1]));
                    }
                }
                // (weights are not negative: as 16-bit patterns they compare as numbers; 0x5c00 is 2^8)
                done = __all_sync(0xffffffffu, max(most & 0xffffu, most >> 16) <= 0x5c00u && sum.x + sum.y < 0x1p100f);
                if (done) l = sum;
            }
            if (!done) {
                float ta = kNone, tb = kNone;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    const uint32_t m = q < 2 ? (q == 0 ? sees[0] : sees[1]) : (q == 2 ? sees[2] : sees[3]);
                    float x[32];
                    tmem_ld_32x32b_x32(s_col + 32u * q, reinterpret_cast<uint32_t(&)[32]>(x));
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        // (a scale that is not there may be anything)
                        const uint4 k4 = ld_shared_v4(tab + (32 * q + e) * 4), l4 = ld_shared_v4(tab + (2 * kRows + 32 * q + e) * 4);
                        const uint32_t ks[4] = {k4.x, k4.y, k4.z, k4.w}, lv[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            const float y = __fmul_rn(x[e + f] * __uint_as_float(ks[f]), c);
                            if (m >> (e + f) & 1) ta = fmaxf(ta, y), tb = fmaxf(tb, y + __uint_as_float(lv[f]));
                        }
                    }
                }
                if (ta > mx) {
                    const float by = mx - ta;  // (-inf for the first maximum)
                    l.x *= ex2(by), l.y *= ex2(by);
                    mb += by;
                    mx = ta, nx = -ta;
                }
                tb = fabsf(nx) < kLarge ? tb + nx : kNoMaxYet;
                if (__any_sync(0xffffffffu, tb == kNoMaxYet)) {
                    // (the logarithm of vs is lost beside exponents of such a size: once more, less the maximum that is known now)
                    float t = kNone;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t m = q < 2 ? (q == 0 ? sees[0] : sees[1]) : (q == 2 ? sees[2] : sees[3]);
                        float x[32];
                        tmem_ld_32x32b_x32(s_col + 32u * q, reinterpret_cast<uint32_t(&)[32]>(x));
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float y = __fmul_rn(x[e] * ld_shared_f32(tab + (32 * q + e) * 4), c);
                            if (m >> e & 1) t = fmaxf(t, __fadd_rn(y, nx) + ld_shared_f32(tab + (2 * kRows + 32 * q + e) * 4));
                        }
                    }
                    if (tb == kNoMaxYet) tb = t;
                }
                const bool over = tb > mb;
                if (__any_sync(0xffffffffu, over)) {
                    float f = 1.f;
                    if (over) {
                        f = ex2(mb - tb);
                        mb = tb;
                    }
                    if (j > 0) {
#pragma unroll 1
                        for (int q = 0; q < DP / 32; ++q) {
                            float o[32];
                            tmem_ld_32x32b_x32(o_col + 32u * q, reinterpret_cast<uint32_t(&)[32]>(o));
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= f;
                            tmem_st_32x32b_x32(o_col + 32u * q, reinterpret_cast<uint32_t(&)[32]>(o));
                        }
                    }
                }
                const float to = mb == kNone ? 0.f : ex2(-mb);
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    const uint32_t m = q < 2 ? (q == 0 ? sees[0] : sees[1]) : (q == 2 ? sees[2] : sees[3]);
                    float x[32];
                    tmem_ld_32x32b_x32(s_col + 32u * q, reinterpret_cast<uint32_t(&)[32]>(x));
                    tmem_ld_wait();
                    uint32_t h[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const uint4 k4 = ld_shared_v4(tab + (32 * q + e) * 4), v4 = ld_shared_v4(tab + (kRows + 32 * q + e) * 4);
                        const uint32_t ks[4] = {k4.x, k4.y, k4.z, k4.w}, vs[4] = {v4.x, v4.y, v4.z, v4.w};
                        float a[4], b[4];
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            a[f] = ex2(__fadd_rn(__fmul_rn(x[e + f] * __uint_as_float(ks[f]), c), nx));
                            b[f] = a[f] * __uint_as_float(vs[f]) * to;
                            if (!(m >> (e + f) & 1)) a[f] = b[f] = 0.f;
                        }
                        l = add2(l, add2(make_float2(a[0], a[1]), make_float2(a[2], a[3])));
                        h[e / 2] = DTypeOps<DT_F16>::pack(b[0], b[1]), h[e / 2 + 1] = DTypeOps<DT_F16>::pack(b[2], b[3]);
                    }
                    tmem_st_32x32b_x16(s_col + 16u * q, h);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_st_32x32b_x16(s_col + 16u * q, w[q]);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(i));
        }
        if (ok && n > 0) {
            ok = __all_sync(0xffffffffu, wait_here(o_full(i), 0, p.status, p.timeout_ns, 70));
            tc_fence_after();
        }
        // the rows' sums, in fp32, once no product reads shared memory any more
        named_bar_sync(1, 2 * kRows);
        if (r < M && rows > i * kRows) {
            const uint32_t part = sbase + r * (Lay::kPitch * 4);
#pragma unroll 1
            for (int q = 0; q < DP / 32; ++q) {
                float o[32];
                if (n > 0) {
                    tmem_ld_32x32b_x32(o_col + 32u * q, reinterpret_cast<uint32_t(&)[32]>(o));
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    st_shared_v4(part + (32 * q + e) * 4, __float_as_uint(o[e]), __float_as_uint(o[e + 1]), __float_as_uint(o[e + 2]),
                                 __float_as_uint(o[e + 3]));
            }
            __syncwarp();
            const float sum = l.x + l.y;
            constexpr int C = DP / 32;
            const int first = r - lane;
            const float2 mine_f = finish(mb, sum, seen ? 1.f : 0.f);
            if (piece.pieces > 1 && r < rows)
                *reinterpret_cast<float4*>(p.part + (long long)slots(kTileResident) * M * DP + ((long long)piece.slot * M + r) * 4) =
                    make_float4(mx, mb, sum, seen ? 1.f : 0.f);
            if (piece.pieces > 1) {
                // (a row is 4 DP bytes in a run: one bulk copy; a row at a time by all lanes took 3 us)
                fence_proxy_async_smem();
                __syncwarp();
                if (r < rows) {
                    float* d = p.part + ((long long)piece.slot * M + r) * DP;
                    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(d), "r"(part), "r"(DP * 4) : "memory");
                    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
                }
            } else {
                // a row at a time to the warp, so that neighbouring lanes store neighbouring channels
                const unsigned long long mine_at = reinterpret_cast<unsigned long long>(row_at(p, s.row0, piece.head, r0 + min(r, rows - 1)));
#pragma unroll 4
                for (int k = 0; k < 32; ++k) {
                    const float fx = __shfl_sync(0xffffffffu, mine_f.x, k), fy = __shfl_sync(0xffffffffu, mine_f.y, k);
                    uint16_t* d = reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, mine_at, k)) + lane * C;
                    if (first + k >= rows || lane * C >= p.head_dim) continue;
                    const uint32_t at = sbase + ((first + k) * Lay::kPitch + lane * C) * 4;
                    if constexpr (C == 4) {
                        const uint4 o = ld_shared_v4(at);
                        uint2 y = make_uint2(Ops::pack(__uint_as_float(o.x) * fx, __uint_as_float(o.y) * fx),
                                             Ops::pack(__uint_as_float(o.z) * fx, __uint_as_float(o.w) * fx));
                        if (fy != 0.f) y = make_uint2(0u, 0u);
                        *reinterpret_cast<uint2*>(d) = y;
                    } else {
                        const uint32_t y = Ops::pack(ld_shared_f32(at) * fx, ld_shared_f32(at + 4) * fx);
                        *reinterpret_cast<uint32_t*>(d) = fy != 0.f ? 0u : y;
                    }
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) tmem_dealloc(0u, 512);
}

}  // namespace

namespace attend {

cudaError_t launch_tile(const AttendParams& p, int dt, int fmt, int hd, int M, long long units, bool split,
                        const host::LaunchContext& ctx, cudaStream_t stream, int* launches) {
    const dim3 grid((unsigned)(units + (split ? kTileResident : 0)));
    auto go = [&](auto dtc, auto fmtc, auto hdc, auto mc) -> cudaError_t {
        constexpr int DT = decltype(dtc)::value, FMT = decltype(fmtc)::value, HD = decltype(hdc)::value, MR = decltype(mc)::value;
        static std::atomic<unsigned long long> done{0};
        constexpr int bytes = Layout<HD, MR / kRows>::kSmem;
        static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
        cudaError_t e = host::allow_smem(fl_kv_attend_tile_kernel<DT, FMT, HD, MR / kRows>, bytes, ctx.device, done);
        if (e == cudaSuccess) e = host::launch(fl_kv_attend_tile_kernel<DT, FMT, HD, MR / kRows>, grid, kThreads, bytes, ctx.pdl, stream, p);
        *launches = 1;
        if (e != cudaSuccess || !split) return e;
        const dim3 join((unsigned)std::min<long long>(ctx.sms * 16ll, units * (MR / 4)));
        *launches = 2;
        return host::launch(fl_kv_attend_join_kernel<DT, HD, kTileResident, MR>, join, kJoinThreads, 0, ctx.pdl, stream, p);
    };
    using std::integral_constant;
    auto by_rows = [&](auto dtc, auto fmtc, auto hdc) {
        return M == 128 ? go(dtc, fmtc, hdc, integral_constant<int, 128>()) : go(dtc, fmtc, hdc, integral_constant<int, 256>());
    };
    auto by_size = [&](auto dtc, auto fmtc) {
        return hd == 64 ? by_rows(dtc, fmtc, integral_constant<int, 64>()) : by_rows(dtc, fmtc, integral_constant<int, 128>());
    };
    if (dt == FL_F16)
        return fmt == FL_KV_INT8 ? by_size(integral_constant<int, DT_F16>(), integral_constant<int, FL_KV_INT8>())
                                 : by_size(integral_constant<int, DT_F16>(), integral_constant<int, FL_KV_E4M3>());
    return fmt == FL_KV_INT8 ? by_size(integral_constant<int, DT_BF16>(), integral_constant<int, FL_KV_INT8>())
                             : by_size(integral_constant<int, DT_BF16>(), integral_constant<int, FL_KV_E4M3>());
}

}  // namespace attend

}  // namespace fl
