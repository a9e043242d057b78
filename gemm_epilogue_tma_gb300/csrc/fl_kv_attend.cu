// Attention of new tokens over the paged 8-bit cache (fl_kv_attend): a decode
// step, or the verification of a tree of drafted tokens.
//
//   out[i, h] = sum_p w v[p] / sum_p w,  w = 2^x,  x = scale log2(e) ks[p] (q[i, h] . kc[p]),  v[p] = vs[p] vc[p]
//
// over the positions p that row i sees. The codes kc, vc are what the MMAs
// multiply: both formats fit fp16 exactly (e4m3 by the conversion instruction), so no
// key or value is rounded; ks goes onto the fp32 scores, and vs into the weights
// of the second product, w vs = 2^(x + log2 vs), which have a running maximum of
// their own, kept less that of x, so that they fill fp16's range whatever the scales are. Rounded are
// those weights (fp16, 2^-12 of each) and the output. bf16 rows of q are
// multiplied as fp16 times a power of two per row, which keeps their 8 bits down
// to 2^-28 of the row's largest value.
//
// The cache is read once for a row block (a sequence's rows and all query heads of the group, 8, 16
// or 32 of them; more are further blocks, which read it again) and nothing is written but the
// output, so HBM bounds it: 2 head_dim + 8 bytes per position and key head. Keys are the rows of the first MMA, 16 positions,
// and channels those of the second, O^T = V^T P^T; the rows of q are its columns, in
// tiles of eight, so that a decode step of a group of four or eight heads pads
// little, and P^T, 16 positions by 8, is the first product's result turned by
// movmatrix. A warp takes 16 positions a step through a ring of its own in shared memory
// (TMA boxes of the rows that lie in one page, no CTA barriers), converts the codes
// to MMA fragments in registers (channels permuted so that 16-byte loads give
// whole fragments), and keeps its own maxima, sums and outputs; the warps of a CTA
// are joined in shared memory at the end.
//
// Long contexts are split into pieces of L tiles of 128 positions at most. The CTAs
// are persistent and take every gridDim-th piece. L is the one of six that makes the
// rounds of CTAs shortest (of sixteen: 4 us longer to find, no better); every CTA finds it,
// and its pieces, from the lengths, which only the GPU knows. Pieces of a split sequence
// are joined by a second launch, in order.
//
// What bounds it, by measurement with 32 and 8 heads of 128, bf16: 64 contexts of 8192
// positions int8 225 us (4.9 TB/s), e4m3 186 (5.9); parts of an earlier form that took 236 and 195: without the arithmetic
// 178, without the loads 210 and 165: for int8 the conversion of codes, whose logical operations are issued at half
// rate. 16 contexts of 500 to 9600, e4m3 fp16: 37.1 us, of which the longest piece takes 27 and
// the start of a CTA (lengths, plan, table, first loads) 7 and the second launch 3. 61 of
// 20 to 300 positions: 14.6 to 14.9 us, 7 of them that start, 5 the longest context, 2 the end; 15.8 with a table of 4096
// positions, which might be split, for a second launch that finds nothing to join.
#include <algorithm>
#include <type_traits>

#include "fl_kv_attend.cuh"

namespace fl {

namespace {

using namespace attend;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kResident = 304;  // CTAs at work at once: two on each of 152 multiprocessors
static_assert(kTile == kStep * kWarps, "a tile is a step of all warps");
// The kernel for many rows is taken for more than kRowsLimit rows of a sequence and key head (on average) and tables
// of kLongTable positions at least; the lengths themselves are not known here. Both sides, us, eight key heads: four contexts
// of 5700 with 16 rows each 29 here, 42 there; with 32 42 and 42, with 36 64 and 44, with 96 82 and 44; 32 contexts of 1000 with
// 48 rows 88 and 65; one of 2000 with 36 rows 18 and 20. In short tables one of 500 with 192 rows 22.6 and 25.8, four of 300 with 48
// rows 14 and 17. What the rule does not see: such short contexts in a wide table (16 and 20), and a short table with
// very many rows, or many sequences, where the other side is the faster (four of 300 with 1024 rows 126 and 38, 32 of 300 with
// 48 rows 50 and 35).
constexpr int kRowsLimit = 32, kLongTable = 1024;


__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The four codes of a word in two pairs, the first product's order of channels: int8 0 and 2, 1
// and 3; e4m3 0 and 1, 2 and 3. (q is laid out to match: kPair.)
template <int FMT>
__device__ __forceinline__ void widen_word(uint32_t w, uint32_t& first, uint32_t& second) {
    first = widen<FMT>(w);
    second = widen<FMT>(FMT == FL_KV_INT8 ? w >> 8 : w >> 16);
}
template <int FMT>
constexpr int kPair = FMT == FL_KV_INT8 ? 2 : 1;  // distance of a pair's channels
// Code b of word lo and of word hi.
template <int FMT>
__device__ __forceinline__ uint32_t widen_pair(uint32_t lo, uint32_t hi, int b) {
    return widen<FMT>(__byte_perm(lo, hi, (uint32_t)(FMT == FL_KV_INT8 ? b | b << 4 | (4 + b) << 8 | (4 + b) << 12 : b | (4 + b) << 4)));
}

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// 16-byte chunk c of row r of a stage's k or v, as TMA lays it out: rows of 64 or
// 128 bytes with the swizzle of that width, 256 channels as two such blocks.
template <int HD>
__device__ __forceinline__ uint32_t place(int r, int c) {
    if constexpr (HD == 64) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    return (uint32_t)((c >> 3) * (kStep * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Shared memory: the warps' rings (k and v of a stage, 1024-byte aligned); what a
// warp leaves to be joined (sums [M][HD + 4], then [M][4]: maxima, sum of weights, seen)
// lies in its own ring where that holds it, so that the warps of other pieces may still
// be at work; per warp and stage scales of k and v and which positions
// are there; the barriers; the rows of q as MMA fragments, where registers do not hold them.
template <int HD, int QT>
struct Layout {
    static constexpr int M = 8 * QT;
    static constexpr int kCtas = HD <= 128 && QT <= 2 ? 2 : 1;  // on a multiprocessor, as registers and shared memory allow
    static constexpr bool kQInRegs = HD * QT <= 128;
    static constexpr int kStages = HD == 64 ? 4 : 3;
    static constexpr int kStage = 2 * kStep * HD;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kSums = M * (HD + 4) * 4;
    static constexpr int kArea = kQInRegs ? kStages * kStage : kSums + M * 16;  // from one warp's sums to the next's
    static_assert(kSums + M * 16 <= kArea, "sums of a warp");
    static constexpr int kFirst = kRing > kWarps * kArea ? kRing : kWarps * kArea;
    static constexpr int kMeta = 2 * kStep * 4 + 16;
    static constexpr int kOffMeta = kFirst;
    static constexpr int kOffQ = kOffMeta + kWarps * kStages * kMeta;
    static constexpr int kQ = kQInRegs ? 0 : QT * (HD / 16) * 32 * 8;
    static constexpr int kOffC = kOffQ + kQ;
    static constexpr int kOffBar = kOffC + M * 4;
    static constexpr int kSmem = kOffBar + kWarps * kStages * 8 + 1024;
};

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// HD: head_dim rounded up to 64, 128 or 256. QT: tiles of eight rows of q (of a
// sequence's rows and a group's heads). TMA: head_dim a multiple of 16, and boxes that
// can start where they have to; otherwise the codes come in copies of 8 bytes.
template <int DT, int FMT, int HD, int QT, bool TMA>
__global__ void __launch_bounds__(kThreads, Layout<HD, QT>::kCtas) fl_kv_attend_kernel(const __grid_constant__ AttendParams p) {
    using Ops = DTypeOps<DT>;
    using Lay = Layout<HD, QT>;
    constexpr int M = 8 * QT, KS = HD / 16, MT = HD / 16, NS = Lay::kStages, VW = HD / 32;  // VW: words of v per lane and position
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (sbase - smem_u32(smem_raw));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    auto full = [&](int s) { return sbase + Lay::kOffBar + (uint32_t)(warp * NS + s) * 8u; };
    if (lane == 0) {
        for (int s = 0; s < NS; ++s) mbar_init(full(s), 33);
        fence_mbar_init();
        if (TMA && warp < 2) tma_prefetch_desc(&p.tm[warp]);
    }
    griddep_wait();
    griddep_launch_dependents();
    const Pieces<kWarps, kResident> pieces(p, M, Lay::kQInRegs);
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.part != nullptr) units_of<kResident, M, HD>(p)->count = (int)pieces.units;
    const uint32_t ring = sbase + warp * NS * Lay::kStage, meta = sbase + Lay::kOffMeta + warp * NS * Lay::kMeta;
    const float kNone = __int_as_float(0xff800000), kNoMax = __int_as_float(0x7f7fffff);
    int stage = 0;       // the ring runs on from piece to piece
    uint32_t phase = 0;

    const int W = pieces.W, group = warp / W, own = warp % W;  // the piece's warps
    const int stride = W * kStep;                              // positions of a step of all of them
    auto group_sync = [&] {
        if (W == kWarps) __syncthreads();
        else if (W > 1) named_bar_sync(1 + group, 32 * W);
        else __syncwarp();
    };

    bool ok = true;
    for (uint32_t turn = 0;; ++turn) {
        Seq s;
        Piece piece;
        if (!pieces.find(turn, piece, s)) break;
        if (piece.seq >= 0) {
            const int r0 = piece.block * M, rows = min(M, s.n * p.group - r0);  // rows of this block: (row of q, head of the group)
            const int t0 = (int)((long long)s.tiles * piece.k / piece.pieces), t1 = (int)((long long)s.tiles * (piece.k + 1) / piece.pieces);
            const int k0 = t0 * kTile, k1 = min(s.keys, t1 * kTile);
            if (piece.k == 0 && own == 0 && lane == 0) {
                if (s.from + s.n > (long long)p.table_pages * p.page_size) atomicCAS(p.range, 0, s.row0 + 1);
                if (piece.pieces > 1)
                    units_of<kResident, M, HD>(p)->unit[piece.units] = Unit{s.row0, s.n, r0, piece.head, piece.pieces, piece.slot, s.blocks * p.heads, 0};
            }

            // ------------------------------------------------------------ the warp's ring
            if (!TMA) {
                // channels past head_dim stay zero
                for (int i = lane; i < NS * Lay::kStage / 16; i += 32) st_shared_v4(ring + 16 * i, 0u, 0u, 0u, 0u);
                __syncwarp();
            }
            const int steps = k1 > k0 + own * kStep ? (k1 - k0 - own * kStep + stride - 1) / stride : 0;
            const int* table = p.page_table + piece.seq * p.table_stride;
            // the table's entry of this lane's position of a step, one step ahead; -2: there is no such position
            int entry = -2, in_page = 0;
            auto look_up = [&](int step, int& entry, int& in_page) {
                const int pos = k0 + own * kStep + step * stride + (lane & 15);
                entry = -2, in_page = 0;
                if (step < steps && pos < k1) {
                    const int j = p.page_shift >= 0 ? pos >> p.page_shift : (int)((uint32_t)pos / (uint32_t)p.page_size);
                    in_page = pos - j * p.page_size;
                    entry = __ldg(table + j);
                }
            };
            // lanes 0-15 ask for k, the others for v
            auto request = [&](int step, int at) {
                if (step >= steps) return;
                const uint32_t bar = full(at), dst = ring + at * Lay::kStage + (lane >> 4) * (kStep * HD), m = meta + at * Lay::kMeta;
                const bool there = entry >= 0 && entry < p.n_pages;
                if (entry != -2 && !there) atomicCAS(p.range, 0, s.row0 + 1);
                const uint32_t bits = __ballot_sync(0xffffffffu, there) & 0xffffu;
                if (lane == 0) {
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(m + 2 * kStep * 4), "r"(bits) : "memory");
                    mbar_arrive_expect_tx(bar, TMA ? Lay::kStage : 0);
                }
                if (TMA) {
                    __syncwarp();
                    const int r = lane & 15;
                    if ((r & ((1 << p.box_log) - 1)) == 0) {
                        // (a page that is not there: past the last, zeros)
                        const CUtensorMap* map = &p.tm[lane >> 4];
                        const int page = there ? entry : p.n_pages, row = there ? in_page : 0;
                        tma_load_4d(dst + r * (HD == 64 ? 64 : 128), map, bar, 0, piece.head, row, page);
                        if (HD == 256) tma_load_4d(dst + kStep * 128 + r * 128, map, bar, 128, piece.head, row, page);
                    }
                } else {
                    const long long from = there ? (((long long)entry * p.page_size + in_page) * p.heads + piece.head) * p.head_dim : 0;
                    const uint8_t* src = (lane < 16 ? p.cache[0] : p.cache[1]) + from;
                    for (int c = 0; c < p.head_dim; c += 8) cp_async8(dst + place<HD>(lane & 15, c / 16) + (c & 8), src + c);
                }
                if (there) cp_async4(m + lane * 4, (lane < 16 ? p.scale[0] : p.scale[1]) + ((long long)entry * p.page_size + in_page) * p.heads + piece.head);
                cp_async_arrive(bar);
            };
            // ------------------------------------------------------------ the first loads
            // (what they depend on, the table's entries, and the rows of q are asked for at once)
            constexpr int QX = Lay::kQInRegs ? QT : 1;
            uint4 qx[QX][KS / 2];
            auto load_q = [&](int qt, uint4* x) {
                const int r = 8 * qt + g, i = (r0 + r) / p.group, h = (r0 + r) - i * p.group;
                const uint16_t* q = p.q + (long long)(s.row0 + i) * p.q_row + (long long)(piece.head * p.group + h) * p.q_head + 16 * t;
#pragma unroll
                for (int j = 0; j < KS / 2; ++j) {
                    const int ch = j / 2 * 64 + j % 2 * 8;
                    x[j] = r < rows && ch + 16 * t < p.head_dim ? ldg_v4(q + ch) : make_uint4(0u, 0u, 0u, 0u);
                }
            };
            // (a lane's entries of steps lane / 16 and 2 + lane / 16)
            int first_entry[2], first_row[2];
            static_assert(NS == 3 || NS == 4, "two look-ups of two steps");
#pragma unroll
            for (int i = 0; i < 2; ++i) look_up(2 * i + (lane >> 4), first_entry[i], first_row[i]);
            if constexpr (Lay::kQInRegs) {
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) load_q(qt, qx[qt]);
            }
            int ahead = stage;
            auto first = [&](int i) {
                const int from = 16 * (i & 1) + (lane & 15);
                entry = __shfl_sync(0xffffffffu, i < 2 ? first_entry[0] : first_entry[1], from);
                in_page = __shfl_sync(0xffffffffu, i < 2 ? first_row[0] : first_row[1], from);
            };
#pragma unroll 1
            for (int i = 0; i < NS - 1; ++i) {
                first(i);
                request(i, ahead);
                if (++ahead == NS) ahead = 0;
            }
            first(NS - 1);

            // ------------------------------------------------------------ q as the first product's B fragments
            // Step ks = 4 h + w takes channels 64 h + 16 t + 4 w + 0 .. 3 of lane t, in widen_word's order, row g of the tile.
            // c: what q' . code is multiplied by, for rows 2 t and 2 t + 1 of a tile.
            uint2 qf[QX][Lay::kQInRegs ? KS : 1];
            uint2* const qs = reinterpret_cast<uint2*>(smem + Lay::kOffQ);
            float* const cs = reinterpret_cast<float*>(smem + Lay::kOffC);
            float c[QT][2];
            auto q_tile = [&](const uint4* x, auto put) {  // returns the factor of row g
                float up = 1.f;
                if (DT == DT_BF16) {
                    // 2^(14 - e) for a largest value of 2^e to 2^(e + 1); rows without a finite, not tiny one stay as they are
                    uint32_t top = 0;
#pragma unroll
                    for (int j = 0; j < KS / 2; ++j) {
                        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
                    }
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    const int ex = (int)(max(top, __shfl_xor_sync(0xffffffffu, top, 2)) >> 7);
                    if (ex > 0 && ex < 255) up = __uint_as_float((uint32_t)min(254, 127 + 14 + 127 - ex) << 23);
                }
#pragma unroll
                for (int j = 0; j < KS / 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 lo = Ops::unpack(e ? x[j].z : x[j].x), hi = Ops::unpack(e ? x[j].w : x[j].y);
                        const float2 second = kPair<FMT> == 2 ? make_float2(lo.y, hi.y) : hi;
                        put(j / 2 * 4 + j % 2 * 2 + e, make_uint2(DTypeOps<DT_F16>::pack(lo.x * up, (kPair<FMT> == 2 ? hi.x : lo.y) * up),
                                                                  DTypeOps<DT_F16>::pack(second.x * up, second.y * up)));
                    }
                return fmaxf(p.log2_scale / up, 0x1p-126f);
            };
            if constexpr (Lay::kQInRegs) {
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) {
                    const float f = q_tile(qx[qt], [&](int ks, uint2 v) { qf[qt][ks] = v; });
                    c[qt][0] = __shfl_sync(0xffffffffu, f, 8 * t), c[qt][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
                }
            } else {
                for (int qt = warp; qt < QT; qt += kWarps) {
                    load_q(qt, qx[0]);
                    const float f = q_tile(qx[0], [&](int ks, uint2 v) { qs[(qt * KS + ks) * 32 + lane] = v; });
                    if (t == 0) cs[8 * qt + g] = f;
                }
                __syncthreads();
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) c[qt][0] = cs[8 * qt + 2 * t], c[qt][1] = cs[8 * qt + 2 * t + 1];
            }

            // ------------------------------------------------------------ the warp's positions
            // nx, nb: minus the maximum of the exponents x, and minus that of x + log2 vs less it; kNoMax, fp32's largest
            // number, where there is none yet, which any exponent exceeds by more than kLazy
            float nx[QT][2], nb[QT][2], l[QT][2], o[QT][MT][4];
            uint32_t seen = 0;  // bit 2 qt + f: the row saw a position (which tells it from one whose scores are all -inf)
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
#pragma unroll
                for (int f = 0; f < 2; ++f) nx[qt][f] = nb[qt][f] = kNoMax, l[qt][f] = 0.f;
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[qt][j][e] = 0.f;
            }

            for (int step = 0; step < steps; ++step) {
                __syncwarp();  // (the stage that is asked for next has been read)
                request(step + NS - 1, ahead);
                look_up(step + NS, entry, in_page);
                if (++ahead == NS) ahead = 0;
                ok = __all_sync(0xffffffffu, wait_bar(full(stage), phase, p.status, p.timeout_ns, 51));
                if (!ok) break;
                const uint32_t src = ring + stage * Lay::kStage, sc = meta + stage * Lay::kMeta;
                if (++stage == NS) stage = 0, phase ^= 1u;
                const int pos0 = k0 + own * kStep + step * stride;

                // scores x[qt][2 i + f] of position g + 8 i and row 2 t + f of the tile
                float x[QT][4];
#pragma unroll
                for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[qt][e] = 0.f;
#pragma unroll
                for (int h = 0; h < KS / 4; ++h) {
                    const uint4 ka = ld_shared_v4(src + place<HD>(g, 4 * h + t)), kb = ld_shared_v4(src + place<HD>(g + 8, 4 * h + t));
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t a[4];
                        widen_word<FMT>(w == 0 ? ka.x : w == 1 ? ka.y : w == 2 ? ka.z : ka.w, a[0], a[2]);
                        widen_word<FMT>(w == 0 ? kb.x : w == 1 ? kb.y : w == 2 ? kb.z : kb.w, a[1], a[3]);
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt) {
                            uint2 b;
                            if constexpr (Lay::kQInRegs) b = qf[qt][4 * h + w];
                            else b = qs[(qt * KS + 4 * h + w) * 32 + lane];
                            mma16816(x[qt], a, b.x, b.y);
                        }
                    }
                }
                // scales of the lane's two positions
                float ks[2], lv[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) ks[i] = ld_shared_f32(sc + 4 * g + 32 * i), lv[i] = lg2(ld_shared_f32(sc + 64 + 4 * g + 32 * i));
                const uint32_t bits = __float_as_uint(ld_shared_f32(sc + 2 * kStep * 4));
                uint32_t hidden = 0;  // bit 4 qt + e: the row does not see the position
                if (bits != 0xffffu || pos0 + kStep > s.from) {
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const int r = min(r0 + 8 * qt + 2 * t + f, s.n * p.group - 1);  // (rows past the last: as the last)
                            const int qi = p.tree == nullptr ? 0 : r / p.group;             // the row of q among the sequence's
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const long long j = pos0 + g + 8 * i - s.from;
                                bool sees = bits >> (g + 8 * i) & 1;
                                if (sees && j >= 0) {
                                    if (p.tree == nullptr) sees = j * p.group <= r;
                                    else sees = j < p.tree_cols && __ldg(p.tree + (s.row0 + qi) * p.tree_stride + j) != 0;
                                }
                                if (sees) seen |= 1u << (2 * qt + f);
                                else hidden |= 1u << (4 * qt + 2 * i + f);
                            }
                        }
                } else {
                    seen = (1u << 2 * QT) - 1;
                }
                // exponents less the maxima, for the sum of weights and for the weights of the values. (Each step is rounded: a fused
                // one would show how the maximum was, by 2^4 and more for exponents of 2^28 on, which a weight cannot hold.)
                float a[QT][4], b[QT][4], most = kNone;
                auto exponents = [&] {
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 y = add2(make_float2(x[qt][2 * i], x[qt][2 * i + 1]), make_float2(nx[qt][0], nx[qt][1]));
                            const float2 z = add2(y, add2(make_float2(lv[i], lv[i]), make_float2(nb[qt][0], nb[qt][1])));
                            a[qt][2 * i] = y.x, a[qt][2 * i + 1] = y.y, b[qt][2 * i] = z.x, b[qt][2 * i + 1] = z.y;
                        }
                    if (hidden != 0) {
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (hidden >> (4 * qt + e) & 1) a[qt][e] = b[qt][e] = kNone;
                    }
                };
#pragma unroll
                for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 y = mul2(mul2(make_float2(x[qt][2 * i], x[qt][2 * i + 1]), make_float2(ks[i], ks[i])), make_float2(c[qt][0], c[qt][1]));
                        x[qt][2 * i] = y.x, x[qt][2 * i + 1] = y.y;
                    }
                exponents();
#pragma unroll
                for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) most = fmaxf(most, fmaxf(a[qt][e], b[qt][e]));
                if (__any_sync(0xffffffffu, most > kLazy)) {
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            float ma = kNone, mb = kNone;
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (!(hidden >> (4 * qt + 2 * i + f) & 1)) ma = fmaxf(ma, x[qt][2 * i + f]);
#pragma unroll
                            for (int w = 4; w < 32; w <<= 1) ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, w));
                            // (a maximum that is there already only grows)
                            const bool first = nx[qt][f] == kNoMax;
                            if (first ? ma > kNone : ma > -nx[qt][f]) {
                                l[qt][f] *= first ? 0.f : ex2(-nx[qt][f] - ma);
                                if (nb[qt][f] != kNoMax) nb[qt][f] += ma + nx[qt][f];  // (that maximum itself stays)
                                nx[qt][f] = -ma;
                            }
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (!(hidden >> (4 * qt + 2 * i + f) & 1)) mb = fmaxf(mb, x[qt][2 * i + f] + nx[qt][f] + lv[i]);
#pragma unroll
                            for (int w = 4; w < 32; w <<= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, w));
                            if (nb[qt][f] == kNoMax ? mb > kNone : mb > -nb[qt][f]) {
                                const float y = nb[qt][f] == kNoMax ? 0.f : ex2(-nb[qt][f] - mb);
#pragma unroll
                                for (int j = 0; j < MT; ++j) o[qt][j][f] *= y, o[qt][j][2 + f] *= y;
                                nb[qt][f] = -mb;
                            }
                        }
                    exponents();
                }
                // P^T: 16 positions (k) by 8 rows
                uint2 w[QT];
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) {
#pragma unroll
                    for (int f = 0; f < 2; ++f) l[qt][f] += ex2(a[qt][f]) + ex2(a[qt][2 + f]);
                    w[qt].x = movmatrix(DTypeOps<DT_F16>::pack(ex2(b[qt][0]), ex2(b[qt][1])));
                    w[qt].y = movmatrix(DTypeOps<DT_F16>::pack(ex2(b[qt][2]), ex2(b[qt][3])));
                }
                // values: row block j is channels 2 j (rows 0-7) and 2 j + 1 (8-15) of the lane's 4 VW, k positions 2 t, 2 t + 1, + 8
                uint32_t v[4][VW];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 8 * (i >> 1) + 2 * t + (i & 1);
                    if constexpr (VW == 2) {
                        const uint32_t at = src + kStep * HD + place<HD>(r, g >> 1) + 8 * (g & 1);
                        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[i][0]), "=r"(v[i][1]) : "r"(at) : "memory");
                    } else {
#pragma unroll
                        for (int q = 0; q < VW / 4; ++q) {
                            const uint4 u = ld_shared_v4(src + kStep * HD + place<HD>(r, g * (VW / 4) + q));
                            v[i][4 * q] = u.x, v[i][4 * q + 1] = u.y, v[i][4 * q + 2] = u.z, v[i][4 * q + 3] = u.w;
                        }
                    }
                }
                if (bits != 0xffffu) {
                    // (what lies behind the last position may hold codes that are not numbers)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!(bits >> (8 * (i >> 1) + 2 * t + (i & 1)) & 1))
#pragma unroll
                            for (int q = 0; q < VW; ++q) v[i][q] = 0u;
                }
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    uint32_t va[4];
                    va[0] = widen_pair<FMT>(v[0][j / 2], v[1][j / 2], j % 2 * 2), va[1] = widen_pair<FMT>(v[0][j / 2], v[1][j / 2], j % 2 * 2 + 1);
                    va[2] = widen_pair<FMT>(v[2][j / 2], v[3][j / 2], j % 2 * 2), va[3] = widen_pair<FMT>(v[2][j / 2], v[3][j / 2], j % 2 * 2 + 1);
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt) mma16816(o[qt][j], va, w[qt].x, w[qt].y);
                }
            }
            if (!ok)  // a wait ran out: every load that was asked for lands before the CTA exits
                for (int i = 0; i < NS; ++i) wait_bar_drain(full(i), (uint32_t)(i >= stage ? phase : phase ^ 1u), 20000000ull);
            if constexpr (!Lay::kQInRegs) __syncthreads();  // (the rings of all warps have been read)
#pragma unroll
            for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) l[qt][f] += __shfl_xor_sync(0xffffffffu, l[qt][f], w);
            // (seen: the same rows in lanes of the same t)
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) seen |= __shfl_xor_sync(0xffffffffu, seen, w);

            // ------------------------------------------------------------ the CTA's warps joined
            constexpr int P = HD + 4;  // pitch of a row of sums
            auto sums = [&](int w, int r) { return reinterpret_cast<float*>(smem + w * Lay::kArea) + r * P; };
            auto stat = [&](int w, int r) { return reinterpret_cast<float4*>(smem + w * Lay::kArea + Lay::kSums) + r; };
            __syncwarp();
#pragma unroll
            for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const int r = 8 * qt + 2 * t + f;
                    float* d = sums(warp, r) + g * (4 * VW);
#pragma unroll
                    for (int j = 0; j < MT; ++j) *reinterpret_cast<float2*>(d + 2 * j) = make_float2(o[qt][j][f], o[qt][j][2 + f]);
                    if (g == 0)  // (this warp's part)
                        *stat(warp, r) =
                            make_float4(nx[qt][f] == kNoMax ? kNone : -nx[qt][f], nb[qt][f] == kNoMax ? kNone : -nb[qt][f], l[qt][f],
                                        seen >> (2 * qt + f) & 1 ? 1.f : 0.f);
                }
            group_sync();
            const bool whole = piece.pieces == 1;
            // A row's maxima over the warps, and f(w) what warp w's sums are multiplied by: max a, max b less it, sum of weights, seen.
            auto over_warps = [&](int r, auto factor) {
                float4 m = make_float4(kNone, kNone, 0.f, 0.f);
#pragma unroll 4
                for (int w = group * W; w < group * W + W; ++w) {
                    const float4 st = *stat(w, r);
                    m.x = fmaxf(m.x, st.x), m.w = fmaxf(m.w, st.w);
                }
#pragma unroll 4
                for (int w = group * W; w < group * W + W; ++w) {
                    const float4 st = *stat(w, r);
                    m.y = fmaxf(m.y, less(st.y, st.x, m.x));
                }
                const float na = m.x == kNone ? 0.f : -m.x, nm = m.y == kNone ? 0.f : -m.y;
#pragma unroll 4
                for (int w = group * W; w < group * W + W; ++w) {
                    const float4 st = *stat(w, r);
                    m.z += st.z * ex2(st.x + na);
                    factor(w, ex2(less(st.y, st.x, m.x) + nm));
                }
                return m;
            };
            auto add = [&](float4& v, int w, int r, int ch, float f) {
                const float4 d = *reinterpret_cast<const float4*>(sums(w, r) + ch);
                v.x = fmaf(d.x, f, v.x), v.y = fmaf(d.y, f, v.y), v.z = fmaf(d.z, f, v.z), v.w = fmaf(d.w, f, v.w);
            };
            auto put = [&](const float4& v, int r, int ch, const float2& f) {
                if (ch >= p.head_dim) return;
                uint2 y = make_uint2(0u, 0u);
                if (f.y == 0.f) y = make_uint2(Ops::pack(v.x * f.x, v.y * f.x), Ops::pack(v.z * f.x, v.w * f.x));
                *reinterpret_cast<uint2*>(row_at(p, s.row0, piece.head, r0 + r) + ch) = y;
            };
            auto part = [&](int r, int ch) { return reinterpret_cast<float4*>(p.part + ((long long)piece.slot * M + r) * HD + ch); };
            auto part_stat = [&](int r) {
                return reinterpret_cast<float4*>(p.part + (long long)slots(kResident) * M * HD + ((long long)piece.slot * M + r) * 4);
            };
            if constexpr (QT == 1) {
                // (a thread has four channels of one row at 128 channels: it finds the row's maxima for itself)
                for (int i = own * 32 + lane; i < rows * (HD / 4); i += 32 * W) {
                    const int r = i / (HD / 4), ch = i % (HD / 4) * 4;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    const float4 m = over_warps(r, [&](int w, float f) { add(v, w, r, ch, f); });
                    if (whole) {
                        put(v, r, ch, finish(m.y, m.z, m.w));
                    } else {
                        *part(r, ch) = v;
                        if (ch == 0) *part_stat(r) = m;
                    }
                }
            } else {
                // (of more rows, once a row: the factors in place of the warps' maxima, what finishes the row behind the first. Both sides, us:
                // four contexts of 5700 with 32 rows 43.0 and 42.2, with one row to a sequence 64 of 8192 225 and 235.)
                for (int r = own * 32 + lane; r < rows; r += 32 * W) {
                    const float4 m = over_warps(r, [&](int w, float f) { stat(w, r)->x = f; });
                    const float2 f = finish(m.y, m.z, m.w);
                    stat(group * W, r)->y = f.x, stat(group * W, r)->z = f.y;
                    if (!whole) *part_stat(r) = m;
                }
                group_sync();
                for (int i = own * 32 + lane; i < rows * (HD / 4); i += 32 * W) {
                    const int r = i / (HD / 4), ch = i % (HD / 4) * 4;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int w = group * W; w < group * W + W; ++w) add(v, w, r, ch, stat(w, r)->x);
                    const float4 f = *stat(group * W, r);
                    if (whole) put(v, r, ch, make_float2(f.y, f.z));
                    else *part(r, ch) = v;
                }
            }
        }
        // the sums have been read before the next round's loads overwrite them
        fence_proxy_async_smem();
        if (!__syncthreads_and(ok)) break;
    }
}

struct Plan {
    int hd, qt, group;
    int tile;         // rows of a row block of the kernel for many rows, or 0
    int box_log;      // log2 of the positions of a TMA box: as many as a page holds whole numbers of, 16 at most
    bool tma;
    long long units;  // row blocks and heads at most
    bool split;       // whether a sequence can be long enough to be split
    int rows() const { return tile ? tile : 8 * qt; }
    int resident() const { return tile ? kTileResident : kResident; }
};
Plan plan_of(const fl_kv_attend_desc* d) {
    Plan p;
    p.group = d->heads_q / d->heads_k;
    p.hd = d->head_dim <= 64 ? 64 : d->head_dim <= 128 ? 128 : 256;
    // tiles for the rows of a sequence, 1, 2 or 4 of them (at 256 channels registers hold two): what does
    // not fit is another row block, which reads the codes again
    const long long each = d->cu_rows == nullptr ? p.group : ((long long)d->rows + d->n_seqs - 1) / d->n_seqs * p.group;
    p.qt = each <= 8 ? 1 : each <= 16 || p.hd == 256 ? 2 : 4;
    p.box_log = 0;
    while (p.box_log < 4 && d->page_size % (2 << p.box_log) == 0) ++p.box_log;
    // (a box starts on 128 bytes of shared memory: two positions of 64 channels)
    p.tma = d->head_dim % 16 == 0 && (p.hd > 64 || p.box_log > 0);
    p.tile = each > kRowsLimit && (long long)d->table_pages * d->page_size >= kLongTable && p.hd <= 128 && p.tma ? (each <= 128 ? 128 : 256) : 0;
    const long long seqs = d->rows < d->n_seqs ? d->rows : d->n_seqs, M = p.rows();
    p.units = d->cu_rows == nullptr ? seqs * ((p.group + M - 1) / M) * d->heads_k
                                    : (((long long)d->rows * p.group + (M - 1) * seqs) / M) * d->heads_k;
    p.split = (long long)d->table_pages * d->page_size > (long long)kWorth * kTile;
    return p;
}
size_t workspace_of(const Plan& p) {
    return p.split ? part_bytes(p.resident(), p.rows(), p.hd) + sizeof(Units) : 0;
}

fl_status check_sizes(const fl_kv_attend_desc* d) {
    using host::fail;
    const char* what = "fl_kv_attend";
    if (d == nullptr) return fail(FL_ERR_INVALID_ARG, "%s: null description", what);
    if (!host::valid_dtype(d->dtype)) return fail(FL_ERR_INVALID_ARG, "%s: bad dtype %d", what, (int)d->dtype);
    if (d->format != FL_KV_INT8 && d->format != FL_KV_E4M3)
        return fail(FL_ERR_INVALID_ARG, "%s: bad cache format %d", what, (int)d->format);
    if (d->rows < 0 || d->heads_q < 1 || d->heads_k < 1 || d->head_dim < 1 || d->page_size < 1 || d->n_pages < 1 ||
        d->n_seqs < 1 || d->table_pages < 1)
        return fail(FL_ERR_INVALID_ARG, "%s: sizes must be positive (rows may be 0)", what);
    if (d->heads_q % d->heads_k != 0)
        return fail(FL_ERR_INVALID_ARG, "%s: heads_q (%d) must be a multiple of heads_k (%d)", what, d->heads_q, d->heads_k);
    if (d->head_dim % 8 != 0) return fail(FL_ERR_ALIGNMENT, "%s: head_dim must be a multiple of 8 (%d)", what, d->head_dim);
    if (d->head_dim > 256) return fail(FL_ERR_UNSUPPORTED, "%s: head_dim above 256 (%d)", what, d->head_dim);
    if (d->n_seqs > 1 << 30) return fail(FL_ERR_UNSUPPORTED, "%s: more than 2^30 sequences", what);
    // (512: the kernels count row blocks of up to 256 rows, the last of them filled up, in 32 bits)
    if ((long long)d->rows * (d->heads_q / d->heads_k) > (1ll << 31) - 1 - 512 || plan_of(d).units + slots(kResident) >= (1ll << 31))
        return fail(FL_ERR_UNSUPPORTED, "%s: too many rows", what);
    return FL_OK;
}

fl_status run(const fl_kv_attend_desc* d, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    using host::fail;
    const char* what = "fl_kv_attend";
    fl_status st = check_sizes(d);
    if (st != FL_OK) return st;
    if (!(d->scale > 0.f) || d->scale > 1e30f) return fail(FL_ERR_INVALID_ARG, "%s: scale must be positive and finite", what);
    if (d->table_stride < 0 || (d->n_seqs > 1 && d->table_stride < d->table_pages))
        return fail(FL_ERR_INVALID_ARG, "%s: table_stride below table_pages", what);
    if (d->tree != nullptr && (d->tree_cols < 0 || d->tree_stride < 0 || (d->rows > 1 && d->tree_stride < d->tree_cols)))
        return fail(FL_ERR_INVALID_ARG, "%s: tree_stride below tree_cols", what);
    if (d->rows == 0) return host::ok();
    if ((st = host::check_ptr("q", d->q, true)) != FL_OK) return st;
    if ((st = host::check_ptr("out", d->out, true)) != FL_OK) return st;
    if ((st = host::check_ptr("k_cache", d->k_cache, true)) != FL_OK) return st;
    if ((st = host::check_ptr("v_cache", d->v_cache, true)) != FL_OK) return st;
    if ((st = host::check_ptr("k_scale", d->k_scale, true)) != FL_OK) return st;
    if ((st = host::check_ptr("v_scale", d->v_scale, true)) != FL_OK) return st;
    if ((st = host::check_ptr("workspace", workspace, false)) != FL_OK) return st;
    if (d->page_table == nullptr || d->start == nullptr)
        return fail(FL_ERR_INVALID_ARG, "%s: page_table and start must not be null", what);
    const uintptr_t words = reinterpret_cast<uintptr_t>(d->page_table) | reinterpret_cast<uintptr_t>(d->cu_rows) |
                            reinterpret_cast<uintptr_t>(d->start);
    if (words & 3u) return fail(FL_ERR_ALIGNMENT, "page_table, cu_rows and start must be 4-byte aligned");
    if ((st = host::check_heads(what, "q", d->rows, d->heads_q, d->head_dim, d->q_row, d->q_head, false)) != FL_OK) return st;
    if ((st = host::check_heads(what, "out", d->rows, d->heads_q, d->head_dim, d->out_row, d->out_head, true)) != FL_OK) return st;
    const Plan plan = plan_of(d);
    const size_t need = workspace_of(plan);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return fail(FL_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", what, need, workspace_bytes);
    const size_t places = (size_t)d->n_pages * d->page_size * d->heads_k;
    const struct { const void* p; size_t n; bool out; } all[] = {
        {d->out, host::span_heads(d->rows, d->heads_q, d->head_dim, d->out_row, d->out_head), true},
        {workspace, need, true},
        {d->q, host::span_heads(d->rows, d->heads_q, d->head_dim, d->q_row, d->q_head), false},
        {d->k_cache, places * d->head_dim, false},
        {d->v_cache, places * d->head_dim, false},
        {d->k_scale, places * 4, false},
        {d->v_scale, places * 4, false},
        {d->page_table, ((size_t)(d->n_seqs - 1) * d->table_stride + d->table_pages) * 4, false},
        {d->cu_rows, ((size_t)d->n_seqs + 1) * 4, false},
        {d->start, (size_t)d->n_seqs * 4, false},
        {d->tree, d->tree == nullptr ? 0 : (size_t)(d->rows - 1) * d->tree_stride + d->tree_cols, false}};
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < (int)(sizeof(all) / sizeof(all[0])); ++j) {
            if (i == 0 && j == 2 && host::apart(d->out, d->out_row, (d->heads_q - 1) * d->out_head + d->head_dim, d->q,
                                                d->q_row, (d->heads_q - 1) * d->q_head + d->head_dim, 2))
                continue;
            if (all[i].p != nullptr && all[i].n > 0 && host::overlap(all[i].p, all[i].n, all[j].p, all[j].n))
                return fail(FL_ERR_INVALID_ARG, "%s: an output or the workspace overlaps another tensor of the call", what);
        }
    host::LaunchContext ctx;
    if ((st = host::launch_context(stream, &ctx)) != FL_OK) return st;
    AttendParams p = {};
    p.q = static_cast<const uint16_t*>(d->q), p.out = static_cast<uint16_t*>(d->out);
    p.q_row = d->q_row, p.q_head = d->q_head, p.o_row = d->out_row, p.o_head = d->out_head;
    p.cache[0] = static_cast<const uint8_t*>(d->k_cache), p.cache[1] = static_cast<const uint8_t*>(d->v_cache);
    p.scale[0] = d->k_scale, p.scale[1] = d->v_scale;
    p.page_table = d->page_table, p.cu_rows = d->cu_rows, p.start = d->start;
    p.tree = d->tree, p.tree_stride = d->tree_stride, p.tree_cols = d->tree_cols, p.table_stride = d->table_stride;
    p.rows = d->rows, p.heads = d->heads_k, p.group = plan.group, p.head_dim = d->head_dim, p.page_size = d->page_size;
    p.page_shift = (d->page_size & (d->page_size - 1)) == 0 ? __builtin_ctz((unsigned)d->page_size) : -1;
    p.n_pages = d->n_pages, p.n_seqs = d->n_seqs, p.table_pages = d->table_pages;
    p.log2_scale = d->scale * 1.44269504088896341f;
    p.part = plan.split ? static_cast<float*>(workspace) : nullptr;
    p.range = ctx.range, p.status = ctx.status, p.timeout_ns = ctx.timeout_ns;
    p.box_log = plan.box_log;
    if (plan.tma)
        for (int w = 0; w < 2; ++w)
            if ((st = host::encode_pages(&p.tm[w], w == 0 ? d->k_cache : d->v_cache, d->head_dim, d->heads_k, d->page_size,
                                         d->n_pages, plan.hd == 64 ? 64 : 128, 1u << p.box_log, plan.tile == 0)) != FL_OK)
                return st;
    if (plan.tile) {
        int launches = 0;
        const cudaError_t e = launch_tile(p, d->dtype, d->format, plan.hd, plan.tile, plan.units, plan.split, ctx, stream, &launches);
        st = host::launched(e, what);
        if (st == FL_OK && launches > 1) st = host::launched(cudaSuccess, what);  // (counted)
        return st;
    }
    // (L is T / kResident at least: that many pieces more than units at most)
    const long long most = plan.units + (plan.split ? kResident : 0);
    const dim3 grid((unsigned)std::min<long long>(most, (long long)ctx.sms * (plan.hd <= 128 && plan.qt <= 2 ? 2 : 1)));
    const dim3 join_grid((unsigned)std::min<long long>(ctx.sms * 4ll, plan.units * 8 * plan.qt));
    auto both = [&](auto dt, auto fmt, auto hd, auto qt, auto by_tma) -> fl_status {
        constexpr int DT = decltype(dt)::value, FMT = decltype(fmt)::value, HD = decltype(hd)::value, QT = decltype(qt)::value;
        constexpr bool TMA = decltype(by_tma)::value;
        static std::atomic<unsigned long long> done{0};
        constexpr int bytes = Layout<HD, QT>::kSmem;
        static_assert(bytes <= 227 * 1024 / Layout<HD, QT>::kCtas - 1024, "shared memory of the resident CTAs");
        cudaError_t e = host::allow_smem(fl_kv_attend_kernel<DT, FMT, HD, QT, TMA>, bytes, ctx.device, done);
        if (e != cudaSuccess) return host::fail(FL_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
        e = host::launch(fl_kv_attend_kernel<DT, FMT, HD, QT, TMA>, grid, kThreads, bytes, ctx.pdl, stream, p);
        const fl_status s = host::launched(e, what);
        if (s != FL_OK || !plan.split) return s;
        e = host::launch(fl_kv_attend_join_kernel<DT, HD, kResident, 8 * QT>, join_grid, kJoinThreads, 0, ctx.pdl, stream, p);
        return host::launched(e, what);
    };
    using std::integral_constant;
    auto by_rows = [&](auto dt, auto fmt, auto hd, auto by_tma) {
        if (plan.qt == 1) return both(dt, fmt, hd, integral_constant<int, 1>(), by_tma);
        if constexpr (decltype(hd)::value <= 128) {
            if (plan.qt == 4) return both(dt, fmt, hd, integral_constant<int, 4>(), by_tma);
        }
        return both(dt, fmt, hd, integral_constant<int, 2>(), by_tma);
    };
    auto by_copies = [&](auto dt, auto fmt, auto hd) {
        return plan.tma ? by_rows(dt, fmt, hd, std::true_type()) : by_rows(dt, fmt, hd, std::false_type());
    };
    auto by_size = [&](auto dt, auto fmt) {
        return plan.hd == 64    ? by_copies(dt, fmt, integral_constant<int, 64>())
               : plan.hd == 128 ? by_copies(dt, fmt, integral_constant<int, 128>())
                                : by_copies(dt, fmt, integral_constant<int, 256>());
    };
    if (d->dtype == FL_F16)
        return d->format == FL_KV_INT8 ? by_size(integral_constant<int, DT_F16>(), integral_constant<int, FL_KV_INT8>())
                                       : by_size(integral_constant<int, DT_F16>(), integral_constant<int, FL_KV_E4M3>());
    return d->format == FL_KV_INT8 ? by_size(integral_constant<int, DT_BF16>(), integral_constant<int, FL_KV_INT8>())
                                   : by_size(integral_constant<int, DT_BF16>(), integral_constant<int, FL_KV_E4M3>());
}

}  // namespace

}  // namespace fl

extern "C" size_t fl_kv_attend_workspace_size(const fl_kv_attend_desc* desc) {
    return fl::check_sizes(desc) != FL_OK ? 0 : fl::workspace_of(fl::plan_of(desc));
}

extern "C" fl_status fl_kv_attend(const fl_kv_attend_desc* desc, void* workspace, size_t workspace_bytes, void* stream) {
    return fl::run(desc, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}
