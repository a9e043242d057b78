// What the kernels of attention over the paged cache share: their arguments, the
// division of the work into pieces, and the arithmetic of a row.
#pragma once

#include <cuda_fp16.h>

#include "fl_attn_mma.cuh"
#include "fl_host.h"

namespace fl {
namespace attend {

constexpr int kStep = 16;     // positions of a warp's step in the kernel for few rows
constexpr int kTile = 128;    // positions of a tile
constexpr int kLeast = 2;     // tiles of a piece at least
constexpr int kStart = 3, kJoin = 3;  // tiles that a piece's start and end, and the second launch, take as long as
constexpr int kWorth = kLeast + kJoin - 1;  // tiles of a sequence up to which a split gains less than the second launch costs
constexpr float kLazy = 8.f;  // a maximum is moved once it is exceeded by 2^8
// The kernel for many rows forms an exponent less its maximum with one rounding. Once the maximum is 2^20 in size its own rounding
// would show in that, as 2^4 and more from 2^28 on, which a weight cannot hold: it then rounds the exponent, as the maximum was, first.
constexpr float kLarge = 0x1p20f;

// Pieces of split sequences at most, with `resident` CTAs at work at once: L is T /
// resident at least, and each piece has more than L / 2 tiles.
constexpr int slots(int resident) { return 2 * resident; }
constexpr int kMostUnits = 304;  // row blocks and heads of split sequences at most: half of the slots

struct AttendParams {
    CUtensorMap tm[2];  // k_cache, v_cache: boxes of 64 or 128 channels of box_rows positions of one head and page
    const uint16_t* q;
    uint16_t* out;
    long long q_row, q_head, o_row, o_head;
    const uint8_t* cache[2];
    const float* scale[2];
    const int* page_table;
    const int* cu_rows;
    const int* start;
    const uint8_t* tree;
    long long table_stride, tree_stride;
    int tree_cols;
    int rows, heads, group, head_dim, page_size, page_shift, n_pages, n_seqs, table_pages;
    int box_log;       // log2 of box_rows
    float log2_scale;  // scale * log2(e)
    float* part;       // [slots][M][HD] sums, [slots][M][4] the two maxima, sum of weights, whether a position was seen; Units
    int* range;
    int* status;
    unsigned long long timeout_ns;
};

// What the second launch joins.
struct Unit {
    int row0, n, first, head, pieces, slot, step, unused;  // the sequence's rows; the block's first row; slots from one piece to the next
};
struct Units {
    int count, unused[7];
    Unit unit[kMostUnits];
};
// Bytes of the sums and statistics of row blocks of M rows, behind which the units stand.
constexpr size_t part_bytes(int resident, int M, int hd) { return (size_t)slots(resident) * M * (hd + 4) * 4; }
template <int RESIDENT, int M, int HD>
__device__ __forceinline__ Units* units_of(const AttendParams& p) {
    return reinterpret_cast<Units*>(reinterpret_cast<uint8_t*>(p.part) + part_bytes(RESIDENT, M, HD));
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two codes as fp16. int8: in bytes 0 and 2 of x (the others are ignored): 1024 + 128 +
// code in the mantissa, less 1152. e4m3: in the low 16 bits, by the conversion
// instruction (moving the bits takes three logical operations, which are issued at half rate:
// 16 contexts of 3750 positions 44 -> 38 us).
template <int FMT>
__device__ __forceinline__ uint32_t widen(uint32_t x) {
    uint32_t r;
    if constexpr (FMT == FL_KV_INT8) {
        const uint32_t m = (x & 0x00ff00ffu) ^ 0x64806480u;
        asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(0x64806480u));
    } else {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(x));
    }
    return r;
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on the barrier when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// A sequence's share of the work.
struct Seq {
    int row0, n;         // its rows of q
    long long from;      // start: the position of its first row
    int keys;            // positions to be read: 0 .. keys - 1
    int blocks, tiles;   // row blocks of M, tiles of its keys
};
__device__ __forceinline__ Seq seq_of(const AttendParams& p, int b, int M) {
    Seq s;
    if (p.cu_rows == nullptr) {
        s.row0 = b;
        s.n = b < p.rows ? 1 : 0;
    } else {
        s.row0 = max(0, min(__ldg(p.cu_rows + b), p.rows));
        s.n = max(0, min(__ldg(p.cu_rows + b + 1), p.rows) - s.row0);
    }
    s.from = p.start != nullptr ? __ldg(p.start + b) : 0;
    const long long end = min(s.from + s.n, (long long)p.table_pages * p.page_size);
    s.keys = (int)max(0ll, min(end, 0x7fffff00ll));
    s.blocks = (s.n * p.group + M - 1) / M;
    s.tiles = (s.keys + kTile - 1) / kTile;
    return s;
}

struct Piece {
    int seq, block, head, k, pieces, slot;  // piece k of `pieces`; its place among the pieces of split sequences
    int units;                              // row blocks and heads of split sequences in front of this one's
};

// Candidates of L: T / RESIDENT times these, / 8, and no split at all. (More than 8
// makes room for the pieces that lengths which are no multiples of L leave over.)
constexpr int kCandidates = 5;
constexpr unsigned long long kTimes = 0x140e0b0908ull;  // 8, 9, 11, 14, 20 (as a number: a table would be loaded from memory)
constexpr uint32_t kWhole = 1u << 30;

// The pieces of all sequences, counted by all threads of a CTA of WARPS warps, for
// RESIDENT CTAs at work at once. Order: sequence,
// piece, row block, head, so that CTAs next to one another read the heads of the same positions.
template <int WARPS, int RESIDENT>
struct Pieces {
    static constexpr int kWarps = WARPS, kThreads = 32 * WARPS, kResident = RESIDENT;
    const AttendParams& p;
    int M, per, b0, b1;      // this thread's sequences
    Seq only;                // with one sequence to a thread it is read once
    uint32_t L;
    int W;                   // warps to a piece: 8, or less where no sequence is split
    uint32_t fn, fs, fu, n;  // pieces, slots and units in front of this thread's sequences; its pieces
    uint32_t units;          // of all split sequences
    Piece (*found)[kWarps];  // [2], in shared memory: the pieces of this round and the next, and their sequences
    Seq (*of)[kWarps];

    __device__ __forceinline__ Seq seq(int b) const { return per == 1 ? only : seq_of(p, b, M); }
    __device__ __forceinline__ uint32_t pieces(const Seq& s) const { return max(1u, ((uint32_t)s.tiles + L - 1) / L); }

    // few: whether pieces may be given to fewer warps than a CTA has
    __device__ __forceinline__ Pieces(const AttendParams& params, int rows, bool few) : p(params), M(rows) {
        __shared__ Piece pieces_at[2][kWarps];
        __shared__ Seq seqs_at[2][kWarps];
        found = pieces_at, of = seqs_at;
        if (threadIdx.x < kWarps) found[0][threadIdx.x].seq = -1;
        __shared__ unsigned long long sum_t[kWarps];
        __shared__ uint32_t top_t[kWarps], pieces_of[kWarps][kCandidates + 1];
        __shared__ uint32_t sum_n[kWarps], sum_s[kWarps], sum_u[kWarps];
        per = (p.n_seqs + kThreads - 1) / kThreads;
        b0 = min(p.n_seqs, (int)threadIdx.x * per), b1 = min(p.n_seqs, b0 + per);
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        unsigned long long t = 0;
        uint32_t top = 0;
        only.blocks = only.tiles = 0;
        for (int b = b0; b < b1; ++b) {
            only = seq_of(p, b, M);
            t += (unsigned long long)only.tiles * only.blocks * p.heads;
            if (only.blocks > 0) top = max(top, (uint32_t)only.tiles);
        }
        t = __reduce_add_sync(0xffffffffu, (uint32_t)t & 0xffffffu) +
            ((unsigned long long)__reduce_add_sync(0xffffffffu, (uint32_t)(t >> 24)) << 24);
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) sum_t[warp] = t, top_t[warp] = top;
        __syncthreads();
        t = 0, top = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t += sum_t[w], top = max(top, top_t[w]);
        L = kWhole;
        if (top > kWorth) {
            // Each lane's candidate, and what it costs: the rounds, times their longest piece and a start. (In
            // a loop: a CTA's first instructions come from far, so the fewer of them the better.)
            const int me = min(lane, kCandidates);
            const unsigned long long want = (t * (kTimes >> 8 * me & 0xff) + 8 * kResident - 1) / (8 * kResident);
            const uint32_t mine = me == kCandidates ? kWhole : (uint32_t)max((unsigned long long)kLeast, min(want, (unsigned long long)kWhole));
            const float inv = __frcp_rn((float)mine);
#pragma unroll 1
            for (int c = 0; c <= kCandidates; ++c) {
                const float by = __shfl_sync(0xffffffffu, inv, c);
                uint32_t k = 0;
                for (int b = b0; b < b1; ++b) {
                    const Seq s = seq(b);
                    // (an estimate: the quotient is not exact next to a whole number)
                    k += (uint32_t)s.blocks * p.heads * (uint32_t)fmaxf(1.f, ceilf((float)s.tiles * by));
                }
                k = __reduce_add_sync(0xffffffffu, k);
                if (lane == 0) pieces_of[warp][c] = k;
            }
            __syncthreads();
            uint32_t cost = 0xffffffffu;
            if (lane <= kCandidates) {
                uint32_t all = 0;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) all += pieces_of[w][me];
                cost = (all + kResident - 1) / kResident * (min(mine, top) + kStart) + (mine < top ? kJoin : 0);
            }
            const int who = __ffs(__ballot_sync(0xffffffffu, cost == __reduce_min_sync(0xffffffffu, cost))) - 1;
            L = __shfl_sync(0xffffffffu, mine, who);
            if (L >= top) L = kWhole;
        }
        uint32_t sl = 0, un = 0;
        n = 0;
        for (int b = b0; b < b1; ++b) {
            const Seq s = seq(b);
            const uint32_t u = (uint32_t)s.blocks * p.heads, k = pieces(s);
            n += u * k;
            if (k > 1) sl += u * k, un += u;
        }
        fn = n, fs = sl, fu = un;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t a = __shfl_up_sync(0xffffffffu, fn, o);
            if (lane >= o) fn += a;
        }
        if (L != kWhole) {
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t c = __shfl_up_sync(0xffffffffu, fs, o), d = __shfl_up_sync(0xffffffffu, fu, o);
                if (lane >= o) fs += c, fu += d;
            }
        }
        if (lane == 31) sum_n[warp] = fn, sum_s[warp] = fs, sum_u[warp] = fu;
        fn -= n, fs -= sl, fu -= un;
        __syncthreads();
        units = 0;
        uint32_t all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) fn += sum_n[w], fs += sum_s[w], fu += sum_u[w];
            units += sum_u[w], all += sum_n[w];
        }
        W = kWarps;
        if (few && L == kWhole) {
            // of 8, 4, 2 and 1 warps to a piece, the least rounds * (steps, a start and the joining)
            const uint32_t w = kWarps >> (lane & 3), at_once = kResident * (kWarps / w);
            const uint32_t c = (all + at_once - 1) / at_once * (top * (kWarps / w) + kStart + (3 - (lane & 3)));
            const int who = __ffs(__ballot_sync(0xffffffffu, c == __reduce_min_sync(0xffffffffu, c))) - 1;
            W = kWarps >> (who & 3);
        }
    }

    // This warp's piece of the CTA's turn-th round, and its sequence: seq -1 if there is
    // none; false if the CTA has none at all. (One barrier: the next round's writes
    // come after the barrier of this one's readers, two rounds apart.)
    __device__ __forceinline__ bool find(uint32_t turn, Piece& piece, Seq& s) const {
        const int per_cta = kWarps / W;
        const uint32_t first = (turn * gridDim.x + blockIdx.x) * per_cta;
        bool any = false;
        // (cleared a round ahead, so that this round's writers find it so)
        if (threadIdx.x < kWarps) found[(turn + 1) & 1][threadIdx.x].seq = -1;
        if (fn < first + per_cta && first < fn + n) {
            uint32_t f = fn, fslots = fs, funits = fu;
            for (int b = b0; b < b1 && f < first + per_cta; ++b) {
                const Seq sq = seq(b);
                const uint32_t u = (uint32_t)sq.blocks * p.heads, k = pieces(sq);
                for (uint32_t index = max(f, first); index < min(f + u * k, first + per_cta); ++index) {
                    const uint32_t rem = index - f, w = rem % u;
                    found[turn & 1][index - first] = Piece{b, (int)(w / p.heads), (int)(w % p.heads), (int)(rem / u), (int)k, (int)(fslots + rem), (int)(funits + w)};
                    of[turn & 1][index - first] = sq;
                    any = true;
                }
                f += u * k;
                if (k > 1) fslots += u * k, funits += u;
            }
        }
        if (!__syncthreads_or(any)) return false;
        const int at = (threadIdx.x >> 5) / W;
        piece = found[turn & 1][at];
        s = of[turn & 1][at];
        return true;
    }
};

// A row's state: the maximum a of the exponents x; the maximum b of x + log2 vs, the exponents of the values' weights, less a (so
// that it keeps its digits whatever the size of a); both -inf where there is none.
// b less another a, the largest of several parts.
__device__ __forceinline__ float less(float b, float a, float top) { return a == top ? b : b + (a - top); }
// What the sums of a row are multiplied by, 0 (and .y) for one that sees nothing.
// (0 / 0 where all scores are -inf)
__device__ __forceinline__ float2 finish(float b, float sum, float any) {
    return any == 0.f ? make_float2(0.f, 1.f) : make_float2(exp2f(b) / sum, 0.f);
}
// Row r (of q, and head of the group) of a sequence in the output.
__device__ __forceinline__ uint16_t* row_at(const AttendParams& p, int row0, int head, int r) {
    const int i = r / p.group, h = r - i * p.group;
    return p.out + (long long)(row0 + i) * p.o_row + (long long)(head * p.group + h) * p.o_head;
}

// The pieces of row blocks of split sequences joined, by CTAs of four warps: all four to a
// row of a small row block, each adding every fourth piece, or a row to each; always
// in the same order.
constexpr int kJoinThreads = 128;

template <int DT, int HD, int RESIDENT, int M>
__global__ void __launch_bounds__(kJoinThreads) fl_kv_attend_join_kernel(const __grid_constant__ AttendParams p) {
    using Ops = DTypeOps<DT>;
    constexpr int C = HD / 32, WR = M >= 128 ? 1 : 4, ROWS = 4 / WR;  // channels of a lane; warps of a row, rows of a CTA
    __shared__ float part[4][HD];
    griddep_wait();
    griddep_launch_dependents();
    const Units* all = units_of<RESIDENT, M, HD>(p);
    const int count = max(0, min(__ldcg(&all->count), slots(RESIDENT) / 2)) * (M / ROWS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part_of = warp % WR;
    const float kNone = __int_as_float(0xff800000);
    for (int at = blockIdx.x; at < count; at += gridDim.x) {
        const int4 u0 = __ldcg(reinterpret_cast<const int4*>(&all->unit[at / (M / ROWS)]));
        const int4 u1 = __ldcg(reinterpret_cast<const int4*>(&all->unit[at / (M / ROWS)]) + 1);
        const int row0 = u0.x, n = u0.y, block0 = u0.z, head = u0.w, pieces = u1.x, slot = u1.y;
        const int r = at % (M / ROWS) * ROWS + warp / WR;
        const long long step = u1.z;  // slots from one piece to the next
        // (records of a workspace that another call is writing at the same time stay harmless)
        const bool fits = row0 >= 0 && n >= 0 && row0 <= p.rows - n && block0 >= 0 && head >= 0 && head < p.heads && pieces > 0 &&
                          slot >= 0 && step > 0 && slot + (pieces - 1) * step < slots(RESIDENT);
        if (!fits || r >= n * p.group - block0) continue;  // (with four warps to a row, all of them)
        float a = kNone, b = kNone, sum = 0.f, any = 0.f, v[C] = {};
        const float* stat = p.part + (long long)slots(RESIDENT) * M * HD + ((long long)slot * M + r) * 4;
        const float* src = p.part + ((long long)slot * M + r) * HD + lane * C;
        // (the first pieces' sums are asked for together with the maxima that they will be weighed by)
        constexpr int U = M >= 128 ? 8 : 4;
        float2 x[U][C / 2];
        auto load = [&](int k, float2* d) {
#pragma unroll
            for (int e = 0; e < C / 2; ++e) d[e] = __ldcg(reinterpret_cast<const float2*>(src + k * step * M * HD) + e);
        };
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (part_of + WR * u < pieces) load(part_of + WR * u, x[u]);
        float4 mine = make_float4(kNone, kNone, 0.f, 0.f);
        for (int k = lane; k < pieces; k += 32) {
            const float4 st = __ldcg(reinterpret_cast<const float4*>(stat + k * step * M * 4));
            if (k < 32) mine = st;
            a = fmaxf(a, st.x), any = fmaxf(any, st.w);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            any = fmaxf(any, __shfl_xor_sync(0xffffffffu, any, o));
        }
        const float na = a == kNone ? 0.f : -a;
        sum = mine.z * ex2(mine.x + na);
        b = mine.y = less(mine.y, mine.x, a);
        for (int k = lane + 32; k < pieces; k += 32) {
            const float4 st = __ldcg(reinterpret_cast<const float4*>(stat + k * step * M * 4));
            sum += st.z * ex2(st.x + na);
            b = fmaxf(b, less(st.y, st.x, a));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
        }
        const float nb = b == kNone ? 0.f : -b;
        for (int k0 = part_of; k0 < pieces; k0 += WR * U) {
            if (k0 != part_of) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (k0 + WR * u < pieces) load(k0 + WR * u, x[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + WR * u;
                float mb = k < 32 ? __shfl_sync(0xffffffffu, mine.y, k) : kNone;
                if (k >= pieces) continue;
                if (k >= 32) {
                    const float2 st = __ldcg(reinterpret_cast<const float2*>(stat + k * step * M * 4));
                    mb = less(st.y, st.x, a);
                }
                const float f = ex2(mb + nb);
#pragma unroll
                for (int e = 0; e < C / 2; ++e) v[2 * e] = fmaf(x[u][e].x, f, v[2 * e]), v[2 * e + 1] = fmaf(x[u][e].y, f, v[2 * e + 1]);
            }
        }
        const float2 f = finish(b, sum, any);
        uint16_t* out = row_at(p, row0, head, block0 + r);
        if constexpr (WR == 1) {
            if (lane * C < p.head_dim) {
#pragma unroll
                for (int e = 0; e < C; e += 2)
                    *reinterpret_cast<uint32_t*>(out + lane * C + e) = f.y != 0.f ? 0u : Ops::pack(v[e] * f.x, v[e + 1] * f.x);
            }
        } else {
#pragma unroll
            for (int e = 0; e < C; ++e) part[warp][lane * C + e] = v[e];
            __syncthreads();
            if (threadIdx.x * 2 < p.head_dim) {
                const int ch = threadIdx.x * 2;
                float y[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) y[e] = (part[0][ch + e] + part[1][ch + e]) + (part[2][ch + e] + part[3][ch + e]);
                *reinterpret_cast<uint32_t*>(out + ch) = f.y != 0.f ? 0u : Ops::pack(y[0] * f.x, y[1] * f.x);
            }
            __syncthreads();
        }
    }
}

// Launches the kernel for many rows (fl_kv_attend_tile.cu), M 128 or 256 rows to a row block.
cudaError_t launch_tile(const AttendParams& p, int dt, int fmt, int hd, int M, long long units, bool split,
                        const host::LaunchContext& ctx, cudaStream_t stream, int* launches);
constexpr int kTileResident = 152;  // its CTAs at work at once
}  // namespace attend
}  // namespace fl
