// Attention of new tokens over the paged 8-bit cache (fl_kv_attend): a decode
// step, or the verification of a tree of drafted tokens.
//
//   out[i, h] = sum_p w v[p] / sum_p w,  w = 2^x,  x = scale log2(e) ks[p] (q[i, h] . kc[p]),  v[p] = vs[p] vc[p]
//
// over the positions p that row i sees. The codes kc, vc are what the MMAs
// multiply: both formats fit fp16 exactly (e4m3 times 2^-8: its bits moved), so no
// key or value is rounded; ks goes onto the fp32 scores, and vs into the weights
// of the second product, w vs = 2^(x + log2 vs), which have a running maximum of
// their own, so that they fill fp16's range whatever the scales are. Rounded are
// those weights (fp16, 2^-12 of each) and the output. bf16 rows of q are
// multiplied as fp16 times a power of two per row, which keeps their 8 bits down
// to 2^-28 of the row's largest value.
//
// The cache is read once and nothing is written but the output, so HBM bounds it:
// 2 head_dim + 8 bytes per position and key head, for all rows of a sequence
// and all query heads of the group, which are the 16 or 32 rows of one MMA tile.
// A warp takes 16 positions a step through a ring of its own in shared memory
// (cp.async, no barriers), converts the codes to MMA fragments in registers (channels
// and positions permuted so that 16-byte loads give whole fragments), and keeps
// its own maxima, sums and outputs; the warps of a CTA are joined in shared
// memory at the end.
//
// Long contexts are split: with T the number of 128-position tiles of all
// sequences and heads, pieces of L = max(kLeast, T / kPieces) tiles at most, each to
// a CTA, so that sequences of any lengths fill the GPU evenly. Every CTA finds
// its piece from the lengths, which only the GPU knows. Pieces of a split
// sequence are joined by a second launch, in order.
#include <cuda_fp16.h>

#include <type_traits>

#include "fl_common.cuh"
#include "fl_host.h"

namespace fl {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 16;               // positions of a warp's step
constexpr int kTile = kStep * kWarps;   // positions of a tile
constexpr int kPieces = 304;            // pieces aimed at: two CTAs on each of 152 multiprocessors
constexpr int kLeast = 2;               // tiles of a piece at least
constexpr int kSlots = 2 * kPieces;     // pieces of split sequences at most (each has more than L / 2 tiles)
constexpr float kLazy = 8.f;            // a maximum is moved once it is exceeded by 2^8

struct AttendParams {
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
    int vec8;          // 8-byte copies (head_dim not a multiple of 16)
    float log2_scale;  // scale * log2(e)
    float* part;       // [kSlots][M][HD] sums, then [kSlots][M][4]: both maxima and the sum of weights
    int* range;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two codes as fp16. int8: in bytes 0 and 2 of x (the others are ignored):
// 1024 + 128 + code in the mantissa, less 1152. e4m3: in bytes 1 and 3, the value
// times 2^-8: exponent and mantissa moved to their places.
template <int FMT>
__device__ __forceinline__ uint32_t widen(uint32_t x) {
    if constexpr (FMT == FL_KV_INT8) {
        const uint32_t m = (x & 0x00ff00ffu) ^ 0x64806480u;
        uint32_t r;
        asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(0x64806480u));
        return r;
    } else {
        return (x & 0x80008000u) | ((x >> 1) & 0x3f803f80u);
    }
}
// Codes 0 and 2, and 1 and 3, of a word.
template <int FMT>
__device__ __forceinline__ void widen_word(uint32_t w, uint32_t& even, uint32_t& odd) {
    even = widen<FMT>(FMT == FL_KV_INT8 ? w : w << 8);
    odd = widen<FMT>(FMT == FL_KV_INT8 ? w >> 8 : w);
}
// Code b of word lo and of word hi.
template <int FMT>
__device__ __forceinline__ uint32_t widen_pair(uint32_t lo, uint32_t hi, int b) {
    const uint32_t sel = FMT == FL_KV_INT8 ? (uint32_t)(b | (4 + b) << 8) : (uint32_t)(b << 4 | (4 + b) << 12);
    return widen<FMT>(__byte_perm(lo, hi, FMT == FL_KV_INT8 ? (uint32_t)(b | b << 4 | (4 + b) << 8 | (4 + b) << 12) : sel));
}
// the value of an e4m3 code times 2^-8 stands in the fragments
template <int FMT>
constexpr float kCodeUnit = FMT == FL_KV_INT8 ? 1.f : 256.f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
};

// The index-th piece (SPLIT: the index-th row block and head of a split
// sequence, with its first piece's slot); seq -1 if there are fewer. All threads
// of the CTA, which holds THREADS of them. Order: sequence, piece, row block, head.
template <bool SPLIT, int THREADS>
__device__ __forceinline__ Piece find_piece(const AttendParams& p, int index, int M) {
    __shared__ unsigned long long warp_sum[THREADS / 32];
    __shared__ Piece found;
    const int per = (p.n_seqs + THREADS - 1) / THREADS;
    const int b0 = min(p.n_seqs, (int)threadIdx.x * per), b1 = min(p.n_seqs, b0 + per);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned long long t = 0;
    for (int b = b0; b < b1; ++b) {
        const Seq s = seq_of(p, b, M);
        t += (unsigned long long)s.tiles * s.blocks * p.heads;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) warp_sum[warp] = t;
    if (threadIdx.x == 0) found.seq = -1;
    __syncthreads();
    t = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) t += warp_sum[w];
    const int L = (int)max((unsigned long long)kLeast, (t + kPieces - 1) / kPieces);
    __syncthreads();
    // pieces in the low half, slots in the high one, of this thread's sequences; then those in front of them
    auto count = [&](const Seq& s) {
        const unsigned long long n = (unsigned long long)s.blocks * p.heads * max(1, (s.tiles + L - 1) / L);
        return s.tiles > L ? n << 32 | n : n;
    };
    unsigned long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += count(seq_of(p, b, M));
    unsigned long long before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long up = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += up;
    }
    if (lane == 31) warp_sum[warp] = before;
    before -= mine;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    if (!SPLIT) {
        if ((uint32_t)before <= (uint32_t)index && (uint32_t)index < (uint32_t)(before + mine))
            for (int b = b0; b < b1; ++b) {
                const Seq s = seq_of(p, b, M);
                const unsigned long long c = count(s);
                if ((uint32_t)index < (uint32_t)(before + c)) {
                    const uint32_t rem = index - (uint32_t)before, units = (uint32_t)s.blocks * p.heads;
                    const uint32_t u = rem % units;
                    found = Piece{b, (int)(u / p.heads), (int)(u % p.heads), (int)(rem / units), max(1, (s.tiles + L - 1) / L),
                                  (int)(before >> 32) + (int)rem};
                    break;
                }
                before += c;
            }
    } else {
        // (rows of a split sequence are joined unit by unit: its first piece's slots)
        unsigned long long units = 0;
        for (int b = b0; b < b1; ++b) {
            const Seq s = seq_of(p, b, M);
            if (s.tiles > L) units += (unsigned long long)s.blocks * p.heads;
        }
        unsigned long long first = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long up = __shfl_up_sync(0xffffffffu, first, o);
            if (lane >= o) first += up;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = first;
        first -= units;
        __syncthreads();
        for (int w = 0; w < warp; ++w) first += warp_sum[w];
        if ((unsigned long long)index >= first && (unsigned long long)index < first + units)
            for (int b = b0; b < b1; ++b) {
                const Seq s = seq_of(p, b, M);
                const unsigned long long c = count(s);
                if (s.tiles > L) {
                    const unsigned long long n = (unsigned long long)s.blocks * p.heads;
                    if ((unsigned long long)index < first + n) {
                        const int u = (int)(index - first);
                        found = Piece{b, u / p.heads, u % p.heads, 0, (s.tiles + L - 1) / L, (int)(before >> 32) + u};
                        break;
                    }
                    first += n;
                }
                before += c;
            }
    }
    __syncthreads();
    return found;
}

// What the sums of a row are multiplied by, 0 (and .y) for one that sees nothing.
// (a = -inf where all scores are: 0 / 0)
template <int FMT>
__device__ __forceinline__ float2 finish(float a, float b, float sum, float any) {
    return any == 0.f ? make_float2(0.f, 1.f) : make_float2(exp2f(b - a) * kCodeUnit<FMT> / sum, 0.f);
}
// Channels ch .. ch + 7 of row r (of q, and head of the group) of a sequence.
template <typename Ops>
__device__ __forceinline__ void store_row(const AttendParams& p, const Seq& s, int head, int r, int ch, const float (&v)[8], float2 f) {
    const int i = r / p.group, h = r - i * p.group;
    uint16_t* d = p.out + (long long)(s.row0 + i) * p.o_row + (long long)(head * p.group + h) * p.o_head + ch;
    uint4 y = make_uint4(Ops::pack(v[0] * f.x, v[1] * f.x), Ops::pack(v[2] * f.x, v[3] * f.x), Ops::pack(v[4] * f.x, v[5] * f.x),
                         Ops::pack(v[6] * f.x, v[7] * f.x));
    if (f.y != 0.f) y = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(d) = y;
}

// 16-byte chunk c of row r of a ring stage: the places that the lanes of one
// load touch lie in different banks.
template <int HD>
__device__ __forceinline__ uint32_t place_k(int r, int c) {
    return (uint32_t)(r * HD + ((HD == 64 ? c : c ^ (r & 4)) << 4));
}
template <int HD>
__device__ __forceinline__ uint32_t place_v(int r, int c) {
    const int f = HD == 64 ? (r & 2) : HD == 128 ? (r & 3) << 1 : (r & 1) | (r & 2) << 1;
    return (uint32_t)(r * HD + ((c ^ f) << 4));
}

template <int HD>
constexpr int kStageBytes = 2 * kStep * HD + 2 * kStep * 4 + 16;  // codes of k and v, their scales, which positions are there
template <int HD>
constexpr int kStages = HD == 64 ? 4 : HD == 128 ? 3 : 3;
// (the ring, or what the warps leave to be joined: sums [warp][M][HD + 2], maxima and sums of weights [warp][M][4])
template <int HD, int MT>
constexpr int kJoinBytes = kWarps * 16 * MT * (HD + 2 + 4) * 4;
template <int HD, int MT>
constexpr int kRingBytes = kWarps * kStages<HD> * kStageBytes<HD>;
template <int HD, int MT>
constexpr bool kQInRegs = HD * MT <= 128;
template <int HD, int MT>
constexpr int kQBytes = kQInRegs<HD, MT> ? 0 : MT * (HD / 16) * 32 * 16;
template <int HD, int MT>
constexpr int kSmem = (kRingBytes<HD, MT> > kJoinBytes<HD, MT> ? kRingBytes<HD, MT> : kJoinBytes<HD, MT>) + kQBytes<HD, MT>;

// HD: head_dim rounded up to 64, 128 or 256. MT: blocks of 16 rows.
template <int DT, int FMT, int HD, int MT>
__global__ void __launch_bounds__(kThreads, HD * MT <= 128 ? 2 : 1) fl_kv_attend_kernel(const __grid_constant__ AttendParams p) {
    using Ops = DTypeOps<DT>;
    constexpr int M = 16 * MT, KS = HD / 16, NT = HD / 8, NS = kStages<HD>, VW = HD / 32;  // VW: words of v per lane and position
    extern __shared__ __align__(16) uint8_t smem[];
    griddep_wait();
    griddep_launch_dependents();
    const Piece piece = find_piece<false, kThreads>(p, blockIdx.x, M);
    if (piece.seq < 0) return;
    const Seq s = seq_of(p, piece.seq, M);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int r0 = piece.block * M, rows = min(M, s.n * p.group - r0);  // rows of this block: (row of q, head of the group)
    const int t0 = (int)((long long)s.tiles * piece.k / piece.pieces), t1 = (int)((long long)s.tiles * (piece.k + 1) / piece.pieces);
    const int k0 = t0 * kTile, k1 = min(s.keys, t1 * kTile);
    if (piece.k == 0 && threadIdx.x == 0 && s.from + s.n > (long long)p.table_pages * p.page_size)
        atomicCAS(p.range, 0, s.row0 + 1);

    // ------------------------------------------------------------ the warp's ring
    const uint32_t sbase = smem_u32(smem);
    const uint32_t ring = sbase + warp * NS * kStageBytes<HD>;
    if (p.head_dim < HD) {
        // channels past head_dim stay zero
        for (int i = threadIdx.x; i < kRingBytes<HD, MT> / 16; i += kThreads)
            reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
    }
    const int steps = k1 > k0 + warp * kStep ? (k1 - k0 - warp * kStep + kTile - 1) / kTile : 0;
    const int* table = p.page_table + piece.seq * p.table_stride;
    const long long row_bytes = (long long)p.heads * p.head_dim;
    auto page_row = [&](int pos, int& in_page) {
        const int j = p.page_shift >= 0 ? pos >> p.page_shift : (int)((uint32_t)pos / (uint32_t)p.page_size);
        in_page = pos - j * p.page_size;
        return j;
    };
    // the table's entry of this lane's position of a step, one step ahead
    int entry = -1, in_page = 0;
    auto look_up = [&](int step) {
        const int pos = k0 + warp * kStep + step * kTile + (lane & 15);
        entry = -2;
        if (step < steps && pos < k1) entry = __ldg(table + page_row(pos, in_page));
    };
    auto request = [&](int step, int stage) {
        const uint32_t dst = ring + stage * kStageBytes<HD>;
        if (step < steps) {
            const bool there = entry >= 0 && entry < p.n_pages;
            if (entry != -2 && !there) atomicCAS(p.range, 0, s.row0 + 1);
            const long long place = there ? (long long)entry * p.page_size + in_page : 0;
            const uint32_t bits = __ballot_sync(0xffffffffu, there) & 0xffffu;
            const long long head = place * p.heads + piece.head;
            cp_async4(dst + 2 * kStep * HD + lane * 4, (lane < 16 ? p.scale[0] : p.scale[1]) + head, there ? 4 : 0);
            if (lane == 0) asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + 2 * kStep * HD + 2 * kStep * 4), "r"(bits) : "memory");
            constexpr int C = HD / 16;  // chunks of a row
#pragma unroll
            for (int i = 0; i < kStep * C / 32; ++i) {
                const int r = (i * 32 + lane) / C, c = lane % C;
                const long long at = __shfl_sync(0xffffffffu, place, r) * row_bytes + piece.head * p.head_dim + c * 16;
                const bool full = bits >> r & 1;
                if (!p.vec8) {
                    if (c * 16 < p.head_dim) {
                        cp_async16(dst + place_k<HD>(r, c), p.cache[0] + (full ? at : 0), full ? 16 : 0);
                        cp_async16(dst + kStep * HD + place_v<HD>(r, c), p.cache[1] + (full ? at : 0), full ? 16 : 0);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (c * 16 + 8 * h < p.head_dim) {
                            cp_async8(dst + place_k<HD>(r, c) + 8 * h, p.cache[0] + (full ? at + 8 * h : 0), full ? 8 : 0);
                            cp_async8(dst + kStep * HD + place_v<HD>(r, c) + 8 * h, p.cache[1] + (full ? at + 8 * h : 0), full ? 8 : 0);
                        }
                }
            }
        }
        cp_commit();
    };
    look_up(0);
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) {
        request(i, i);
        look_up(i + 1);
    }

    // ------------------------------------------------------------ q as MMA fragments
    // Step ks = 4 h + w of the first product takes channels 64 h + 16 t + 4 w + {0, 2} and {1, 3} of lane t.
    uint32_t qf[kQInRegs<HD, MT> ? MT : 1][kQInRegs<HD, MT> ? KS : 1][4];
    uint8_t* const qs = smem + kSmem<HD, MT> - kQBytes<HD, MT>;
    auto q_of = [&](int r) {  // row r of the block
        const int i = (r0 + r) / p.group, h = (r0 + r) - i * p.group;
        return p.q + (long long)(s.row0 + i) * p.q_row + (long long)(piece.head * p.group + h) * p.q_head;
    };
    // bf16: the power of two that brings the row's largest value to 2^14 .. 2^15
    float up[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) up[mt][e] = 1.f;
    auto each_q = [&](auto f) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 16 * mt + 8 * e + g;
                const uint16_t* q = r < rows ? q_of(r) : nullptr;
#pragma unroll
                for (int h = 0; h < KS / 4; ++h)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const int c = 64 * h + 16 * t + 8 * v;
                        const uint4 x = q != nullptr && c < p.head_dim ? ldg_v4(q + c) : make_uint4(0u, 0u, 0u, 0u);
                        f(mt, e, 4 * h + 2 * v, x);
                    }
            }
    };
    if constexpr (DT == DT_BF16) {
        uint32_t top[MT][2] = {};
        each_q([&](int mt, int e, int, const uint4& x) {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) top[mt][e] = max(top[mt][e], max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
        });
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t m = max(top[mt][e], __shfl_xor_sync(0xffffffffu, top[mt][e], 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                // 2^(14 - e) for a largest value of 2^e to 2^(e + 1); rows without a finite, not tiny one stay as they are
                const int ex = (int)(m >> 7);
                if (ex > 0 && ex < 255) up[mt][e] = __uint_as_float((uint32_t)min(254, 127 + 14 + 127 - ex) << 23);
            }
    }
    const bool writes_q = kQInRegs<HD, MT> || warp == 0;
    if (writes_q)
        each_q([&](int mt, int e, int ks, const uint4& x) {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float2 lo = Ops::unpack(w[2 * i]), hi = Ops::unpack(w[2 * i + 1]);
                const uint32_t even = DTypeOps<DT_F16>::pack(lo.x * up[mt][e], hi.x * up[mt][e]);
                const uint32_t odd = DTypeOps<DT_F16>::pack(lo.y * up[mt][e], hi.y * up[mt][e]);
                if constexpr (kQInRegs<HD, MT>) {
                    qf[mt][ks + i][e] = even;
                    qf[mt][ks + i][2 + e] = odd;
                } else {
                    uint32_t* d = reinterpret_cast<uint32_t*>(qs) + ((mt * KS + ks + i) * 32 + lane) * 4;
                    d[e] = even;
                    d[2 + e] = odd;
                }
            }
        });
    if (!kQInRegs<HD, MT>) __syncthreads();
    float c[MT][2];  // onto q' . code
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) c[mt][e] = p.log2_scale * kCodeUnit<FMT> / up[mt][e];

    // ------------------------------------------------------------ the warp's positions
    const float kNone = __int_as_float(0xff800000);
    float mx[MT][2], mw[MT][2], nx[MT][2], nw[MT][2], l[MT][2], o[MT][NT][4];  // n*: minus the maxima, 0 where there is none yet
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) mx[mt][e] = mw[mt][e] = kNone, nx[mt][e] = nw[mt][e] = l[mt][e] = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][j][e] = 0.f;
    }
    bool seen[MT][2] = {};  // (which tells a row that sees nothing from one whose scores are all -inf)
    // this lane's rows: the row of q among the sequence's
    int qi[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) qi[mt][e] = min(r0 + 16 * mt + 8 * e + g, s.n * p.group - 1) / p.group;

    int stage = 0, ahead = NS - 1;
    for (int step = 0; step < steps; ++step) {
        cp_wait<NS - 2>();
        __syncwarp();
        request(step + NS - 1, ahead);
        look_up(step + NS);
        if (++ahead == NS) ahead = 0;
        const uint32_t src = ring + stage * kStageBytes<HD>;
        if (++stage == NS) stage = 0;
        const int pos0 = k0 + warp * kStep + step * kTile;

        // scores: positions t + 4 i, i = 2 nt + column
        float x[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[mt][nt][e] = 0.f;
        const int krow = (g >> 1) + 4 * (g & 1);
#pragma unroll
        for (int h = 0; h < KS / 4; ++h) {
            uint4 kv[2];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) kv[nt] = ld_shared_v4(src + place_k<HD>(krow + 8 * nt, 4 * h + t));
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t a[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if constexpr (kQInRegs<HD, MT>) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) a[mt][e] = qf[mt][4 * h + w][e];
                    } else {
                        const uint4 v = *reinterpret_cast<const uint4*>(qs + ((mt * KS + 4 * h + w) * 32 + lane) * 16);
                        a[mt][0] = v.x, a[mt][1] = v.y, a[mt][2] = v.z, a[mt][3] = v.w;
                    }
                }
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    uint32_t b0, b1;
                    widen_word<FMT>(w == 0 ? kv[nt].x : w == 1 ? kv[nt].y : w == 2 ? kv[nt].z : kv[nt].w, b0, b1);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) mma16816(x[mt][nt], a[mt], b0, b1);
                }
            }
        }
        // scales of the lane's four positions
        const uint32_t sc = src + 2 * kStep * HD;
        float ks[4], lv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ks[i] = ld_shared_f32(sc + 4 * (t + 4 * i));
            lv[i] = lg2(ld_shared_f32(sc + kStep * 4 + 4 * (t + 4 * i)));
        }
        const uint32_t bits = __float_as_uint(ld_shared_f32(sc + 2 * kStep * 4));
        const bool all = bits == 0xffffu && pos0 + kStep <= s.from;  // every row sees every position
        float y[MT][2][4];
        bool over = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 2 * nt + (e & 1);
                    float v = x[mt][nt][e] * c[mt][e >> 1] * ks[i], u = v + lv[i];
                    if (!all) {
                        const long long j = pos0 + t + 4 * i - s.from;
                        bool sees = bits >> (t + 4 * i) & 1;
                        if (sees && j >= 0) {
                            if (p.tree == nullptr) sees = j <= qi[mt][e >> 1];
                            else sees = j < p.tree_cols && __ldg(p.tree + (s.row0 + qi[mt][e >> 1]) * p.tree_stride + j) != 0;
                        }
                        if (!sees) v = u = kNone;
                        seen[mt][e >> 1] |= sees;
                    } else {
                        seen[mt][e >> 1] = true;
                    }
                    x[mt][nt][e] = v;
                    y[mt][nt][e] = u;
                    over |= v > mx[mt][e >> 1] + kLazy || u > mw[mt][e >> 1] + kLazy;
                }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float a = mx[mt][e], b = mw[mt][e];
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int f = 0; f < 2; ++f) a = fmaxf(a, x[mt][nt][2 * e + f]), b = fmaxf(b, y[mt][nt][2 * e + f]);
#pragma unroll
                    for (int w = 1; w < 4; w <<= 1) {
                        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, w));
                        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, w));
                    }
                    const float na = a == kNone ? 0.f : -a, nb = b == kNone ? 0.f : -b;
                    l[mt][e] *= ex2(mx[mt][e] + na);
                    const float f = ex2(mw[mt][e] + nb);
#pragma unroll
                    for (int j = 0; j < NT; ++j) o[mt][j][2 * e] *= f, o[mt][j][2 * e + 1] *= f;
                    mx[mt][e] = a, mw[mt][e] = b, nx[mt][e] = na, nw[mt][e] = nb;
                }
        }
        uint32_t w[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[mt][e] += ex2(x[mt][nt][2 * e] + nx[mt][e]) + ex2(x[mt][nt][2 * e + 1] + nx[mt][e]);
                    w[mt][2 * nt + e] = DTypeOps<DT_F16>::pack(ex2(y[mt][nt][2 * e] + nw[mt][e]), ex2(y[mt][nt][2 * e + 1] + nw[mt][e]));
                }
        // values: n tile j is channel j of the lane's 4 VW
        uint32_t v[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = t + 4 * i;
            if constexpr (VW == 2) {
                const uint32_t at = src + kStep * HD + place_v<HD>(r, g >> 1) + 8 * (g & 1);
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[i][0]), "=r"(v[i][1]) : "r"(at) : "memory");
            } else {
#pragma unroll
                for (int q = 0; q < VW / 4; ++q) {
                    const uint4 u = ld_shared_v4(src + kStep * HD + place_v<HD>(r, g * (VW / 4) + q));
                    v[i][4 * q] = u.x, v[i][4 * q + 1] = u.y, v[i][4 * q + 2] = u.z, v[i][4 * q + 3] = u.w;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t b0 = widen_pair<FMT>(v[0][j / 4], v[1][j / 4], j % 4), b1 = widen_pair<FMT>(v[2][j / 4], v[3][j / 4], j % 4);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma16816(o[mt][j], w[mt], b0, b1);
        }
    }
    cp_wait<0>();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int f = 1; f < 4; f <<= 1) {
                l[mt][e] += __shfl_xor_sync(0xffffffffu, l[mt][e], f);
                seen[mt][e] |= __shfl_xor_sync(0xffffffffu, (int)seen[mt][e], f) != 0;
            }
    __syncthreads();

    // ------------------------------------------------------------ the CTA's warps joined
    constexpr int P = HD + 2;  // pitch of a row of sums
    float* const sums = reinterpret_cast<float*>(smem);
    float* const stat = sums + kWarps * M * P;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 16 * mt + 8 * e + g;
            float* d = sums + (warp * M + r) * P;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                d[2 * t * (4 * VW) + j] = o[mt][j][2 * e];
                d[(2 * t + 1) * (4 * VW) + j] = o[mt][j][2 * e + 1];
            }
            if (t == 0) *reinterpret_cast<float4*>(stat + (warp * M + r) * 4) = make_float4(mx[mt][e], mw[mt][e], l[mt][e], seen[mt][e] ? 1.f : 0.f);
        }
    __syncthreads();
    const bool whole = piece.pieces == 1;
    for (int i = threadIdx.x; i < rows * (HD / 8); i += kThreads) {
        const int r = i / (HD / 8), ch = i % (HD / 8) * 8;
        float a = kNone, b = kNone, any = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 st = *reinterpret_cast<const float4*>(stat + (w * M + r) * 4);
            a = fmaxf(a, st.x), b = fmaxf(b, st.y), any = fmaxf(any, st.w);
        }
        const float na = a == kNone ? 0.f : -a, nb = b == kNone ? 0.f : -b;
        float sum = 0.f, v[8] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 st = *reinterpret_cast<const float4*>(stat + (w * M + r) * 4);
            sum += st.z * ex2(st.x + na);
            const float f = ex2(st.y + nb);
            const float* d = sums + (w * M + r) * P + ch;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf(d[e], f, v[e]);
        }
        if (whole) {
            if (ch < p.head_dim) store_row<Ops>(p, s, piece.head, r0 + r, ch, v, finish<FMT>(a, b, sum, any));
        } else {
            float* d = p.part + ((long long)piece.slot * M + r) * HD + ch;
            *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(d + 4) = make_float4(v[4], v[5], v[6], v[7]);
            if (ch == 0)
                *reinterpret_cast<float4*>(p.part + (long long)kSlots * M * HD + ((long long)piece.slot * M + r) * 4) =
                    make_float4(a, b, sum, any);
        }
    }
}

// The pieces of row blocks of split sequences joined: one CTA to four rows of a
// block and head, four warps to a row, each of which adds every fourth piece; always in the same order.
constexpr int kJoinThreads = 512;

template <int DT, int FMT, int HD, int MT>
__global__ void __launch_bounds__(kJoinThreads) fl_kv_attend_join_kernel(const __grid_constant__ AttendParams p) {
    using Ops = DTypeOps<DT>;
    constexpr int M = 16 * MT, C = HD / 32;  // channels of a lane
    __shared__ float part[16][HD];
    // (the lengths are older than the kernel in front, which waited for them itself before it let this one in)
    const Piece u = find_piece<true, kJoinThreads>(p, blockIdx.x, M);
    griddep_wait();
    griddep_launch_dependents();
    if (u.seq < 0) return;
    const Seq s = seq_of(p, u.seq, M);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * 4 + (warp >> 2), first = warp & 3, rows = min(M, s.n * p.group - u.block * M);
    const long long step = (long long)s.blocks * p.heads;  // slots from one piece to the next
    const float kNone = __int_as_float(0xff800000);
    float a = kNone, b = kNone, sum = 0.f, any = 0.f, v[C] = {};
    if (r < rows) {
        const float* stat = p.part + (long long)kSlots * M * HD + ((long long)u.slot * M + r) * 4;
        for (int k = lane; k < u.pieces; k += 32) {
            const float4 st = __ldcg(reinterpret_cast<const float4*>(stat + k * step * M * 4));
            a = fmaxf(a, st.x), b = fmaxf(b, st.y), any = fmaxf(any, st.w);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
            any = fmaxf(any, __shfl_xor_sync(0xffffffffu, any, o));
        }
        const float na = a == kNone ? 0.f : -a, nb = b == kNone ? 0.f : -b;
        for (int k = lane; k < u.pieces; k += 32) {
            const float4 st = __ldcg(reinterpret_cast<const float4*>(stat + k * step * M * 4));
            sum += st.z * ex2(st.x + na);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float* src = p.part + ((long long)u.slot * M + r) * HD + lane * C;
#pragma unroll 4
        for (int k = first; k < u.pieces; k += 4) {
            const float f = ex2(__ldcg(stat + k * step * M * 4 + 1) + nb);
            const float* d = src + k * step * M * HD;
#pragma unroll
            for (int e = 0; e < C; e += 2) {
                const float2 x = __ldcg(reinterpret_cast<const float2*>(d + e));
                v[e] = fmaf(x.x, f, v[e]);
                v[e + 1] = fmaf(x.y, f, v[e + 1]);
            }
        }
#pragma unroll
        for (int e = 0; e < C; ++e) part[warp][lane * C + e] = v[e];
    }
    __syncthreads();
    if (r >= rows || first != 0) return;
    const float2 f = finish<FMT>(a, b, sum, any);
    for (int ch = lane * 8; ch < p.head_dim; ch += 256) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (part[warp][ch + e] + part[warp + 1][ch + e]) + (part[warp + 2][ch + e] + part[warp + 3][ch + e]);
        store_row<Ops>(p, s, u.head, u.block * M + r, ch, x, f);
    }
}

struct Plan {
    int hd, mt, group;
    long long units;  // row blocks and heads at most
    bool split;       // whether a sequence can be long enough to be split
};
Plan plan_of(const fl_kv_attend_desc* d) {
    Plan p;
    p.group = d->heads_q / d->heads_k;
    p.hd = d->head_dim <= 64 ? 64 : d->head_dim <= 128 ? 128 : 256;
    // rows of a sequence: more than 16 fill two blocks (no registers for that at 256 channels)
    const long long each = d->cu_rows == nullptr ? p.group : ((long long)d->rows + d->n_seqs - 1) / d->n_seqs * p.group;
    p.mt = each > 16 && p.hd <= 128 ? 2 : 1;
    const long long seqs = d->rows < d->n_seqs ? d->rows : d->n_seqs, M = 16 * p.mt;
    p.units = d->cu_rows == nullptr ? seqs * ((p.group + M - 1) / M) * d->heads_k
                                    : ((long long)d->rows * p.group / M + seqs) * d->heads_k;
    p.split = (long long)d->table_pages * d->page_size > (long long)kLeast * kTile;
    return p;
}
size_t workspace_of(const Plan& p) { return p.split ? (size_t)kSlots * 16 * p.mt * (p.hd + 4) * 4 : 0; }

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
    if ((long long)d->rows * (d->heads_q / d->heads_k) >= (1ll << 31) - 64 || plan_of(d).units + kPieces >= (1ll << 31))
        return fail(FL_ERR_UNSUPPORTED, "%s: too many rows", what);
    return FL_OK;
}

fl_status attend(const fl_kv_attend_desc* d, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
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
    p.vec8 = d->head_dim % 16 != 0;
    p.log2_scale = d->scale * 1.44269504088896341f;
    p.part = static_cast<float*>(workspace);
    p.range = ctx.range;
    const dim3 grid((unsigned)(plan.units + (plan.split ? kPieces : 0)));
    const dim3 join_grid((unsigned)(plan.units < kPieces ? plan.units : kPieces), 4u * plan.mt);
    cudaError_t e = cudaErrorInvalidValue;
    auto both = [&](auto dt, auto fmt, auto hd, auto mt) -> fl_status {
        constexpr int DT = decltype(dt)::value, FMT = decltype(fmt)::value, HD = decltype(hd)::value, MT = decltype(mt)::value;
        static std::atomic<unsigned long long> done{0};
        constexpr int bytes = kSmem<HD, MT>;
        static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
        e = host::allow_smem(fl_kv_attend_kernel<DT, FMT, HD, MT>, bytes, ctx.device, done);
        if (e != cudaSuccess) return host::fail(FL_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
        e = host::launch(fl_kv_attend_kernel<DT, FMT, HD, MT>, grid, kThreads, bytes, ctx.pdl, stream, p);
        const fl_status s = host::launched(e, what);
        if (s != FL_OK || !plan.split) return s;
        e = host::launch(fl_kv_attend_join_kernel<DT, FMT, HD, MT>, join_grid, kJoinThreads, 0, ctx.pdl, stream, p);
        return host::launched(e, what);
    };
    auto by_size = [&](auto dt, auto fmt) {
        using std::integral_constant;
        if (plan.hd == 64) return plan.mt == 2 ? both(dt, fmt, integral_constant<int, 64>(), integral_constant<int, 2>())
                                               : both(dt, fmt, integral_constant<int, 64>(), integral_constant<int, 1>());
        if (plan.hd == 128) return plan.mt == 2 ? both(dt, fmt, integral_constant<int, 128>(), integral_constant<int, 2>())
                                                : both(dt, fmt, integral_constant<int, 128>(), integral_constant<int, 1>());
        return both(dt, fmt, integral_constant<int, 256>(), integral_constant<int, 1>());
    };
    using std::integral_constant;
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
    return fl::attend(desc, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}
