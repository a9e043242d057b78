// Dense layers on 4-bit weights (fl_w4_gemm, fl_w4_swiglu_ffn) and their
// quantiser (fl_w4_quantize).
//
//   out[m, n] = act(r[m] * sum_k x'[m, k] w[n, k] + bias[n]) (+ residual[m, n])
//   w[n, k]   = scale[n, k / G] * (code[n, k] - zero[n, k / G])
//
// with x' = x * gamma and r the RMSNorm row scale where there is a prologue
// (else x and 1). fl_w4_rows.cu computes few rows, fl_w4_tile.cu many.
//
// The quantiser is bound by HBM, 2.5 bytes a weight and 2 per group: 20.6 us at
// 11008 x 4096, group 128 (5.5 TB/s), where its lanes' arithmetic is next.
#include "fl_common.cuh"
#include "fl_host.h"
#include "fl_quant.cuh"
#include "fl_w4.h"

namespace fl {

namespace {

// ---------------------------------------------------------------------------
// quantiser
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 256;
constexpr int kQuantUnits = 2;  // units of 16 weights per lane in flight

// A code next to a tie: which side of lo + 1/2 the quotient lies is the sign of
// w - (lo + 1/2) s, one FMA (exact: both have at most 11 significant bits), and
// 0 is the tie, which goes to even. Returned as 8 + the integer.
__device__ __forceinline__ uint32_t code_exact(float w, float s, float inv) {
    const float lo = floorf(w * inv), d = fmaf(-(lo + 0.5f), s, w);
    if (fabsf(w * inv - (lo + 0.5f)) > 0.001f) return (uint32_t)(8 + (int)rintf(w * inv));
    return (uint32_t)(8 + (int)(d > 0.f ? lo + 1.f : d < 0.f ? lo : 2.f * rintf(0.5f * (lo + 0.5f))));
}

// Codes of 8 weights of a group, two to a byte. The quotient lies between
// w * dn and w * up (1 / s, within 2^-24 of it, times 1 -+ 2^-21), and rounding
// is monotonic: where both round to the same code it is the exact quotient's;
// the others (16-bit weights over 16-bit scales are ties now and then: one in some
// hundred) are decided exactly. Where the clamp or an overflowed 1 / s (a
// subnormal scale) may matter, the quotients are divided out: of two 16-bit
// values it is a tie or at least 2^-13 away from one, so fp32 division decides it.
// fma(w, up, 1.5 * 2^23 + 8) has 8 + the integer in its low bits, r_i = B +
// code_i, and sum_i r_i 16^i = 0x11111111 B + the packed word, modulo 2^32.
template <int DT>
__device__ __forceinline__ uint32_t codes8(const uint4& v, float s, float up, float dn, bool clamped) {
    using Ops = DTypeOps<DT>;
    constexpr float kShift = 12582912.0f + 8.0f;
    constexpr uint32_t kBase = 0x4b400000u;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4], d[4];  // 272 B + two codes, from above and from below
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = Ops::unpack(w[e]);
        c[e] = __float_as_uint(fmaf(f.y, up, kShift)) * 16u + __float_as_uint(fmaf(f.x, up, kShift));
        d[e] = __float_as_uint(fmaf(f.y, dn, kShift)) * 16u + __float_as_uint(fmaf(f.x, dn, kShift));
    }
    if (((c[0] ^ d[0]) | (c[1] ^ d[1]) | (c[2] ^ d[2]) | (c[3] ^ d[3])) != 0u) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (c[e] == d[e]) continue;
            const float2 f = Ops::unpack(w[e]);
            c[e] = (kBase + code_exact(f.y, s, up)) * 16u + (kBase + code_exact(f.x, s, up));
        }
    }
    uint32_t out = ((c[3] * 256u + c[2]) * 256u + c[1]) * 256u + c[0] - kBase * 0x11111111u;
    if (clamped) {
        out = 0;
#pragma unroll
        for (int e = 3; e >= 0; --e) {
            const float2 f = Ops::unpack(w[e]);
            out = out * 16u + (uint32_t)(8 + (int)fminf(fmaxf(rintf(__fdiv_rn(f.y, s)), -7.f), 7.f));
            out = out * 16u + (uint32_t)(8 + (int)fminf(fmaxf(rintf(__fdiv_rn(f.x, s)), -7.f), 7.f));
        }
    }
    return out;
}

// Groups are consecutive in W [N, K] taken as one array, so are their codes
// and scales: lane i of a warp takes the i-th unit of 16 weights, G / 16
// neighbouring lanes share a group. HBM moves 2.5 bytes per weight and a
// little, which leaves about 9 instructions a weight: the group's maximum, scale and
// reciprocal cost as much as the codes, so a lane takes two vectors for them.
template <int DT>
__global__ void __launch_bounds__(kQuantThreads)
    fl_w4_quantize_kernel(const uint16_t* __restrict__ W, uint32_t* __restrict__ q, uint16_t* __restrict__ scales,
                          long long units, int lanes_log) {
    using Ops = DTypeOps<DT>;
    griddep_wait();
    griddep_launch_dependents();
    const long long i0 = (long long)blockIdx.x * (kQuantThreads * kQuantUnits) + threadIdx.x;
    const uint4* src = reinterpret_cast<const uint4*>(W) + i0 * 2;
    uint4 v[kQuantUnits][2];
#pragma unroll
    for (int u = 0; u < kQuantUnits; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            v[u][e] = i0 + u * kQuantThreads < units ? __ldg(src + u * (2 * kQuantThreads) + e) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < kQuantUnits; ++u) {
        uint32_t m = absmax2<DT>(absmax8<DT>(v[u][0]), absmax8<DT>(v[u][1]));
        for (int o = 1 << lanes_log >> 1; o > 0; o >>= 1) m = absmax2<DT>(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (i0 + u * kQuantThreads >= units) continue;
        m = absmax_halves<DT>(m);
        const bool fine = m < Bits16<DT>::kInf;
        // (amax / 7 is never within 2^-13 of a border of the 16-bit format
        // without lying on it, so the fp32 product with 1 / 7, 2^-23 off at
        // most, rounds to the same 16 bits)
        const float amax = Ops::unpack(m).x;
        uint32_t sb = Ops::pack(amax * (1.0f / 7.0f), 0.f) & 0xffffu;
        if (sb == 0u) sb = 1u;  // smallest positive value
        const float s = Ops::unpack(sb).x, inv = rcp_approx(s), up = inv * (1.0f + 0x1p-21f), dn = inv * (1.0f - 0x1p-21f);
        const bool clamped = !(amax * inv < 7.4f);
        uint2 out = make_uint2(0x88888888u, 0x88888888u);
        if (fine) out = make_uint2(codes8<DT>(v[u][0], s, up, dn, clamped), codes8<DT>(v[u][1], s, up, dn, clamped));
        reinterpret_cast<uint2*>(q)[i0 + u * kQuantThreads] = out;
        if ((threadIdx.x & ((1 << lanes_log) - 1)) == 0)
            scales[(i0 + u * kQuantThreads) >> lanes_log] = fine ? (uint16_t)sb : (uint16_t)0x7fffu;
    }
}

fl_status check_weight(const char* name, const fl_w4_weight* w, long long N, long long K) {
    using host::fail;
    if (w == nullptr) return fail(FL_ERR_INVALID_ARG, "%s must not be null", name);
    if (w->group != 32 && w->group != 64 && w->group != 128)
        return fail(FL_ERR_INVALID_ARG, "%s: group must be 32, 64 or 128 (%d)", name, w->group);
    if (N < 1 || K < 1) return fail(FL_ERR_INVALID_ARG, "%s: sizes must be positive (N=%lld K=%lld)", name, N, K);
    // (tiles of rows and steps of k run past the ends before they are cut off: room for that below 2^31)
    if (N > 0x7fffff00ll) return fail(FL_ERR_UNSUPPORTED, "%s: too many rows (%lld)", name, N);
    if (K > 0x7ffff000ll) return fail(FL_ERR_UNSUPPORTED, "%s: rows too long (%lld)", name, K);
    if (N % 8 != 0 || K % w->group != 0)
        return fail(FL_ERR_ALIGNMENT, "%s: N must be a multiple of 8 and K of the group (N=%lld K=%lld group %d)", name,
                    N, K, w->group);
    fl_status st;
    if ((st = host::check_ptr(name, w->q, true)) != FL_OK) return st;
    if ((st = host::check_ptr(name, w->scales, true)) != FL_OK) return st;
    return host::check_ptr(name, w->zeros, false);
}

// Every tensor of one call: outputs overlap no input and no other output.
struct Ranges {
    struct R {
        const void* p;
        size_t n;
    } in[16];
    int n = 0;
    void add(const void* p, size_t bytes) { in[n++] = R{p, bytes}; }
    void add(const fl_w4_weight* w, size_t N, size_t K) {
        add(w->q, N * K / 2);
        add(w->scales, N * (K / w->group) * 2);
        add(w->zeros, N * (K / w->group));
    }
    bool hit(const void* p, size_t bytes) const {
        for (int i = 0; i < n; ++i)
            if (host::overlap(p, bytes, in[i].p, in[i].n)) return true;
        return false;
    }
};

void set_weight(W4Params& p, int j, const fl_w4_weight* w) {
    p.q[j] = static_cast<const uint8_t*>(w->q);
    p.scales[j] = static_cast<const uint16_t*>(w->scales);
    p.zeros[j] = static_cast<const uint8_t*>(w->zeros);
    p.group = w->group;
}

constexpr int kMaxRows = 65000 * 256;  // token tiles of one grid

// One product whose arguments have been checked.
fl_status run(int dt, bool dual, const W4Params& p, void* workspace, const host::LaunchContext& ctx, cudaStream_t stream) {
    return w4_few_rows(p.M, p.N, p.K, dual) ? w4_rows(dt, dual, p, ctx, stream) : w4_tile(dt, dual, p, workspace, ctx, stream);
}

fl_status check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (need == 0) return FL_OK;
    if (workspace == nullptr) return host::fail(FL_ERR_WORKSPACE, "workspace must not be null");
    if (reinterpret_cast<uintptr_t>(workspace) & 15u)
        return host::fail(FL_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
    if (bytes < need) return host::fail(FL_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
    return FL_OK;
}

}  // namespace

}  // namespace fl

extern "C" {

fl_status fl_w4_quantize(const void* W, void* q, void* scales, int N, int K, int group, fl_dtype dtype,
                         void* stream) {
    using namespace fl;
    if (!host::valid_dtype(dtype)) return host::fail(FL_ERR_INVALID_ARG, "bad dtype %d", (int)dtype);
    const fl_w4_weight w = {q, scales, nullptr, group};
    fl_status st;
    if ((st = check_weight("fl_w4_quantize", &w, N, K)) != FL_OK) return st;
    if ((st = host::check_ptr("W", W, true)) != FL_OK) return st;
    const size_t n = (size_t)N * K;
    if (host::overlap(q, n / 2, W, n * 2) || host::overlap(scales, n / group * 2, W, n * 2) ||
        host::overlap(q, n / 2, scales, n / group * 2))
        return host::fail(FL_ERR_INVALID_ARG, "q or scales overlaps another tensor of the call");
    const long long units = (long long)(n / 16), per = kQuantThreads * kQuantUnits;
    if ((units + per - 1) / per > 0x7fffffffll) return host::fail(FL_ERR_UNSUPPORTED, "fl_w4_quantize: too many weights");
    host::LaunchContext ctx;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = host::launch_context(s, &ctx)) != FL_OK) return st;
    const dim3 grid((unsigned)((units + per - 1) / per));
    auto kern = dtype == FL_F16 ? fl_w4_quantize_kernel<DT_F16> : fl_w4_quantize_kernel<DT_BF16>;
    return host::launched(host::launch(kern, grid, kQuantThreads, 0, ctx.pdl, s, static_cast<const uint16_t*>(W),
                                       static_cast<uint32_t*>(q), static_cast<uint16_t*>(scales), units, group == 32 ? 1 : group == 64 ? 2 : 3),
                          "4-bit quantiser");
}

size_t fl_w4_gemm_workspace_size(int M, int K, int norm) {
    return M > 0 && K > 0 && !fl::w4_always_few(M, K) ? fl::w4_tile_workspace(M, norm != 0) : 0;
}

fl_status fl_w4_gemm(const void* x, const void* gamma, const fl_w4_weight* W, const void* bias, const void* residual,
                     void* out, int M, int N, int K, float eps, fl_act act, void* workspace, size_t workspace_bytes,
                     fl_dtype dtype, void* stream) {
    using namespace fl;
    if (!host::valid_dtype(dtype)) return host::fail(FL_ERR_INVALID_ARG, "bad dtype %d", (int)dtype);
    if ((int)act < 0 || (int)act > FL_ACT_RELU) return host::fail(FL_ERR_INVALID_ARG, "bad activation %d", (int)act);
    if (!(eps >= 0.0f) || eps > 1e30f) return host::fail(FL_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (M < 1) return host::fail(FL_ERR_INVALID_ARG, "fl_w4_gemm: sizes must be positive (M=%d)", M);
    if (M > kMaxRows) return host::fail(FL_ERR_UNSUPPORTED, "fl_w4_gemm: more than %d rows", kMaxRows);
    fl_status st;
    if ((st = check_weight("fl_w4_gemm: W", W, N, K)) != FL_OK) return st;
    if ((st = host::check_ptr("x", x, true)) != FL_OK) return st;
    if ((st = host::check_ptr("out", out, true)) != FL_OK) return st;
    if ((st = host::check_ptr("gamma", gamma, false)) != FL_OK) return st;
    if ((st = host::check_ptr("bias", bias, false)) != FL_OK) return st;
    if ((st = host::check_ptr("residual", residual, false)) != FL_OK) return st;
    const size_t need = fl_w4_gemm_workspace_size(M, K, gamma != nullptr), ob = (size_t)M * N * 2;
    if ((st = check_workspace(workspace, workspace_bytes, need)) != FL_OK) return st;
    Ranges r;
    r.add(x, (size_t)M * K * 2);
    r.add(W, N, K);
    r.add(gamma, (size_t)K * 2);
    r.add(bias, (size_t)N * 2);
    if (r.hit(out, ob)) return host::fail(FL_ERR_INVALID_ARG, "out overlaps an input");
    if (residual != nullptr && residual != out && host::overlap(out, ob, residual, ob))
        return host::fail(FL_ERR_INVALID_ARG, "out may alias residual only exactly");
    if (need > 0 && (r.hit(workspace, need) || host::overlap(workspace, need, out, ob) ||
                     host::overlap(workspace, need, residual, ob)))
        return host::fail(FL_ERR_INVALID_ARG, "workspace overlaps another tensor of the call");
    host::LaunchContext ctx;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = host::launch_context(s, &ctx)) != FL_OK) return st;
    W4Params p = {};
    p.x = static_cast<const uint16_t*>(x), p.gamma = static_cast<const uint16_t*>(gamma);
    set_weight(p, 0, W);
    p.bias = static_cast<const uint16_t*>(bias), p.residual = static_cast<const uint16_t*>(residual);
    p.out = static_cast<uint16_t*>(out);
    p.M = M, p.N = N, p.K = K, p.eps = eps, p.act = act;
    return run(dtype, false, p, workspace, ctx, s);
}

size_t fl_w4_swiglu_ffn_workspace_size(int M, int D, int F) {
    if (M < 1 || F < 1 || D < 1) return 0;
    return (size_t)M * F * 2 + fl_w4_gemm_workspace_size(M, D, 1);
}

fl_status fl_w4_swiglu_ffn(const void* x, const void* gamma, const fl_w4_weight* Wg, const fl_w4_weight* Wu,
                           const fl_w4_weight* Wd, const void* bias_down, void* out, int M, int D, int F, float eps,
                           void* workspace, size_t workspace_bytes, fl_dtype dtype, void* stream) {
    using namespace fl;
    if (!host::valid_dtype(dtype)) return host::fail(FL_ERR_INVALID_ARG, "bad dtype %d", (int)dtype);
    if (!(eps >= 0.0f) || eps > 1e30f) return host::fail(FL_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (M < 1) return host::fail(FL_ERR_INVALID_ARG, "fl_w4_swiglu_ffn: sizes must be positive (M=%d)", M);
    if (M > kMaxRows) return host::fail(FL_ERR_UNSUPPORTED, "fl_w4_swiglu_ffn: more than %d rows", kMaxRows);
    fl_status st;
    if ((st = check_weight("fl_w4_swiglu_ffn: Wg", Wg, F, D)) != FL_OK) return st;
    if ((st = check_weight("fl_w4_swiglu_ffn: Wu", Wu, F, D)) != FL_OK) return st;
    if ((st = check_weight("fl_w4_swiglu_ffn: Wd", Wd, D, F)) != FL_OK) return st;
    if (Wg->group != Wu->group || (Wg->zeros == nullptr) != (Wu->zeros == nullptr))
        return host::fail(FL_ERR_INVALID_ARG, "fl_w4_swiglu_ffn: Wg and Wu must have the same group, and zero points both or neither");
    if ((st = host::check_ptr("x", x, true)) != FL_OK) return st;
    if ((st = host::check_ptr("gamma", gamma, true)) != FL_OK) return st;
    if ((st = host::check_ptr("out", out, true)) != FL_OK) return st;
    if ((st = host::check_ptr("bias_down", bias_down, false)) != FL_OK) return st;
    const size_t need = fl_w4_swiglu_ffn_workspace_size(M, D, F), ob = (size_t)M * D * 2;
    if ((st = check_workspace(workspace, workspace_bytes, need)) != FL_OK) return st;
    Ranges r;
    r.add(x, ob);
    r.add(gamma, (size_t)D * 2);
    r.add(bias_down, (size_t)D * 2);
    r.add(Wg, F, D);
    r.add(Wu, F, D);
    r.add(Wd, D, F);
    if (r.hit(out, ob)) return host::fail(FL_ERR_INVALID_ARG, "out overlaps an input");
    if (r.hit(workspace, need)) return host::fail(FL_ERR_INVALID_ARG, "workspace overlaps an input");
    if (host::overlap(workspace, need, out, ob)) return host::fail(FL_ERR_INVALID_ARG, "workspace overlaps out");
    host::LaunchContext ctx;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = host::launch_context(s, &ctx)) != FL_OK) return st;
    // (h in front, then the row scales of the tile kernel)
    // h = silu(RMSNorm(x) Wg^T) * (RMSNorm(x) Wu^T)
    W4Params p = {};
    p.x = static_cast<const uint16_t*>(x), p.gamma = static_cast<const uint16_t*>(gamma);
    set_weight(p, 0, Wg);
    set_weight(p, 1, Wu);
    p.out = static_cast<uint16_t*>(workspace);
    p.M = M, p.N = F, p.K = D, p.eps = eps;
    if ((st = run(dtype, true, p, static_cast<uint8_t*>(workspace) + (size_t)M * F * 2, ctx, s)) != FL_OK) return st;
    // out = h Wd^T (+ bias_down) + x
    W4Params d = {};
    d.x = static_cast<const uint16_t*>(workspace);
    set_weight(d, 0, Wd);
    d.bias = static_cast<const uint16_t*>(bias_down), d.residual = static_cast<const uint16_t*>(x);
    d.out = static_cast<uint16_t*>(out);
    d.M = M, d.N = D, d.K = F;
    return run(dtype, false, d, nullptr, ctx, s);
}

}  // extern "C"
