"""The serving operators on the GPU against the float64 oracle (needs an sm_103a GPU).

Bounds. u is the largest relative error of one rounding to the dtype (2^-8 bf16, 2^-11 fp16).
  w4: three operands are rounded at most once (x * gamma, the weight scale * (code - zero), the output), sums are fp32
  with 2^-22 per term at most. Element by element: |err| <= u |y| + (2.1 u + K 2^-22) sum |x w|, plus 2^-9 |v| for the
  hardware tanh of an activation (relative error 2^-10.9). The roundings are independent, so the mean square
  is at most u^2 (mean y^2 + 2 mean sum x^2 w^2), of which a uniformly spread rounding reaches a third; the square root
  is tested with the bound itself, 1.7 times what is expected.
  rope: sine and cosine to 2^-22 (fixed-point angle, sincospif), one rounding: u |y| + 2^-21 (|a| + |b|).
  kv: codes are equal, scales equal to fp32 division's; reading back is one fp32 product and one rounding.
"""
import numpy as np
import pytest
import torch

import gemm_epilogue_tma_gb300 as fl
import oracle
from gemm_epilogue_tma_gb300 import _build

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()
    fl.lib()
    torch.cuda.set_device(0)
    yield
    fl.device_status()


def gen(*seed):
    return np.random.default_rng(seed)


def put(a, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.to(DT[dt]) if dt else t).cuda()


def f64(t):
    return t.detach().float().cpu().double().numpy() if t.dtype != torch.float64 else t.cpu().numpy()


def round16(dt):
    return lambda v: torch.from_numpy(np.asarray(v, dtype=np.float32)).to(DT[dt]).double().numpy()


# ---------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("N,K,group", [(8, 32, 32), (8, 128, 128), (24, 320, 64), (136, 1056, 32), (1000, 4096, 128)])
def test_w4_quantize(dt, N, K, group):
    rng = gen(1, N, K, group)
    W = rng.standard_normal((N, K)) * np.exp2(rng.integers(-8, 3, (N, 1)))
    W[0, :group] = 0                                             # a group of zeros
    W[1, :32] = np.tile([7, 3.5, 2.5, 1.5, -2.5, 0.5, -0.5, -7], 4)  # ties
    W[2, :32] = 2.0 ** -24 * np.arange(32)                       # fp16 subnormals
    W[3, :32] = 1e-38 if dt == "bf16" else 6e-5
    W = put(W, dt)
    q, s = fl.w4_quantize(W, group)
    fl.device_status()
    code, scale = oracle.w4_quantize(f64(W), group, round16(dt), 2.0 ** (-24 if dt == "f16" else -133))
    assert np.array_equal(f64(s), scale)
    assert np.array_equal(q.cpu().numpy(), oracle.w4_pack(code))
    assert s.dtype == DT[dt]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_w4_quantize_not_finite(dt):
    W = put(gen(2).standard_normal((8, 256)), dt)
    W[0, 3], W[1, 70], W[2, 140] = float("inf"), float("nan"), -float("inf")
    q, s = fl.w4_quantize(W, 64)
    s, q = f64(s), q.cpu().numpy()
    bad = np.zeros((8, 4), dtype=bool)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert np.array_equal(np.isnan(s), bad) and (q[0, :32] == 0x88).all()
    code, scale = oracle.w4_quantize(f64(W), 64, round16(dt), 2.0 ** -24)
    assert np.array_equal(q, oracle.w4_pack(code)) and np.array_equal(s[~bad], scale[~bad])


def w4_tensors(rng, N, K, group, zeros, dt):
    q = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    s = rng.uniform(0.5, 1.5, (N, K // group)) / (4.6 * np.sqrt(K))
    z = rng.integers(0, 16, (N, K // group)).astype(np.uint8) if zeros else None
    return put(q), put(s, dt), None if z is None else put(z)


def w4_ref(x, w, gamma, eps):
    W = oracle.w4_weight(w[0].cpu().numpy(), f64(w[1]), None if w[2] is None else w[2].cpu().numpy())
    xn = f64(x) if gamma is None else oracle.rms_norm(f64(x), f64(gamma), eps)
    return xn @ W.T, np.abs(xn) @ np.abs(W).T, (xn ** 2) @ (W ** 2).T


def w4_check(got, y, mag, sq, K, dt, act_mag=0.0, what=""):
    g, u = f64(got), U[dt]
    assert np.isfinite(g).all(), what
    err = np.abs(g - y)
    bound = u * np.abs(y) + (2.1 * u + K * 2.0 ** -22) * mag + 2.0 ** -9 * act_mag + 1e-7
    assert (err <= bound).all(), f"{what}: {(err / bound).max()} times the bound"
    rms = np.sqrt((err ** 2).mean())
    most = np.sqrt((u * u * (y ** 2 + 2 * sq)).mean() + ((2.0 ** -9 * act_mag) ** 2 if np.isscalar(act_mag) else
                                                        ((2.0 ** -9 * act_mag) ** 2).mean()))
    assert rms <= most + 1e-7, f"{what}: rms {rms} above {most}"


SHAPES = [(1, 8, 32, 32), (1, 1024, 1024, 128), (2, 264, 320, 64), (3, 40, 4096, 32), (7, 2048, 2048, 128),
          (8, 520, 11008, 128), (9, 136, 256, 64), (16, 1032, 1056, 32), (33, 8, 128, 128), (65, 392, 640, 64),
          (128, 128, 512, 128), (129, 512, 512, 32), (100, 1024, 1024, 64), (60, 2048, 2048, 128), (32, 4104, 1024, 32),
          (17, 264, 11008, 128), (130, 2048, 4096, 128), (257, 264, 96, 32), (300, 6144, 1024, 64),
          (40, 20488, 2048, 128)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_w4_gemm(dt, M, N, K, group):
    for k, (zeros, norm, act, bias, res) in enumerate([(False, True, "none", False, False),
                                                       (True, False, "none", True, True),
                                                       (True, True, ("gelu", "silu", "relu")[M % 3], True, False)]):
        rng = gen(3, M, N, K, k)
        x = rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.01, 20.0, 1.0)
        x = put(x, dt)
        w = w4_tensors(rng, N, K, group, zeros, dt)
        gamma = put(1 + 0.1 * rng.standard_normal(K), dt) if norm else None
        b = put(0.1 * rng.standard_normal(N), dt) if bias else None
        r = put(rng.standard_normal((M, N)), dt) if res else None
        out = fl.w4_gemm(x, w[0], w[1], zeros=w[2], gamma=gamma, bias=b, residual=r, act=act)
        fl.device_status()
        y, mag, sq = w4_ref(x, w, gamma, 1e-6)
        if bias:
            y = y + f64(b)
        pre = np.abs(y)
        y = oracle.ACTIVATIONS[act](y)
        if res:
            y = y + f64(r)
        # (the activations' slopes are below 1.13)
        w4_check(out, y, 1.13 * mag, 1.28 * sq, K, dt, pre if act in ("gelu", "silu") else 0.0,
                 f"{dt} {M}x{N}x{K} g{group} {k}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,D,F,group,zeros", [(1, 1024, 2816, 128, False), (3, 256, 384, 32, True), (8, 320, 64, 64, True),
                                               (20, 512, 1408, 64, False), (200, 384, 1024, 128, True),
                                               (513, 1024, 2816, 128, False), (40, 2048, 9856, 64, False)])
def test_w4_swiglu_ffn(dt, M, D, F, group, zeros):
    rng = gen(4, M, D, F)
    x = put(rng.standard_normal((M, D)), dt)
    gamma = put(1 + 0.1 * rng.standard_normal(D), dt)
    Wg, Wu = (w4_tensors(rng, F, D, group, zeros, dt) for _ in range(2))
    Wd = w4_tensors(rng, D, F, group, zeros, dt)
    bias = put(0.1 * rng.standard_normal(D), dt)
    out = fl.w4_swiglu_ffn(x, gamma, Wg, Wu, Wd, bias_down=bias)
    ws = torch.full((fl.w4_swiglu_ffn_workspace_size(M, D, F),), 0xff, dtype=torch.uint8, device="cuda")
    again = fl.w4_swiglu_ffn(x, gamma, Wg, Wu, Wd, bias_down=bias, workspace=ws)
    fl.device_status()
    assert torch.equal(out, again)
    g, gm, _ = w4_ref(x, Wg, gamma, 1e-6)
    u, um, _ = w4_ref(x, Wu, gamma, 1e-6)
    h = oracle.silu(g) * u
    W = oracle.w4_weight(Wd[0].cpu().numpy(), f64(Wd[1]), None if Wd[2] is None else Wd[2].cpu().numpy())
    y = h @ W.T + f64(bias) + f64(x)
    # h: the gate's and the up product's errors, the tanh's, its rounding; then the down product's
    e = U[dt]
    dg, du = (2.1 * e + D * 2.0 ** -22) * gm, (2.1 * e + D * 2.0 ** -22) * um
    dh = (1.1 * dg + 2.0 ** -9 * np.abs(g)) * (np.abs(u) + du) + np.abs(oracle.silu(g)) * du + e * np.abs(h)
    bound = e * np.abs(y) + dh @ np.abs(W).T + (1.05 * e + F * 2.0 ** -22) * (np.abs(h) @ np.abs(W).T)
    err = np.abs(f64(out) - y)
    assert (err <= bound).all(), (err / bound).max()
    # independent roundings: the relative error of the whole is a few roundings
    assert np.sqrt((err ** 2).mean()) <= 4 * e * np.sqrt((y ** 2).mean())


def test_w4_gemm_exact_cases():
    """Products with one exact answer, on few and on many rows: an identity weight, rows of zeros."""
    for M in (1, 8, 40, 300):
        K = 256
        code = np.full((K, K), 8)
        np.fill_diagonal(code, 12)                    # 4 * 0.25
        q = put(oracle.w4_pack(code))
        s = put(np.full((K, 4), 0.25), "bf16")
        x = put(gen(5, M).standard_normal((M, K)), "bf16")
        x[M // 2] = 0
        assert torch.equal(fl.w4_gemm(x, q, s), x)
        bias = put(gen(6).standard_normal(K), "bf16")
        gamma = torch.ones(K, dtype=torch.bfloat16, device="cuda")
        out = fl.w4_gemm(x, q, s, gamma=gamma, bias=bias)
        assert torch.equal(out[M // 2], bias)


def test_w4_gemm_in_place_residual_and_not_finite_rows():
    for M in (3, 70):
        rng = gen(7, M)
        x = put(rng.standard_normal((M, 512)), "f16")
        w = w4_tensors(rng, 256, 512, 64, True, "f16")
        r = put(rng.standard_normal((M, 256)), "f16")
        want = fl.w4_gemm(x, w[0], w[1], zeros=w[2], residual=r)
        got = r.clone()
        fl.w4_gemm(x, w[0], w[1], zeros=w[2], residual=got, out=got)
        assert torch.equal(got, want)
        # a NaN or an infinity stays in its own row
        x2 = x.clone()
        x2[1, 17], x2[2, 5] = float("nan"), float("inf")
        y = fl.w4_gemm(x2, w[0], w[1], zeros=w[2], residual=r)
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
        keep = [m for m in range(M) if m not in (1, 2)]
        assert torch.equal(y[keep], want[keep])


def test_w4_rows_do_not_depend_on_their_number():
    """Outputs are written for the rows given and no others, at every row count around the kernels' borders."""
    rng = gen(8)
    w = w4_tensors(rng, 136, 384, 128, False, "bf16")
    x = put(rng.standard_normal((300, 384)), "bf16")
    gamma = put(1 + 0.1 * rng.standard_normal(384), "bf16")
    y, mag, sq = w4_ref(x, (*w[:2], None), gamma, 1e-6)
    for M in (1, 2, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300):
        buf = torch.full((M + 2, 136), 7.0, dtype=torch.bfloat16, device="cuda")
        fl.w4_gemm(x[:M].contiguous(), w[0], w[1], gamma=gamma, out=buf[1:M + 1])
        assert (buf[0] == 7).all() and (buf[M + 1] == 7).all()
        w4_check(buf[1:M + 1], y[:M], mag[:M], sq[:M], 384, "bf16", what=f"{M} rows")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M", [3, 20, 200])
def test_w4_gemm_small_gamma(dt, M):
    """Weights and gammas that are small together lose nothing to the type's smallest values (fp16 x * gamma and
    64 * w * gamma stay above 2^-14 but for a share too small to see)."""
    rng = gen(9, M)
    x = put(rng.standard_normal((M, 512)), dt)
    q, s, z = w4_tensors(rng, 264, 512, 64, False, dt)
    s = put(rng.uniform(0.5, 1.5, s.shape) * 1e-3, dt)
    gamma = put((1 + 0.1 * rng.standard_normal(512)) * 4e-3, dt)
    w = (q, s, z)
    y, mag, sq = w4_ref(x, w, gamma, 1e-6)
    y, mag, sq = y * 4096, mag * 4096, sq * 4096 ** 2   # (outputs of some 1e-4: the last rounding, fp16's too, is absolute)
    got = f64(fl.w4_gemm(x, q, s, gamma=gamma)) * 4096
    fl.device_status()
    err, u = np.abs(got - y), U[dt]
    last = 4096 * 2.0 ** -25 if dt == "f16" else 0.0
    # x * gamma below 2^-14 (|x| < 0.015) is rounded by 2^-25 absolutely, 2^-11 of 2^-14
    lost = 4096 * 2.0 ** -25 * 512 * 8 * 1.5e-3 if dt == "f16" else 0.0
    assert (err <= u * np.abs(y) + (2.1 * u + 512 * 2.0 ** -22) * mag + last + lost).all()
    assert np.sqrt((err ** 2).mean()) <= np.sqrt((u * u * (y ** 2 + 2 * sq)).mean()) + last


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K,group", [(1, 264, 1024, 32), (2, 136, 4096, 128), (3, 520, 320, 64), (4, 1024, 2048, 128)])
def test_w4_gemm_up_to_four_rows_round_the_output_alone(dt, M, N, K, group):
    """x * gamma is carried as two numbers of the dtype, off by u^2 of it (and half of fp16's smallest value), the codes are
    exact and the sums fp32: next to those the output's rounding is the only one."""
    rng = gen(13, M, N, K)
    x = put(rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.01, 20.0, 1.0), dt)
    w = w4_tensors(rng, N, K, group, True, dt)
    gamma = put(1 + 0.1 * rng.standard_normal(K), dt)
    got = fl.w4_gemm(x, w[0], w[1], zeros=w[2], gamma=gamma)
    fl.device_status()
    y, mag, _ = w4_ref(x, w, gamma, 1e-6)
    W = oracle.w4_weight(w[0].cpu().numpy(), f64(w[1]), w[2].cpu().numpy())
    rms = 1 / np.sqrt((f64(x) ** 2).mean(1, keepdims=True) + 1e-6)
    small = 2.0 ** -25 * rms * np.abs(W).sum(1) if dt == "f16" else 0.0
    u = U[dt]
    assert (np.abs(f64(got) - y) <= u * np.abs(y) + (u * u + K * 2.0 ** -22) * mag + small + 2.0 ** -25).all()


@pytest.mark.parametrize("M", [1, 8, 20, 40, 300])
def test_w4_gemm_not_finite_weights(M):
    """A NaN or infinite scale, bias or residual stays in the outputs that it belongs to."""
    rng = gen(10, M)
    x = put(rng.standard_normal((M, 512)), "bf16")
    q, s, z = w4_tensors(rng, 264, 512, 128, True, "bf16")
    r = put(rng.standard_normal((M, 264)), "bf16")
    b = put(rng.standard_normal(264), "bf16")
    gamma = put(1 + 0.1 * rng.standard_normal(512), "bf16")
    want = fl.w4_gemm(x, q, s, zeros=z, gamma=gamma, bias=b, residual=r)
    s[5, 1], s[140, 3], b[77], r[M - 1, 200] = float("nan"), float("inf"), float("inf"), float("nan")
    got = fl.w4_gemm(x, q, s, zeros=z, gamma=gamma, bias=b, residual=r)
    fl.device_status()
    bad = torch.zeros((M, 264), dtype=torch.bool, device="cuda")
    bad[:, 5] = bad[:, 140] = bad[:, 77] = bad[M - 1, 200] = True
    assert torch.equal(got[~bad], want[~bad]) and not torch.isfinite(got[bad]).any()


@pytest.mark.parametrize("M,N,K,group", [(16401, 264, 128, 64), (16400, 8, 64, 32), (4099, 128, 64, 64)])
def test_w4_gemm_many_rows_and_exact_workspace(M, N, K, group):
    """Tokens in many tiles, whose last ends anywhere, with no byte of workspace or output more than said."""
    rng = gen(11, M)
    x = put(rng.standard_normal((M, K)), "f16")
    w = w4_tensors(rng, N, K, group, False, "f16")
    gamma = put(1 + 0.1 * rng.standard_normal(K), "f16")
    need = fl.w4_gemm_workspace_size(M, K, True)
    ws = torch.full((need + 512,), 0xa5, dtype=torch.uint8, device="cuda")
    out = torch.full((M + 2, N), 7.0, dtype=torch.float16, device="cuda")
    fl.w4_gemm(x, w[0], w[1], gamma=gamma, out=out[1:M + 1], workspace=ws[256:need + 256])
    fl.device_status()
    assert (ws[:256] == 0xa5).all() and (ws[need + 256:] == 0xa5).all() and (out[0] == 7).all() and (out[-1] == 7).all()
    y, mag, sq = w4_ref(x, w, gamma, 1e-6)
    w4_check(out[1:M + 1], y, mag, sq, K, "f16")
    with pytest.raises(fl.FusedLinError):
        fl.w4_gemm(x, w[0], w[1], gamma=gamma, workspace=ws[256:need + 240])


def test_w4_tiles_left_over_from_whole_rounds():
    """Sizes whose last tiles take a launch of their own beside the others: what follows reads a whole result, however
    the launches are issued."""
    rng = gen(12)
    M, D, F = 40, 2048, 9856
    x = put(rng.standard_normal((M, D)), "bf16")
    gamma = put(1 + 0.1 * rng.standard_normal(D), "bf16")
    Wg, Wu = (w4_tensors(rng, F, D, 128, False, "bf16")[:2] for _ in range(2))
    Wd = w4_tensors(rng, D, F, 128, False, "bf16")[:2]
    big = w4_tensors(rng, 20488, D, 128, True, "bf16")
    ws = torch.empty(fl.w4_swiglu_ffn_workspace_size(M, D, F), dtype=torch.uint8, device="cuda")
    y, z = torch.empty_like(x), torch.empty((M, 20488), dtype=torch.bfloat16, device="cuda")

    def chain():
        fl.w4_swiglu_ffn(x, gamma, Wg, Wu, Wd, out=y, workspace=ws)
        fl.w4_gemm(y, big[0], big[1], zeros=big[2], gamma=gamma, out=z)
        fl.w4_gemm(z[:, :F].contiguous(), Wd[0], Wd[1], residual=y, out=y)
    fl.set_option("pdl", 0)
    try:
        n = fl.kernel_launches()
        chain()
        torch.cuda.synchronize()
        assert fl.kernel_launches() - n > 3 + 2 + 1  # a row-scale kernel and two launches of tiles, twice; the down products
    finally:
        fl.set_option("pdl", 1)
    want = y.clone(), z.clone()
    for _ in range(20):
        y.zero_(), z.zero_(), ws.fill_(0xff)
        chain()
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(5):
        y.zero_(), z.zero_(), ws.fill_(0xff)
        graph.replay()
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])
    fl.device_status()


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rope_check(got, x, pos, f, axis, dt, interleaved, inverse):
    want = oracle.rope(f64(x), pos, f, axis, interleaved, inverse)
    n = len(f)
    lo = np.arange(n) * (2 if interleaved else 1)
    hi = lo + (1 if interleaved else n)
    pair = np.zeros_like(want)
    pair[..., lo] = pair[..., hi] = np.abs(f64(x)[..., lo]) + np.abs(f64(x)[..., hi])
    err = np.abs(f64(got) - want)
    assert (err <= U[dt] * np.abs(want) + 2.0 ** -21 * pair + 2.0 ** -25).all(), err.max()
    assert np.array_equal(f64(got)[..., 2 * n:], f64(x)[..., 2 * n:])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows,hq,hk,D,R,axes", [(1, 1, 1, 8, 2, 1), (1, 32, 8, 128, 128, 1), (3, 5, 0, 64, 32, 2),
                                                 (17, 4, 2, 80, 80, 3), (50, 3, 1, 96, 48, 4), (33, 2, 2, 72, 36, 2),
                                                 (700, 8, 2, 128, 64, 3), (5, 2, 1, 512, 512, 1), (6, 1, 3, 14, 10, 1)])
@pytest.mark.parametrize("interleaved,inverse", [(False, False), (True, False), (False, True), (True, True)])
def test_rope(dt, rows, hq, hk, D, R, axes, interleaved, inverse):
    rng = gen(20, rows, D, R)
    q = put(rng.standard_normal((rows, hq, D)), dt)
    k = put(rng.standard_normal((rows, hk, D)), dt) if hk else None
    n = R // 2
    f = (10000.0 ** (-np.arange(n) / n)).astype(np.float32)
    pos = rng.integers(-2 ** 31, 2 ** 31, (axes, rows)) if rows % 2 else rng.integers(0, 5000, (axes, rows))
    cut = [n // axes] * (axes - 1)
    sections = cut + [n - sum(cut)]
    axis = np.repeat(np.arange(axes), sections)
    tq, tk = fl.rope(q, k, put(pos.astype(np.int32)), put(f), sections=sections, interleaved=interleaved, inverse=inverse)
    fl.device_status()
    rope_check(tq, q, pos, f, axis, dt, interleaved, inverse)
    if hk:
        rope_check(tk, k, pos, f, axis, dt, interleaved, inverse)


@pytest.mark.parametrize("shift", [0, 1])
def test_rope_strided_views_and_in_place(shift):
    """q and k as column ranges of a stacked projection's output, vector-aligned and not: in place, v untouched."""
    rng = gen(21)
    rows, hq, hk, D = 37, 6, 2, 64
    wide = put(rng.standard_normal((rows, (hq + 2 * hk) * D + 8)), "bf16")
    view = wide[:, shift:shift + (hq + 2 * hk) * D]
    q, k = view[:, :hq * D].unflatten(1, (hq, D)), view[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    before = wide.clone()
    f = (1e4 ** (-np.arange(24) / 24)).astype(np.float32)
    pos = np.arange(rows)[None] * 1000
    oq, ok = fl.rope(q, k, put(pos.astype(np.int32)), put(f))
    assert torch.equal(wide, before)
    fl.rope(q, k, put(pos[0].astype(np.int32)), put(f), out_q=q, out_k=k)
    fl.device_status()
    assert torch.equal(q, oq) and torch.equal(k, ok)
    rope_check(oq, before[:, shift:shift + hq * D].unflatten(1, (hq, D)), pos, f, [0] * 24, "bf16", False, False)
    rest = torch.ones(wide.shape[1], dtype=torch.bool)
    rest[shift:shift + (hq + hk) * D] = False
    assert torch.equal(wide[:, rest], before[:, rest])
    # heads first, as some attention kernels want it
    out = torch.empty((hq, rows, D), dtype=torch.bfloat16, device="cuda")
    fl.rope(before[:, shift:shift + hq * D].unflatten(1, (hq, D)), None, put(pos.astype(np.int32)), put(f),
            out_q=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), oq)


def test_rope_inverse_is_the_gradient():
    """<g, rope(x)> = <rope_inverse(g), x> and differences along a direction, in the dtype's precision."""
    rng = gen(22)
    x, g, d = (put(rng.standard_normal((9, 4, 64)), "f16") for _ in range(3))
    pos, f = put(rng.integers(0, 9000, (1, 9)).astype(np.int32)), put((1e4 ** (-np.arange(32) / 32)).astype(np.float32))
    grad = fl.rope(g, None, pos, f, inverse=True)[0]
    y = fl.rope(x, None, pos, f)[0]
    size = np.sqrt((f64(g) ** 2).sum() * (f64(x) ** 2).sum())
    assert abs((f64(g) * f64(y)).sum() - (f64(grad) * f64(x)).sum()) <= 2 * U["f16"] * size
    xp, xm = (x + d), (x - d)                       # linear: the difference is exact up to the roundings
    diff = (f64(fl.rope(xp, None, pos, f)[0]) - f64(fl.rope(xm, None, pos, f)[0]))
    along = f64(xp) - f64(xm)
    assert abs((f64(g) * diff).sum() - (f64(grad) * along).sum()) <= 8 * U["f16"] * size


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def cache(pages, size, H, D, fmt, fill=3):
    c = [torch.full((pages, size, H, D), fill, dtype=torch.uint8, device="cuda").view(CODES[fmt]) for _ in "kv"]
    s = [torch.full((pages, size, H), 0.5, device="cuda") for _ in "kv"]
    return c, s


def numbers(codes):
    return codes.float().cpu().double().numpy()


def check_write(x, codes, scales, places, fmt, old_codes, old_scales):
    """Written places hold the oracle's codes and scales, all others what they held."""
    want_c, want_s = numbers(old_codes), f64(old_scales)
    code, scale = oracle.kv_quantize(f64(x), fmt)
    for i, place in enumerate(places):
        if isinstance(place, tuple):
            want_c[place], want_s[place] = code[i], scale[i]
    assert np.array_equal(f64(scales), want_s, equal_nan=True)
    assert np.array_equal(numbers(codes), want_c)


KV = [  # seqs, rows of each, start, H, D, page, dtype
    ([1], [0], 1, 8, 1, "f16"), ([1], [5], 2, 64, 16, "bf16"), ([37], [0], 8, 128, 16, "bf16"),
    ([5, 0, 1, 19], [3, 7, 16, 0], 3, 80, 16, "f16"), ([1] * 40, list(range(40)), 5, 128, 32, "f16"),
    ([64, 1, 130], [0, 63, 64], 2, 256, 64, "bf16"), ([9, 4], [100, 0], 40, 24, 8, "bf16"), ([33, 2], [1, 1], 4, 40, 7, "f16"), ([1, 2] * 50, [4] * 100, 1, 16, 8, "bf16"),
      ([1, 0, 3] * 110, [1] * 330, 1, 8, 4, "f16")]


def kv_set_up(lens, start, page, rng, spare=2):
    B = len(lens)
    need = [-(-(s + n) // page) for s, n in zip(start, lens)]
    per = max(max(need), 1) + 1
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table, at = np.full((B, per), -1, dtype=np.int32), 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return table, pages, cu


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,start,H,D,page,dt", KV)
def test_kv_write_and_read(fmt, lens, start, H, D, page, dt):
    rng = gen(30, len(lens), D, H)
    table, pages, cu = kv_set_up(lens, start, page, rng)
    T = int(cu[-1])
    # k and v as column ranges of one matrix, with rows behind the last sequence
    kv = rng.standard_normal((T + 3, 2 * H * D)) * np.exp2(rng.integers(-10, 4, (T + 3, 1)))
    kv = put(kv, dt)
    k, v = kv[:, :H * D].unflatten(1, (H, D)), kv[:, H * D:].unflatten(1, (H, D))
    (kc, vc), (ks, vs) = cache(pages, page, H, D, fmt)
    old = [t.clone() for t in (kc, vc, ks, vs)]
    tt, tcu, ts = put(table), put(cu), put(np.array(start, dtype=np.int32))
    fl.kv_write(k, v, kc, vc, ks, vs, tt, ts, cu_rows=tcu)
    fl.device_status()
    places = oracle.kv_places(T + 3, len(lens), page, pages, table, cu, start)
    check_write(k, kc, ks, places, fmt, old[0], old[2])
    check_write(v, vc, vs, places, fmt, old[1], old[3])
    # read back: whole contexts, from position 0
    ctx = np.concatenate([[0], np.cumsum(np.array(start) + np.array(lens))]).astype(np.int32)
    out = torch.full((int(ctx[-1]) + 2, 2, H, D), 9.0, dtype=DT[dt], device="cuda")
    fl.kv_read(kc, vc, ks, vs, tt, put(ctx), out_k=out[:, 0], out_v=out[:, 1])
    fl.device_status()
    assert (out[int(ctx[-1]):] == 9).all()
    places = oracle.kv_places(int(ctx[-1]), len(lens), page, pages, table, ctx)
    for w, (c, s) in enumerate(((kc, ks), (vc, vs))):
        c, s = numbers(c), f64(s)
        want = np.stack([c[p] * s[p][:, None] for p in places]) if places else np.zeros((0, H, D))
        got = f64(out[:len(places), w])
        assert (np.abs(got - want) <= (U[dt] + 2.0 ** -23) * np.abs(want) + 2.0 ** -25).all()
    # one position of each sequence, without row offsets
    last = np.array(start) + np.array(lens) - 1
    if (last >= 0).all():
        one = torch.empty((2, len(lens), H, D), dtype=DT[dt], device="cuda")
        fl.kv_read(kc, vc, ks, vs, tt, None, start=put(last.astype(np.int32)), out_k=one[0], out_v=one[1])
        fl.device_status()
        rows = [int(ctx[b]) + int(last[b]) for b in range(len(lens))]
        assert torch.equal(one[0], out[rows, 0]) and torch.equal(one[1], out[rows, 1])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_kv_codes_at_borders(fmt, dt):
    """Rows made of values on and next to the borders between codes, tiny, huge and zero rows, NaN and infinities."""
    rng = gen(31)
    H, D = 1, 128
    r16 = round16(dt)
    rows = []
    for n in range(300):
        amax = float(r16(abs(rng.standard_normal()) * 2.0 ** rng.integers(-8, 8) + 1e-3))
        top = {"int8": 127.0, "e4m3": 448.0}[fmt]
        s = float(np.float32(np.float32(amax) / np.float32(top)))
        if fmt == "int8":
            c = rng.integers(-127, 127, D) + 0.5
        else:
            every = np.unique(oracle.e4m3_round(rng.uniform(-448, 448, 4 * D)))
            c = rng.choice((every[:-1] + every[1:]) / 2, D)
        x = r16(c * s)
        x = np.where(np.abs(x) > amax, amax / 2, x)
        x[0] = amax
        rows.append(x)
    big = 65504.0 if dt == "f16" else float(r16(3.38e38))
    least = 2.0 ** -24 if dt == "f16" else 2.0 ** -133
    rows += [np.zeros(D), np.full(D, least), np.where(np.arange(D) % 2, big, -big),
             np.where(np.arange(D) % 3, least, big), np.arange(D) * least]
    x = put(np.stack(rows)[:, None], dt)
    T = x.shape[0]
    x = torch.cat([x, x[:4].clone()])
    x[T, 0, 5], x[T + 1, 0, 0], x[T + 2, 0, 127] = float("nan"), float("inf"), -float("inf")
    T += 4
    (kc, vc), (ks, vs) = cache(T, 1, H, D, fmt)
    old = [t.clone() for t in (kc, vc, ks, vs)]
    table = put(np.arange(T, dtype=np.int32)[:, None])
    zero = torch.zeros(T, dtype=torch.int32, device="cuda")
    fl.kv_write(x, -x, kc, vc, ks, vs, table, zero)
    fl.device_status()
    places = [(i, 0) for i in range(T)]
    check_write(x, kc, ks, places, fmt, old[0], old[2])
    check_write(-x, vc, vs, places, fmt, old[1], old[3])
    out = torch.empty((2, T, H, D), dtype=DT[dt], device="cuda")
    fl.kv_read(kc, vc, ks, vs, table, None, start=zero, out_k=out[0], out_v=out[1])
    assert torch.isnan(out[0, T - 4:T - 1]).all() and torch.isfinite(out[0, :T - 4]).all()


def test_kv_rows_without_a_page_are_skipped_and_reported():
    """Page numbers outside the pool, positions outside the table and negative ones: skipped, the others handled."""
    H, D, page, pages = 2, 64, 16, 6
    rng = gen(32)
    table = np.array([[0, 99], [-1, 1], [2, 3]], dtype=np.int32)
    start = np.array([14, 14, -2], dtype=np.int32)
    cu = np.array([0, 4, 8, 30], dtype=np.int32)
    k = put(rng.standard_normal((45, H, D)), "bf16")
    start[2] = -2
    (kc, vc), (ks, vs) = cache(pages, page, H, D, "int8")
    old = [t.clone() for t in (kc, vc, ks, vs)]
    args = (put(table), put(start))
    fl.kv_write(k, k, kc, vc, ks, vs, *args, cu_rows=put(cu))
    with pytest.raises(fl.FusedLinError) as e:
        fl.device_status()
    assert e.value.status == 7
    fl.device_status()  # read and cleared
    places = oracle.kv_places(45, 3, page, pages, table, cu, start)
    assert places.count("bad") == 6 and places.count(None) == 15
    check_write(k, kc, ks, places, "int8", old[0], old[2])
    out = torch.full((2, 45, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    fl.kv_read(kc, vc, ks, vs, args[0], put(cu), start=args[1], out_k=out[0], out_v=out[1])
    with pytest.raises(fl.FusedLinError):
        fl.device_status()
    left = [not isinstance(p, tuple) for p in places]
    assert (out[:, left] == 5).all()
    # a position past the table
    fl.kv_write(k[:3], k[:3], kc, vc, ks, vs, args[0], put(np.array([32, 31, 2 ** 31 - 1], dtype=np.int32)))
    with pytest.raises(fl.FusedLinError):
        fl.device_status()
    # a skipped row does not make the products of other calls give up
    x = put(rng.standard_normal((300, 512)), "bf16")
    w = put(rng.standard_normal((256, 512)), "bf16")
    fl.kv_write(k[:1], k[:1], kc, vc, ks, vs, args[0][:1], put(np.array([40], dtype=np.int32)))
    y = fl.gemm_epilogue(x, w, pattern="gemm_gelu")
    with pytest.raises(fl.FusedLinError) as e:
        fl.device_status()
    assert e.value.status == 7
    assert torch.equal(y, fl.gemm_epilogue(x, w, pattern="gemm_gelu"))


def test_kv_large_pool_offsets():
    """Places whose byte offset passes 2^32."""
    H, D, page, pages = 8, 128, 64, 66000                      # 4.3 GB of codes for each of k and v
    kc = torch.zeros((pages, page, H, D), dtype=torch.int8, device="cuda")
    ks = torch.zeros((pages, page, H), device="cuda")
    vc, vs = torch.zeros_like(kc), torch.zeros_like(ks)
    k = put(gen(33).standard_normal((4, H, D)), "f16")
    table = put(np.array([[pages - 1], [3]], dtype=np.int32))
    start = put(np.array([62, 0], dtype=np.int32))
    cu = put(np.array([0, 2, 4], dtype=np.int32))
    fl.kv_write(k, -k, kc, vc, ks, vs, table, start, cu_rows=cu)
    fl.device_status()
    code, scale = oracle.kv_quantize(f64(k), "int8")
    assert np.array_equal(numbers(kc[-1, 62:]), code[:2]) and np.array_equal(numbers(vc[3, :2]), -code[2:])
    assert np.array_equal(f64(ks[-1, 62:]), scale[:2]) and int(kc[:3].abs().max()) == 0
    out = torch.empty((2, 4, H, D), dtype=torch.float16, device="cuda")
    fl.kv_read(kc, vc, ks, vs, table, cu, start=start, out_k=out[0], out_v=out[1])
    assert torch.equal(out[0], -out[1]) and (out[0] - k).abs().max() < 0.03


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_decode_steps_together():
    """A prompt and decode steps of two sequences through projection, rotation, cache and FFN on 4-bit weights, against
    the same steps of the oracle; the decode step captured in a graph and replayed gives the direct calls' bits."""
    rng = gen(40)
    D, hq, hk, hd, F, page = 512, 4, 2, 128, 1024, 16
    dt = "bf16"
    W16 = {n: put(rng.standard_normal(s) / np.sqrt(s[1]), dt) for n, s in
           (("qkv", ((hq + 2 * hk) * hd, D)), ("o", (D, hq * hd)), ("g", (F, D)), ("u", (F, D)), ("d", (D, F)))}
    W = {n: fl.w4_quantize(w, 64) for n, w in W16.items()}
    gamma = put(1 + 0.1 * rng.standard_normal(D), dt)
    f = put((1e4 ** (-np.arange(64) / 64)).astype(np.float32))
    table = put(np.array([[4, 1], [0, 3]], dtype=np.int32))
    (kc, vc), (ks, vs) = cache(5, page, hk, hd, "int8", fill=0)

    def layer(x, pos, start, cu, ctx, buf):
        T = x.shape[0]
        fl.w4_gemm(x, *W["qkv"], gamma=gamma, out=buf["qkv"])
        q = buf["qkv"][:, :hq * hd].unflatten(1, (hq, hd))
        k = buf["qkv"][:, hq * hd:(hq + hk) * hd].unflatten(1, (hk, hd))
        v = buf["qkv"][:, (hq + hk) * hd:].unflatten(1, (hk, hd))
        fl.rope(q, k, pos, f, out_q=q, out_k=k)
        fl.kv_write(k, v, kc, vc, ks, vs, table, start, cu_rows=cu)
        fl.kv_read(kc, vc, ks, vs, table, ctx, out_k=buf["ck"], out_v=buf["cv"])
        fl.w4_gemm(q.reshape(T, hq * hd) if q.is_contiguous() else buf["qkv"][:, :hq * hd].contiguous(), *W["o"],
                   residual=x, out=buf["h"])
        fl.w4_swiglu_ffn(buf["h"], gamma, W["g"], W["u"], W["d"], out=buf["y"], workspace=buf["ws"])

    def buffers(T, rows):
        e = lambda *s: torch.zeros(s, dtype=DT[dt], device="cuda")  # noqa: E731
        return {"qkv": e(T, (hq + 2 * hk) * hd), "ck": e(rows, hk, hd), "cv": e(rows, hk, hd), "h": e(T, D), "y": e(T, D),
                "ws": torch.empty(fl.w4_swiglu_ffn_workspace_size(T, D, F), dtype=torch.uint8, device="cuda")}

    def i32(*v):
        return put(np.array(v, dtype=np.int32))
    # prompt of 13 and 7 rows
    x = put(rng.standard_normal((20, D)), dt)
    pos = i32(*range(13), *range(7))
    buf = buffers(20, 32)
    layer(x, pos, i32(0, 0), i32(0, 13, 20), i32(0, 13, 20), buf)
    fl.device_status()
    k = f64(buf["qkv"])[:, hq * hd:(hq + hk) * hd].reshape(20, hk, hd)
    code, scale = oracle.kv_quantize(k, "int8")
    back = code * scale[..., None]
    assert np.abs(f64(buf["ck"])[:20] - back).max() <= U[dt] * np.abs(back).max()
    raw = oracle.linear(oracle.rms_norm(f64(x), f64(gamma), 1e-6), oracle.w4_weight(W["qkv"][0].cpu().numpy(), f64(W["qkv"][1])))
    kk = oracle.rope(raw[:, hq * hd:(hq + hk) * hd].reshape(20, hk, hd), [pos.cpu().numpy()], f.cpu().numpy(), [0] * 64)
    assert np.sqrt(((k - kk) ** 2).mean()) <= 4 * U[dt] * np.sqrt((kk ** 2).mean())
    # a decode step, direct and captured
    x1 = put(rng.standard_normal((2, D)), dt)
    args = (i32(13, 7), i32(13, 7), None, i32(0, 14, 22))
    b1 = buffers(2, 22)
    layer(x1, *args, b1)
    fl.device_status()
    want = {n: b1[n].clone() for n in ("qkv", "ck", "cv", "h", "y")}
    state = [t.clone() for t in (kc, vc, ks, vs)]
    step = buf["qkv"].new_empty(2, hq * hd)

    def captured():
        fl.w4_gemm(x1, *W["qkv"], gamma=gamma, out=b1["qkv"])
        q = b1["qkv"][:, :hq * hd].unflatten(1, (hq, hd))
        k = b1["qkv"][:, hq * hd:(hq + hk) * hd].unflatten(1, (hk, hd))
        v = b1["qkv"][:, (hq + hk) * hd:].unflatten(1, (hk, hd))
        fl.rope(q, k, args[0], f, out_q=step.unflatten(1, (hq, hd)), out_k=k)
        fl.kv_write(k, v, kc, vc, ks, vs, table, args[1])
        fl.kv_read(kc, vc, ks, vs, table, args[3], out_k=b1["ck"], out_v=b1["cv"])
        fl.w4_gemm(step, *W["o"], residual=x1, out=b1["h"])
        fl.w4_swiglu_ffn(b1["h"], gamma, W["g"], W["u"], W["d"], out=b1["y"], workspace=b1["ws"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = fl.Graph.capture(captured)
    torch.cuda.current_stream().wait_stream(side)
    for t in (kc, vc, ks, vs, b1["ck"], b1["cv"], b1["h"], b1["y"]):
        (t.view(torch.uint8) if t.dtype == torch.int8 else t)[-1:].zero_()
    kc.copy_(state[0]), vc.copy_(state[1]), ks.copy_(state[2]), vs.copy_(state[3])
    for _ in range(2):
        graph.launch()
    torch.cuda.synchronize()
    fl.device_status()
    for n in ("ck", "cv", "h", "y"):
        assert torch.equal(b1[n], want[n]), n
    for t, s in zip((kc, vc, ks, vs), state):
        assert torch.equal(t, s)
    graph.close()


@pytest.mark.parametrize("dt,fmt", [("f16", "int8"), ("bf16", "e4m3")])
def test_decoder_layer_with_cache(dt, fmt):
    """A prepared layer with rotary positions and a cache attached: half 0 gives what the calls one by one give, direct
    and captured, follows positions and starts rewritten in place, and goes back to the plain half when detached."""
    rng = gen(42)
    M, D, Dkv, F, hd, page = 3, 512, 256, 512, 64, 16
    e = lambda *s: torch.zeros(s, dtype=DT[dt], device="cuda")  # noqa: E731
    T = {n: put(rng.standard_normal(s) / np.sqrt(s[-1]), dt) for n, s in
         (("Wq", (D, D)), ("Wk", (Dkv, D)), ("Wv", (Dkv, D)), ("Wo", (D, D)), ("Wg", (F, D)), ("Wu", (F, D)), ("Wd", (D, F)))}
    T.update(x=put(rng.standard_normal((M, D)), dt), gamma_attn=put(1 + 0.1 * rng.standard_normal(D), dt),
             gamma_ffn=put(1 + 0.1 * rng.standard_normal(D), dt), q=e(M, D), k=e(M, Dkv), v=e(M, Dkv), attn=e(M, D), h=e(M, D),
             out=e(M, D))
    layer = fl.DecoderLayer(**T)
    layer.issue(0)
    q, k, v = (T[n].clone() for n in "qkv")
    f = put((1e4 ** (-np.arange(24) / 24)).astype(np.float32))
    pos = put(np.array([[5, 90, 17], [1, 2, 3]], dtype=np.int32))
    table, start = put(np.array([[2, 4], [1, 0], [3, 5]], dtype=np.int32)), put(np.array([5, 30, 17], dtype=np.int32))
    (kc, vc), (ks, vs) = cache(6, page, Dkv // hd, hd, fmt)
    (kc2, vc2), (ks2, vs2) = cache(6, page, Dkv // hd, hd, fmt)
    for head_dim in (60, 0):
        with pytest.raises(ValueError):
            layer.attach_cache(head_dim, positions=pos, inv_freq=f, sections=(16, 8))
    with pytest.raises(fl.FusedLinError):                      # 24 pairs do not fit in 32 channels
        layer.attach_cache(32, positions=pos, inv_freq=f, sections=(16, 8))
    with pytest.raises(ValueError):
        layer.attach_cache(hd, positions=pos, inv_freq=f, sections=(16, 9))
    with pytest.raises(ValueError):
        layer.attach_cache(hd, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, page_table=table)
    layer.issue(0)
    assert torch.equal(T["q"], q) and torch.equal(T["k"], k)  # refused: as it was
    layer.attach_cache(hd, positions=pos, inv_freq=f, sections=(16, 8), k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs,
                       page_table=table, start=start)

    def expect():
        rq, rk = fl.rope(q.unflatten(1, (D // hd, hd)), k.unflatten(1, (Dkv // hd, hd)), pos, f, sections=(16, 8))
        fl.kv_write(rk, v.unflatten(1, (Dkv // hd, hd)), kc2, vc2, ks2, vs2, table, start)
        return rq.flatten(1), rk.flatten(1)

    def check():
        rq, rk = expect()
        assert torch.equal(T["q"], rq) and torch.equal(T["k"], rk) and torch.equal(T["v"], v)
        for a, b in ((kc, kc2), (vc, vc2)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(ks, ks2) and torch.equal(vs, vs2)
    layer.issue(0)
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = fl.Graph.capture(lambda: (layer.issue(0), layer.issue(1)))
    torch.cuda.current_stream().wait_stream(side)
    pos += 1
    start += 1
    graph.launch()
    torch.cuda.synchronize()
    check()
    graph.close()
    layer.attach_cache(hd)
    layer.issue(0)
    assert torch.equal(T["q"], q) and torch.equal(T["k"], k)
    fl.device_status()
    layer.close()


def test_calls_on_two_streams_at_once():
    """The same operators issued on two streams with their own buffers give what they give alone."""
    rng = gen(41)
    w = w4_tensors(rng, 1024, 1024, 128, True, "f16")
    xs = [put(rng.standard_normal((M, 1024)), "f16") for M in (4, 200)]
    gamma = put(1 + 0.1 * rng.standard_normal(1024), "f16")
    want = [fl.w4_gemm(x, w[0], w[1], zeros=w[2], gamma=gamma) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(20):
        for i, (x, s) in enumerate(zip(xs, streams)):
            got[i].append(fl.w4_gemm(x, w[0], w[1], zeros=w[2], gamma=gamma, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])
        fl.device_status(streams[i])


def serving_calls(rng, M):
    """Every operator as a function that leaves its result in fixed tensors, those tensors, and the launches it makes."""
    w = w4_tensors(rng, 512, 512, 64, True, "bf16")
    wide = [w4_tensors(rng, 768, 512, 64, False, "bf16")[:2] for _ in range(2)] + [w4_tensors(rng, 512, 768, 64, False, "bf16")[:2]]
    x, gamma = put(rng.standard_normal((M, 512)), "bf16"), put(1 + 0.1 * rng.standard_normal(512), "bf16")
    e = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o, y, q, k, ck, cv = e(M, 512), e(M, 512), e(M, 8, 64), e(M, 2, 64), e(M, 2, 64), e(M, 2, 64)
    codes, scales = torch.zeros((512, 384), dtype=torch.uint8, device="cuda"), e(512, 24)
    W = put(rng.standard_normal((512, 768)), "bf16")
    pos, f = put(rng.integers(0, 5000, M).astype(np.int32)), put((1e4 ** (-np.arange(32) / 32)).astype(np.float32))
    (kc, vc), (ks, vs) = cache((M + 15) // 16, 16, 2, 64, "e4m3")
    table = put(np.arange((M + 15) // 16, dtype=np.int32)[None])
    cu, start = put(np.array([0, M], dtype=np.int32)), put(np.zeros(1, dtype=np.int32))
    heads = x.unflatten(1, (8, 64))
    few = M <= 32
    return [(lambda: fl.w4_quantize(W, 32, q=codes, scales=scales), (codes, scales), 1),
            (lambda: fl.w4_gemm(x, *w[:2], zeros=w[2], gamma=gamma, out=o), (o,), 1 if few else 2),
            (lambda: fl.w4_swiglu_ffn(x, gamma, *wide, out=y), (y,), 2 if few else 3),
            (lambda: fl.rope(heads, heads[:, :2], pos, f, out_q=q, out_k=k), (q, k), 1),
            (lambda: fl.kv_write(heads[:, :2], heads[:, 2:4], kc, vc, ks, vs, table, start, cu_rows=cu), (kc, vc, ks, vs), 1),
            (lambda: fl.kv_read(kc, vc, ks, vs, table, cu, out_k=ck, out_v=cv), (ck, cv), 1)]


def snapshot(tensors):
    return [t.view(torch.uint8).clone() if t.element_size() == 1 else t.clone() for t in tensors]


@pytest.mark.parametrize("M", [2, 300])
@pytest.mark.parametrize("how", ["direct", "torch graph", "library graph", "no overlap of launches"])
def test_every_way_of_issuing(M, how):
    """Each operator's results are the same issued directly, captured and replayed after its tensors were overwritten,
    and without programmatic launches; each counts its kernels."""
    for call, made, launches in serving_calls(gen(43, M), M):
        before = snapshot(made)
        call()
        torch.cuda.synchronize()
        want = snapshot(made)
        n = fl.kernel_launches()
        if how == "direct":
            call()
            assert fl.kernel_launches() - n == launches
        elif how == "no overlap of launches":
            fl.set_option("pdl", 0)
            try:
                call()
                torch.cuda.synchronize()
            finally:
                fl.set_option("pdl", 1)
        elif how == "torch graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
            for t, b in zip(made, before):
                t.view(b.dtype).copy_(b)
            graph.replay()
        else:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                graph = fl.Graph.capture(call)
            for t, b in zip(made, before):
                t.view(b.dtype).copy_(b)
            # (a workspace that the call made belongs to the graph: this must not get it)
            other = [torch.full((M * 768 * 2 + 4096,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(4)]
            with torch.cuda.stream(side):
                other += [torch.full((M * 768 * 2 + 4096,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(4)]
            torch.cuda.synchronize()
            graph.launch()
            torch.cuda.synchronize()
            assert all((t == 0xff).all() for t in other)
            graph.close()
        torch.cuda.synchronize()
        for t, s in zip(made, want):
            assert torch.equal(t.view(torch.uint8), s.view(torch.uint8))
    fl.device_status()


def test_tensors_made_on_a_stream():
    """A call on a stream other than the current one takes its workspace and outputs from that stream's memory, so that
    they are not blocks which the current stream's kernels still write."""
    rng = gen(44)
    w = w4_tensors(rng, 512, 512, 64, True, "bf16")
    x, gamma = put(rng.standard_normal((300, 512)), "bf16"), put(1 + 0.1 * rng.standard_normal(512), "bf16")
    want = fl.w4_gemm(x, *w[:2], zeros=w[2], gamma=gamma)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        t = torch.empty((300, 512), dtype=torch.bfloat16, device="cuda")
        for _ in range(50):
            t.fill_(3.0)
        del t
        got = fl.w4_gemm(x, *w[:2], zeros=w[2], gamma=gamma, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    fl.device_status(side)


def test_python_refusals():
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    q, s = torch.zeros((64, 128), dtype=torch.uint8, device="cuda"), torch.ones((64, 4), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        fl.w4_gemm(x, q, s.float())
    with pytest.raises(ValueError):
        fl.w4_gemm(x, q[:, :64], s)
    with pytest.raises(ValueError):
        fl.w4_gemm(x, q, s, zeros=torch.zeros((64, 2), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fl.w4_gemm(x, q, s, bias=torch.zeros(60, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        fl.w4_gemm(x.cpu(), q, s)
    with pytest.raises(ValueError):
        fl.w4_gemm(x, q, s, out=torch.zeros((4, 63), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(fl.FusedLinError):
        fl.w4_gemm(x[:0], q, s)
    with pytest.raises(ValueError):
        fl.w4_quantize(x, 48)
    h = x.unflatten(1, (4, 64))
    f = torch.ones(32, device="cuda")
    with pytest.raises(TypeError):
        fl.rope(h, None, torch.zeros(4, dtype=torch.int64, device="cuda"), f)
    with pytest.raises(ValueError):
        fl.rope(h, None, torch.zeros((2, 4), dtype=torch.int32, device="cuda"), f)
    with pytest.raises(ValueError):
        fl.rope(h, None, torch.zeros((2, 4), dtype=torch.int32, device="cuda"), f, sections=(16, 17))
    with pytest.raises(ValueError):
        fl.rope(h.transpose(1, 2), None, torch.zeros(4, dtype=torch.int32, device="cuda"), f)
    empty = fl.rope(h[:0], h[:0], torch.zeros(0, dtype=torch.int32, device="cuda"), f)
    assert empty[0].shape == (0, 4, 64)
    (kc, vc), (ks, vs) = cache(2, 16, 4, 64, "int8")
    table, start = torch.zeros((4, 1), dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        fl.kv_write(h[..., :32], h[..., :32], kc, vc, ks, vs, table, start)
    with pytest.raises(TypeError):
        fl.kv_write(h, h, kc.float(), vc, ks, vs, table, start)
    with pytest.raises(TypeError):
        fl.kv_write(h, h, kc, vc, ks, vs, table.long(), start)
    with pytest.raises(ValueError):
        fl.kv_write(h, h, kc, vc, ks, vs, table, None)
    with pytest.raises(ValueError):
        fl.kv_read(kc, vc, ks, vs, table, None, start=start)
    with pytest.raises(fl.FusedLinError):  # outputs that are one another
        fl.kv_read(kc, vc, ks, vs, table, None, start=start, out_k=h, out_v=h)
    fl.kv_write(h[:0], h[:0], kc, vc, ks, vs, table, start)
    fl.device_status()
