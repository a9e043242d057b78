"""Edges of the serving operators on the GPU: ranges, long rows, small activations, what graphs keep (needs an sm_103a GPU).

Bounds are those of tests/test_gpu_serving.py, u the largest relative error of one rounding to the dtype (2^-8 bf16,
2^-11 fp16 with the type's smallest values next to it), each derived beside its test. The cache's scales are amax times
1 / top rounded to fp32, as the header has them, which may differ from fp32's quotient in the last bit.
"""
import numpy as np
import pytest
import torch

import gemm_epilogue_tma_gb300 as fl
import oracle
from test_gpu_serving import (DT, U, cache, f64, gen, library, put, serving_calls, snapshot, w4_check,  # noqa: F401
                              w4_ref, w4_tensors)  # (library: the fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# range of x * gamma
# ---------------------------------------------------------------------------
def wide_rows(rng, M, K, size):
    """Rows of about `size`, each with a few channels up to 40 times larger, within fp16."""
    x = rng.standard_normal((M, K)) * np.where(rng.random((M, K)) < 0.01, 40.0, 1.0) * size
    return put(np.clip(x, -65504.0, 65504.0), "f16")


@pytest.mark.parametrize("size,eps", [(1e4, 1e-6), (6e4, 1e-6), (1e-4, 1e-12), (3e-6, 0.0), (1.0, 1e-6)])
@pytest.mark.parametrize("M", [1, 2, 4, 8, 24, 300])
def test_w4_gemm_takes_every_fp16_row(M, size, eps):
    """The normalised row is of size 1 whatever x is, so the answer is finite and as exact for rows near fp16's largest
    and smallest values as for rows of size 1, on few rows and on many. Element by element: x * gamma (or the weight
    with gamma in it), the weight and the output rounded once (2.1 u of the terms, u of the sum), sums fp32 with
    2^-22 per term at most; no term for values lost to the type's smallest."""
    rng = gen(50, M, 64 + int(np.log2(size)))
    K, N, group = 1024, 264, 64
    x = wide_rows(rng, M, K, size)
    if M > 1:
        x[M // 2] = put(rng.standard_normal(K), "f16")           # sizes of rows do not mix
    gamma = put(3 + rng.uniform(0, 60, K) * (rng.random(K) < 0.1), "f16")
    w = w4_tensors(rng, N, K, group, True, "f16")
    got = f64(fl.w4_gemm(x, w[0], w[1], zeros=w[2], gamma=gamma, eps=eps))
    fl.device_status()
    y, mag, _ = w4_ref(x, w, gamma, eps)
    assert np.isfinite(got).all()
    u = U["f16"]
    bound = u * np.abs(y) + (2.1 * u + K * 2.0 ** -22) * mag + 2.0 ** -25
    err = np.abs(got - y)
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("M", [1, 4, 7, 20])
def test_w4_swiglu_ffn_takes_large_fp16_rows(M):
    """The block's gate and up products of rows whose x * gamma passes 65504: finite, and the residual's own size."""
    rng = gen(51, M)
    D, F = 512, 256
    x = wide_rows(rng, M, D, 3e3)
    gamma = put(np.full(D, 30.0), "f16")
    Wg, Wu, Wd = (w4_tensors(rng, n, k, 64, False, "f16") for n, k in ((F, D), (F, D), (D, F)))
    got = f64(fl.w4_swiglu_ffn(x, gamma, Wg[:2], Wu[:2], Wd[:2]))
    fl.device_status()
    g, gm, _ = w4_ref(x, Wg, gamma, 1e-6)
    v, vm, _ = w4_ref(x, Wu, gamma, 1e-6)
    h = oracle.silu(g) * v
    assert np.abs(h).max() < 6e4                                  # h itself fits
    W = oracle.w4_weight(Wd[0].cpu().numpy(), f64(Wd[1]))
    y = h @ W.T + f64(x)
    # the gate's and the up product's errors through silu (slope below 1.1), h's rounding, the down product's and the output's
    u = U["f16"]
    dg, dv = ((1.05 * u + D * 2.0 ** -22) * m for m in (gm, vm))
    dh = (1.1 * dg + 2.0 ** -9 * np.abs(g)) * (np.abs(v) + dv) + np.abs(oracle.silu(g)) * dv + u * np.abs(h)
    bound = u * np.abs(y) + dh @ np.abs(W).T + (1.05 * u + F * 2.0 ** -22) * (np.abs(h) @ np.abs(W).T)
    # (fp16 ends at 65504, and 65520 and more round to infinity: the residual of one element is 65504 itself, and its exact
    # answer -65645. So an infinity is right where the answer may lie past 65520 within its bound.)
    with np.errstate(invalid="ignore"):
        past = np.isinf(got) & (got * y > 0) & (np.abs(y) + bound >= 65520)
    assert (past | (np.abs(got - y) <= bound)).all()


def test_w4_gemm_row_without_a_finite_sum_stays_alone():
    """An infinite or NaN element makes its own row so, zero rows stay zero, and rows beside them keep their bits."""
    rng = gen(52)
    K, N = 512, 136
    w = w4_tensors(rng, N, K, 128, False, "f16")
    gamma = put(1 + 0.1 * rng.standard_normal(K), "f16")
    for M in (4, 8, 20):
        x = put(rng.standard_normal((M, K)), "f16")
        x[0] *= 3e4 / 8
        want = fl.w4_gemm(x, *w[:2], gamma=gamma)
        assert torch.isfinite(want).all()
        x2 = x.clone()
        x2[1, 5], x2[2, 9] = float("inf"), float("nan")
        x2[3] = 0
        got = fl.w4_gemm(x2, *w[:2], gamma=gamma)
        fl.device_status()
        assert not torch.isfinite(got[1]).any() and torch.isnan(got[2]).all() and (got[3] == 0).all()
        keep = [m for m in range(M) if m not in (1, 2, 3)]
        assert torch.equal(got[keep], want[keep])


# ---------------------------------------------------------------------------
# long rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K,group", [(1, 136, 28672, 128), (4, 264, 8192, 64), (7, 264, 14336, 128), (8, 264, 12736, 64),
                                         (8, 264, 12800, 64), (8, 136, 28672, 128), (24, 264, 14336, 128), (40, 264, 14336, 32),
                                         (300, 136, 28672, 128)])
def test_w4_gemm_of_long_rows(dt, M, N, K, group):
    """K past what eight rows take in shared memory (12736), on both sides of it and on both kernels."""
    for k, (zeros, norm) in enumerate([(True, True), (False, False)]):
        rng = gen(58, M, K, k)
        x = put(rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.01, 20.0, 1.0), dt)
        w = w4_tensors(rng, N, K, group, zeros, dt)
        gamma = put(1 + 0.1 * rng.standard_normal(K), dt) if norm else None
        got = fl.w4_gemm(x, w[0], w[1], zeros=w[2], gamma=gamma)
        fl.device_status()
        y, mag, sq = w4_ref(x, w, gamma, 1e-6)
        w4_check(got, y, mag, sq, K, dt, what=f"{dt} {M}x{N}x{K} {k}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,group", [(1, 26496, 128), (2, 13248, 32), (3, 8832, 64), (4, 6592, 32), (4, 6528, 128)])
def test_w4_gemm_up_to_four_rows_of_the_longest_k(dt, M, K, group):
    """Up to M (K + 32) = 26624 the rows' x * gamma is not rounded to speak of: u^2 of the terms, the output's u, and
    the sums' K 2^-24 per term at most (fp32 sums of K terms, each addition off by 2^-24 of a partial sum that is
    at most the terms' sum; a group's within the matrix unit, so K is far above their number)."""
    rng = gen(59, M, K)
    N = 136
    assert M * ((K + 63) // 64 * 64 + 32) <= 26624
    x = put(rng.standard_normal((M, K)), dt)
    w = w4_tensors(rng, N, K, group, False, dt)
    gamma = put(1 + 0.1 * rng.standard_normal(K), dt)
    got = f64(fl.w4_gemm(x, w[0], w[1], gamma=gamma))
    fl.device_status()
    y, mag, _ = w4_ref(x, w, gamma, 1e-6)
    u = U[dt]
    err = np.abs(got - y)
    assert (err <= u * np.abs(y) + (u * u + K * 2.0 ** -24) * mag + 2.0 ** -25).all()
    # mean square: the output's rounding, and a tenth of it for all else
    assert np.sqrt((err ** 2).mean()) <= 1.1 * u / np.sqrt(3) * np.sqrt((y ** 2).mean())


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M", [1, 3, 8, 20, 200])
def test_w4_swiglu_ffn_of_a_wide_block(dt, M):
    """F = 14336: the down product's rows are past the decode kernel's room from eight rows on."""
    rng = gen(60, M)
    D, F, group = 512, 14336, 128
    x, gamma = put(rng.standard_normal((M, D)), dt), put(1 + 0.1 * rng.standard_normal(D), dt)
    Wg, Wu, Wd = (w4_tensors(rng, n, k, group, False, dt) for n, k in ((F, D), (F, D), (D, F)))
    got = f64(fl.w4_swiglu_ffn(x, gamma, Wg[:2], Wu[:2], Wd[:2]))
    fl.device_status()
    g, gm, _ = w4_ref(x, Wg, gamma, 1e-6)
    v, vm, _ = w4_ref(x, Wu, gamma, 1e-6)
    h = oracle.silu(g) * v
    W = oracle.w4_weight(Wd[0].cpu().numpy(), f64(Wd[1]))
    y = h @ W.T + f64(x)
    u = U[dt]
    dg, dv = ((2.1 * u + D * 2.0 ** -22) * m for m in (gm, vm))
    dh = (1.1 * dg + 2.0 ** -15 * np.abs(g)) * (np.abs(v) + dv) + np.abs(oracle.silu(g)) * dv + u * np.abs(h)
    bound = u * np.abs(y) + dh @ np.abs(W).T + (1.05 * u + F * 2.0 ** -22) * (np.abs(h) @ np.abs(W).T)
    err = np.abs(got - y)
    assert (err <= bound).all(), (err / bound).max()
    assert np.sqrt((err ** 2).mean()) <= 4 * u * np.sqrt((y ** 2).mean())


# ---------------------------------------------------------------------------
# activations
# ---------------------------------------------------------------------------
def exact_act(name, v):
    """v sigmoid(z), which cancels nowhere."""
    z = v if name == "silu" else 2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)
    return v / (1 + np.exp(-np.minimum(np.maximum(z, -700), 700)))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [1, 8, 40, 300])
def test_w4_gemm_activation_of_negative_values(dt, act, M):
    """Pre-activations that are exact (x times a code of 1, a bias; all of them multiples of 1/8), mostly -10 .. -2, where
    the activation is small next to them: the output is its rounding alone. The kernel's sigmoid form is within 2^-16 of
    the value (an exponential within 2^-18 for arguments down to -20, a sum, a quotient of 2^-22), or 0 where its
    exponential passes 2^126: below 16 * 2^-126."""
    rng = gen(53, M)
    K, N = 128, 512
    x = np.zeros((M, K))
    x[:, 0] = np.round(rng.uniform(-2, 2, M) * 8) / 8
    b = np.round(np.concatenate([rng.uniform(-8, -4, N - 64), rng.uniform(-14, 14, 62), [0, -0.5]]) * 8) / 8
    code = np.full((N, K), 8)
    code[:, 0] = 9
    q, s = put(oracle.w4_pack(code)), put(np.ones((N, 1)), dt)
    got = f64(fl.w4_gemm(put(x, dt), q, s, bias=put(b, dt), act=act))
    fl.device_status()
    y = exact_act(act, x[:, :1] + b)
    least = 2.0 ** -25 if dt == "f16" else 2.0 ** -122
    bound = (U[dt] + 2.0 ** -16) * np.abs(y) + least
    err = np.abs(got - y)
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M", [2, 6, 40, 300])
def test_w4_swiglu_ffn_activation_of_negative_gates(dt, M):
    """Gates that are exact (rows of one size, whose norm is 1; one code a row), up 1, the down product an identity: the
    output is x + silu(gate) with h's rounding and its own."""
    D, F = 256, 256
    gate = np.linspace(-12, -1, F)
    x = np.full((M, D), 2.0 ** -10)
    x[:, 1::2] *= -1
    gamma = put(np.ones(D), dt)
    code = np.full((F, D), 8)
    code[:, 0] = 9                                                             # x[:, 0] / rms = 1
    one = put(oracle.w4_pack(code))
    sg = np.tile(gate[:, None], (1, D // 64))
    Wg, Wu = (one, put(sg, dt)), (one, put(np.ones((F, D // 64)), dt))
    code = np.full((D, F), 8)
    np.fill_diagonal(code, 9)
    Wd = put(oracle.w4_pack(code)), put(np.ones((D, F // 64)), dt)
    got = f64(fl.w4_swiglu_ffn(put(x, dt), gamma, Wg, Wu, Wd, eps=0.0))
    fl.device_status()
    h = exact_act("silu", f64(Wg[1])[:, 0])[None]
    y = h + x
    # (the norm's factor and the sums: 2^-21 of the gate, which changes h by its slope (1 + |gate|) h / gate, and of up)
    small = 2.0 ** -21 * (2 + np.abs(f64(Wg[1])[:, 0]))[None]
    u, least = U[dt], 2.0 ** -25 if dt == "f16" else 0.0
    bound = u * np.abs(y) + (u + 2.0 ** -16 + small) * np.abs(h) * (1 + u) + 2 * least
    err = np.abs(got - y)
    assert (err <= bound).all(), (err / bound).max()


# ---------------------------------------------------------------------------
# graphs
# ---------------------------------------------------------------------------
def test_library_graph_keeps_what_its_calls_made():
    """A captured chain whose calls make their own outputs and workspaces, dropped as soon as the next call has seen
    them: tensors allocated after the capture, on either stream, are not written by replays, and each replay gives the
    direct calls' bits."""
    rng = gen(54)
    M, D, F = 40, 512, 768
    x = put(rng.standard_normal((M, D)), "bf16")
    gamma = put(1 + 0.1 * rng.standard_normal(D), "bf16")
    W16 = [put(rng.standard_normal(s) / np.sqrt(s[1]), "bf16") for s in ((F, D), (F, D), (D, F), (D, D))]
    Q = [fl.w4_quantize(w, 64) for w in W16]
    pos, f = put(np.arange(M, dtype=np.int32)), put((1e4 ** (-np.arange(32) / 32)).astype(np.float32))
    y = torch.zeros_like(x)

    def chain():
        h = fl.swiglu_ffn(fl.norm_gemm(x, gamma, W16[3]), gamma, *W16[:3])
        h = fl.w4_swiglu_ffn(fl.w4_gemm(h, *Q[3], gamma=gamma), gamma, *Q[:3])
        q, _ = fl.rope(h.unflatten(1, (8, 64)), None, pos, f)
        fl.w4_gemm(fl.rms_norm(q.flatten(1), gamma), *fl.w4_quantize(W16[3], 32), out=y)
    chain()
    torch.cuda.synchronize()
    want = y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain()                                     # (this stream's blocks exist before the capture)
        side.synchronize()
        graph = fl.Graph.capture(chain)

    def guards():
        return [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in (64, 4096, 40960, M * D * 2, M * F * 2, D * D)
                for _ in range(4)]
    other = guards()
    with torch.cuda.stream(side):
        other += guards()
    torch.cuda.synchronize()
    for _ in range(3):
        y.zero_()
        torch.cuda.synchronize()
        graph.launch()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and all((t == 0xff).all() for t in other)
    graph.close()
    fl.device_status()
    fl.device_status(side)


def test_graph_of_a_layer_whose_attachment_was_replaced():
    """A graph goes on with the positions that were attached when it was captured, although nobody else holds them."""
    rng = gen(55)
    M, D, Dkv, F, hd = 3, 256, 128, 256, 64
    e = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    T = {n: put(rng.standard_normal(s) / np.sqrt(s[-1]), "f16") for n, s in
         (("Wq", (D, D)), ("Wk", (Dkv, D)), ("Wv", (Dkv, D)), ("Wo", (D, D)), ("Wg", (F, D)), ("Wu", (F, D)), ("Wd", (D, F)))}
    one = put(np.ones(D), "f16")
    T.update(x=put(rng.standard_normal((M, D)), "f16"), gamma_attn=one, gamma_ffn=one, q=e(M, D), k=e(M, Dkv), v=e(M, Dkv),
             attn=e(M, D), h=e(M, D), out=e(M, D))
    layer = fl.DecoderLayer(**T)
    f = put((1e4 ** (-np.arange(32) / 32)).astype(np.float32))

    def i32(*v):
        return put(np.array(v, dtype=np.int32))
    layer.attach_cache(hd, positions=i32(5, 900, 70), inv_freq=f)
    layer.issue(0)
    torch.cuda.synchronize()
    want = T["q"].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = fl.Graph.capture(lambda: layer.issue(0))
    layer.attach_cache(hd, positions=i32(1, 2, 3), inv_freq=f)
    guards = [torch.full((3,), 7, dtype=torch.int32, device="cuda") for _ in range(64)]
    layer.issue(0)
    torch.cuda.synchronize()
    assert not torch.equal(T["q"], want)
    graph.launch()
    torch.cuda.synchronize()
    assert torch.equal(T["q"], want) and all((g == 7).all() for g in guards)
    graph.close()
    layer.close()
    fl.device_status()


# ---------------------------------------------------------------------------
# device status
# ---------------------------------------------------------------------------
def skipped_row(stream):
    """A row without a page, written on `stream`."""
    (kc, vc), (ks, vs) = cache(1, 16, 1, 64, "int8")
    k = torch.ones((3, 1, 64), dtype=torch.float16, device="cuda")
    table = put(np.zeros((3, 1), dtype=np.int32))
    start = put(np.array([0, 1, 99], dtype=np.int32))
    torch.cuda.synchronize()
    fl.kv_write(k, k, kc, vc, ks, vs, table, start, stream=stream)
    return kc, vc, ks, vs, k, table, start


def test_a_timeout_and_a_skipped_row_are_told_one_after_the_other():
    """Each stream has both words: the timeout is told first and the row by the next call, with its number; another
    stream's stay its own."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    kept = skipped_row(a), skipped_row(b)
    fl.debug_wait_timeout(1000, stream=a)
    told = []
    for stream in (a, a, a, b, b):
        try:
            fl.device_status(stream)
            told.append(0)
        except fl.FusedLinError as e:
            told.append(e.status)
            assert e.status != 7 or "row 2" in str(e)
    assert told == [6, 7, 0, 7, 0]
    del kept


# ---------------------------------------------------------------------------
# positions
# ---------------------------------------------------------------------------
def test_rope_of_expanded_positions():
    """Text rows under several axes: one row of positions, expanded, gives what its copies give, also attached to a layer."""
    rng = gen(56)
    M, D, hd = 7, 256, 64
    q, k = (put(rng.standard_normal((M, h, hd)), "bf16") for h in (4, 2))
    row, f = put(rng.integers(0, 9000, M).astype(np.int32)), put((1e4 ** (-np.arange(32) / 32)).astype(np.float32))
    want = fl.rope(q, k, row.repeat(3, 1), f, sections=(16, 8, 8))
    got = fl.rope(q, k, row.expand(3, -1), f, sections=(16, 8, 8))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(got[0], fl.rope(q, None, row, f)[0])
    T = {n: put(rng.standard_normal(s) / 16, "bf16") for n, s in
         (("Wq", (D, D)), ("Wk", (128, D)), ("Wv", (128, D)), ("Wo", (D, D)), ("Wg", (64, D)), ("Wu", (64, D)), ("Wd", (D, 64)),
          ("x", (M, D)), ("q", (M, D)), ("k", (M, 128)), ("v", (M, 128)), ("attn", (M, D)), ("h", (M, D)), ("out", (M, D)))}
    T["gamma_attn"] = T["gamma_ffn"] = put(np.ones(D), "bf16")
    layer = fl.DecoderLayer(**T)
    out = []
    for pos in (row.repeat(3, 1), row.expand(3, -1)):
        layer.attach_cache(hd, positions=pos, inv_freq=f, sections=(16, 8, 8))
        layer.issue(0)
        torch.cuda.synchronize()
        out.append((T["q"].clone(), T["k"].clone()))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    with pytest.raises(ValueError):
        layer.attach_cache(hd, positions=row.repeat(3, 2)[:, ::2], inv_freq=f, sections=(16, 8, 8))
    layer.close()
    fl.device_status()


def test_rope_of_as_many_rows_as_an_int_holds():
    """2^31 - 1 rows: places past 2^32 bytes, and a row count next to which no sum of ints may be formed."""
    rows, hd = 2 ** 31 - 1, 8
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    x = put(gen(57).standard_normal((1, 1, hd)), "f16")
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    f = put((1e4 ** (-np.arange(4) / 4)).astype(np.float32))
    got = fl.rope(x.expand(rows, 1, hd), None, pos, f)[0]       # (every row the same x)
    fl.device_status()
    at = torch.tensor([0, 1, 5000, 2 ** 28 - 1, 2 ** 28, 2 ** 30 + 3, rows - 2, rows - 1], device="cuda")
    want = oracle.rope(np.tile(f64(x), (len(at), 1, 1)), [at.cpu().numpy()], f.cpu().numpy(), [0] * 4)
    pair = np.abs(f64(x)).reshape(2, 4).sum(0)
    bound = U["f16"] * np.abs(want) + 2.0 ** -21 * np.tile(pair, 2) + 2.0 ** -25
    assert (np.abs(f64(got[at]) - want) <= bound).all()
    del got, pos
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# every way of issuing, from tensors that do not hold the answer
# ---------------------------------------------------------------------------
def put_back(tensors, held):
    for t, h in zip(tensors, held):
        t.view(h.dtype).copy_(h)


@pytest.mark.parametrize("M", [2, 300])
@pytest.mark.parametrize("pdl", [1, 0])
def test_second_calls_write_the_result_again(M, pdl):
    """The same call on the same tensors, which hold what they held before the first one: its whole result again, with and
    without programmatic launches. (Of a tensor that the call fills, nothing of the old content is left.)"""
    for call, made, launches in serving_calls(gen(61, M), M):
        before = snapshot(made)
        call()
        torch.cuda.synchronize()
        want = snapshot(made)
        assert not all(torch.equal(w, b) for w, b in zip(want, before))
        fl.set_option("pdl", pdl)
        try:
            for fill in (None, 0x5a):
                put_back(made, before)
                if fill is not None and made[0].dim() != 4:            # (all but the cache, of which a call writes places)
                    for t in made:
                        t.view(torch.uint8).fill_(fill)
                torch.cuda.synchronize()
                n = fl.kernel_launches()
                call()
                torch.cuda.synchronize()
                assert fl.kernel_launches() - n == launches
                assert all(torch.equal(t.view(torch.uint8), w.view(torch.uint8)) for t, w in zip(made, want))
        finally:
            fl.set_option("pdl", 1)
    fl.device_status()


def test_replayed_decode_step_writes_the_cache():
    """A captured decode step (products, rotation, cache written and read back, FFN), replayed from the cache as it was
    before the step and with every other tensor poisoned: the direct step's bits everywhere, twice."""
    rng = gen(62)
    D, hq, hk, hd, F, page, B = 512, 4, 2, 128, 1024, 16, 2
    W = {n: fl.w4_quantize(put(rng.standard_normal(s) / np.sqrt(s[1]), "bf16"), 64) for n, s in
         (("qkv", ((hq + 2 * hk) * hd, D)), ("o", (D, hq * hd)), ("g", (F, D)), ("u", (F, D)), ("d", (D, F)))}
    gamma, x = put(1 + 0.1 * rng.standard_normal(D), "bf16"), put(rng.standard_normal((B, D)), "bf16")
    f = put((1e4 ** (-np.arange(64) / 64)).astype(np.float32))

    def i32(*v):
        return put(np.array(v, dtype=np.int32))
    table, at, ctx = put(np.array([[4, 1], [0, 3]], dtype=np.int32)), i32(15, 7), i32(0, 16, 24)
    (kc, vc), (ks, vs) = cache(5, page, hk, hd, "int8")
    held = [kc, vc, ks, vs]
    for t in held[:2]:
        t.copy_(put(rng.integers(-127, 128, t.shape).astype(np.int8)))
    e = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    qkv, q1, ck, cv, h, y = e(B, (hq + 2 * hk) * hd), e(B, hq, hd), e(24, hk, hd), e(24, hk, hd), e(B, D), e(B, D)
    ws = torch.empty(fl.w4_swiglu_ffn_workspace_size(B, D, F), dtype=torch.uint8, device="cuda")
    out = [qkv, q1, ck, cv, h, y]

    def step():
        fl.w4_gemm(x, *W["qkv"], gamma=gamma, out=qkv)
        q, k, v = (t.unflatten(1, (-1, hd)) for t in qkv.split((hq * hd, hk * hd, hk * hd), 1))
        fl.rope(q, k, at, f, out_q=q1, out_k=k)
        fl.kv_write(k, v, kc, vc, ks, vs, table, at)
        fl.kv_read(kc, vc, ks, vs, table, ctx, out_k=ck, out_v=cv)
        fl.w4_gemm(q1.flatten(1), *W["o"], residual=x, out=h)
        fl.w4_swiglu_ffn(h, gamma, W["g"], W["u"], W["d"], out=y, workspace=ws)
    before = snapshot(held)
    step()
    fl.device_status()
    want = snapshot(held + out)
    assert all(not torch.equal(a, b) for a, b in zip(want, before))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = fl.Graph.capture(step)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        put_back(held, before)
        for t in out + [ws]:
            t.view(torch.uint8).fill_(0xff)
        torch.cuda.synchronize()
        graph.launch()
        torch.cuda.synchronize()
        assert all(torch.equal(t.view(torch.uint8), w.view(torch.uint8)) for t, w in zip(held + out, want))
    graph.close()
    fl.device_status()
    fl.device_status(side)
