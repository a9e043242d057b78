"""The serving operators without a GPU: refusals of the C ABI, pins of their oracle, and the kernels' index and
rounding steps restated on the CPU."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import gemm_epilogue_tma_gb300 as fl
import oracle
from gemm_epilogue_tma_gb300 import _build

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE, CUDA, TIMEOUT, RANGE = range(8)
BASE = 0x7F0000000000
PASSES = (UNSUPPORTED,)  # validation passed: the device query fails on this machine


@pytest.fixture(scope="module")
def L():
    _build.build()
    return fl.lib()


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses must not reach a device")


def addr(i, off=0):
    return BASE + i * (1 << 36) + off


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def weight(i=10, **kw):
    return fl.W4Weight(**{**dict(q=addr(i), scales=addr(i + 1), zeros=None, group=64), **kw})


@no_gpu
def test_w4_quantize_refusals(L):
    def call(W=addr(0), q=addr(1), s=addr(2), N=64, K=256, group=64, dt=0):
        return L.fl_w4_quantize(W, q, s, N, K, group, dt, None)
    assert call() in PASSES
    assert call(W=None) == INVALID and call(q=None) == INVALID and call(s=None) == INVALID
    assert call(group=16) == INVALID and call(group=0) == INVALID and call(group=256) == INVALID
    assert call(N=0) == INVALID and call(K=0) == INVALID and call(K=-64) == INVALID
    assert call(K=96) == ALIGN and call(N=12) == ALIGN
    assert call(q=addr(1, 4)) == ALIGN and call(W=addr(0, 2)) == ALIGN
    assert call(dt=2) == INVALID
    assert call(q=addr(0, 64)) == INVALID and call(s=addr(1, 16)) == INVALID


@no_gpu
def test_w4_gemm_refusals(L):
    def call(x=addr(0), gamma=addr(1), W=None, bias=addr(2), res=addr(3), out=addr(4), M=5, N=64, K=256, eps=1e-6,
             act=0, ws=addr(5), size=1 << 30, dt=0, no_weight=False):
        w = None if no_weight else ctypes.byref(W or weight())
        return L.fl_w4_gemm(x, gamma, w, bias, res, out, M, N, K, eps, act, ws, size, dt, None)
    assert call() in PASSES
    assert call(gamma=None, bias=None, res=None) in PASSES
    assert call(res=addr(4)) in PASSES
    assert call(no_weight=True) == INVALID
    assert call(x=None) == INVALID and call(out=None) == INVALID
    assert call(W=weight(q=None)) == INVALID and call(W=weight(scales=None)) == INVALID
    assert call(W=weight(group=48)) == INVALID and call(W=weight(group=128), K=192) == ALIGN
    assert call(W=weight(q=addr(10, 8))) == ALIGN and call(W=weight(zeros=addr(12, 2))) == ALIGN
    assert call(M=0) == INVALID and call(N=0) == INVALID and call(N=60) == ALIGN
    assert call(N=0x7ffffff8) == UNSUPPORTED and "too many rows" in fl.last_error()
    assert call(act=4) == INVALID and call(dt=7) == INVALID
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID and call(eps=float("inf")) == INVALID
    assert call(out=addr(0, 16)) == INVALID and call(out=addr(10, 16)) == INVALID and call(out=addr(11)) == INVALID
    assert call(res=addr(4, 16)) == INVALID
    for rows in (1, 9, 300):
        need = fl.w4_gemm_workspace_size(rows, 256, True)
        if need:
            assert call(M=rows, ws=None) == WORKSPACE and call(M=rows, size=need - 1) == WORKSPACE
            assert call(M=rows, ws=addr(5, 8)) == ALIGN
            assert call(M=rows, ws=addr(0)) == INVALID and call(M=rows, ws=addr(4)) == INVALID
            assert call(M=rows, ws=addr(3)) == INVALID


@no_gpu
def test_w4_swiglu_refusals(L):
    def call(x=addr(0), gamma=addr(1), g=None, u=None, d=None, bias=addr(2), out=addr(4), M=5, D=128, F=256, ws=addr(5),
             size=1 << 30):
        g, u, d = g or weight(20), u or weight(22), d or weight(24)
        return L.fl_w4_swiglu_ffn(x, gamma, ctypes.byref(g), ctypes.byref(u), ctypes.byref(d), bias, out, M, D, F, 1e-6,
                                  ws, size, 1, None)
    assert call() in PASSES
    assert call(bias=None) in PASSES
    assert call(gamma=None) == INVALID and call(x=None) == INVALID
    assert call(u=weight(22, group=128)) == INVALID          # another group than Wg's
    assert call(u=weight(22, zeros=addr(26))) == INVALID     # zero points on one of the pair
    assert call(g=weight(20, zeros=addr(27)), u=weight(22, zeros=addr(26))) in PASSES
    assert call(d=weight(24, group=128), F=192) == ALIGN
    assert call(ws=None) == WORKSPACE and call(size=fl.w4_swiglu_ffn_workspace_size(5, 128, 256) - 1) == WORKSPACE
    assert call(ws=addr(20, 64)) == INVALID and call(ws=addr(4)) == INVALID and call(ws=addr(0)) == INVALID
    assert call(out=addr(0)) == INVALID and call(out=addr(23)) == INVALID


def rope_desc(**kw):
    d = dict(dtype=1, rows=10, heads_q=4, heads_k=2, head_dim=64, rotary_dim=64, n_axes=1, interleaved=0, inverse=0,
             axis_of=None, positions=addr(0), positions_stride=10, inv_freq=addr(1), q=addr(2), k=addr(3),
             q_out=addr(4), k_out=addr(5), q_row=256, q_head=64, k_row=128, k_head=64, q_out_row=256, q_out_head=64,
             k_out_row=128, k_out_head=64)
    return fl.RopeDesc(**{**d, **kw})


@no_gpu
def test_rope_refusals(L):
    def call(**kw):
        return L.fl_rope(ctypes.byref(rope_desc(**kw)), None)
    assert L.fl_rope(None, None) == INVALID
    assert call() in PASSES
    assert call(rows=0, q=None) == OK
    assert call(heads_k=0, k=None, k_out=None) in PASSES
    assert call(q_out=addr(2), k_out=addr(3)) in PASSES                       # in place
    assert call(q_out=addr(2), q_out_row=512) == INVALID                      # in place needs the same strides
    assert call(q_out=addr(2, 128)) == INVALID and call(q_out=addr(3)) == INVALID and call(k_out=addr(4)) == INVALID
    # q and k as column ranges of one matrix, in place and to another such matrix
    both = dict(q_row=384, k_row=384, q=addr(2), k=addr(2, 512), q_out_row=384, k_out_row=384)
    assert call(**both, q_out=addr(2), k_out=addr(2, 512)) in PASSES
    assert call(**both, q_out=addr(4), k_out=addr(4, 512)) in PASSES
    assert call(**both, q_out=addr(4), k_out=addr(4, 510)) == INVALID
    assert call(**both, q_out=addr(2, 512), k_out=addr(2)) == INVALID
    assert call(rotary_dim=63) == INVALID and call(rotary_dim=66) == INVALID and call(rotary_dim=0) == INVALID
    assert call(head_dim=520, rotary_dim=64) == UNSUPPORTED
    assert call(heads_q=4096) == UNSUPPORTED and "heads" in fl.last_error()
    assert call(n_axes=0) == INVALID and call(n_axes=5) == INVALID
    assert call(n_axes=2, axis_of=bytes([0, 1] * 16)) in PASSES
    assert call(n_axes=2, axis_of=bytes([0, 2] * 16)) == INVALID
    assert call(n_axes=2, axis_of=bytes(32), positions_stride=9) == INVALID
    assert call(dtype=3) == INVALID and call(rows=-1) == INVALID and call(heads_q=0) == INVALID
    assert call(positions=None) == INVALID and call(k=None) == INVALID
    assert call(q=addr(2, 1)) == ALIGN and call(positions=addr(0, 2)) == ALIGN
    assert call(q=addr(2, 2)) in PASSES                                       # the scalar form
    assert call(q_out_row=32) == INVALID and call(q_out_head=32) == INVALID and call(q_row=-256) == INVALID
    assert call(q_row=0, q_head=0) in PASSES                                  # a broadcast input
    assert call(q_out=addr(0)) == INVALID and call(k_out=addr(1)) == INVALID


def kv_desc(**kw):
    d = dict(dtype=1, format=0, rows=20, heads=2, head_dim=64, page_size=16, n_pages=8, n_seqs=3, table_pages=4,
             table_stride=4, page_table=addr(0), cu_rows=addr(1), start=addr(2), k=addr(3), v=addr(4), k_row=128,
             k_head=64, v_row=128, v_head=64, k_cache=addr(5), v_cache=addr(6), k_scale=addr(7), v_scale=addr(8))
    return fl.KvDesc(**{**d, **kw})


@no_gpu
@pytest.mark.parametrize("name", ["fl_kv_write", "fl_kv_read"])
def test_kv_refusals(L, name):
    fn, write = getattr(L, name), name == "fl_kv_write"

    def call(**kw):
        return fn(ctypes.byref(kv_desc(**kw)), None)
    assert fn(None, None) == INVALID
    assert call() in PASSES
    assert call(cu_rows=None, start=None) in PASSES
    assert call(rows=0) == OK
    for n in ("rows", "heads", "head_dim", "page_size", "n_pages", "n_seqs", "table_pages"):
        assert call(**{n: -1}) == INVALID
    assert call(head_dim=60) == ALIGN and call(head_dim=264) == UNSUPPORTED
    assert call(n_seqs=(1 << 30) + 1) == UNSUPPORTED and "sequences" in fl.last_error()
    assert call(format=2) == INVALID and call(dtype=2) == INVALID
    for n in ("k", "v", "k_cache", "v_cache", "k_scale", "v_scale", "page_table"):
        assert call(**{n: None}) == INVALID
    assert call(k=addr(3, 8)) == ALIGN and call(k_row=132) == ALIGN and call(page_table=addr(0, 2)) == ALIGN
    assert call(table_stride=3) == INVALID
    # k and v as column ranges of one matrix
    both = dict(k_row=384, v_row=384, k=addr(3), v=addr(3, 256))
    assert call(**both) in PASSES
    assert call(**{**both, "v": addr(3, 240)}) == (UNSUPPORTED if write else INVALID)
    assert call(v=addr(3)) == (UNSUPPORTED if write else INVALID)
    assert call(k_row=0) == (UNSUPPORTED if write else INVALID)               # a broadcast input
    assert call(k_head=32) == (UNSUPPORTED if write else INVALID)
    assert call(k_row=64, k_head=64) == (UNSUPPORTED if write else INVALID)
    # heads-first outputs: [heads, rows, dim]
    assert call(k_row=64, k_head=20 * 64, v_row=64, v_head=20 * 64) in PASSES
    assert call(k_cache=addr(6)) == (INVALID if write else UNSUPPORTED)
    assert call(k_cache=addr(3)) == INVALID and call(k_scale=addr(4)) == INVALID
    assert call(rows=1 << 30, k_row=8, v_row=8, heads=1, head_dim=8) == UNSUPPORTED
    assert "rows" in fl.last_error()


def test_struct_layouts_match_the_header(L):
    # sizes of the C structs on LP64: ints, then 8-byte pointers and strides
    assert ctypes.sizeof(fl.W4Weight) == 32
    assert ctypes.sizeof(fl.RopeDesc) == 9 * 4 + 4 + 4 * 8 + 4 * 8 + 8 * 8
    assert ctypes.sizeof(fl.KvDesc) == 9 * 4 + 4 + 8 + 5 * 8 + 4 * 8 + 4 * 8
    assert ctypes.sizeof(fl.LayerCacheDesc) == 4 * 4 + 4 * 8 + 5 * 4 + 4 + 8 + 7 * 8


def test_attach_cache_refuses_a_null_layer(L):
    assert L.fl_layer_attach_cache(None, None) == INVALID


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------
def round16(dt):
    t = {"f16": torch.float16, "bf16": torch.bfloat16}[dt]
    return lambda v: torch.from_numpy(np.asarray(v, dtype=np.float32)).to(t).double().numpy()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_w4_codes_are_the_exact_nearest(dt):
    rng = np.random.default_rng(5)
    W = round16(dt)(rng.standard_normal((4, 64)))
    W[0, :8] = [7, 3.5, 2.5, 1.5, -2.5, 0.5, -0.5, 0]        # exact ties with a scale of 1
    W[0, 8:32] = 0
    code, scale = oracle.w4_quantize(W, 32, round16(dt), 2.0 ** -24)
    assert scale[0, 0] == 1.0 and list(code[0, :8] - 8) == [7, 4, 2, 2, -2, 0, 0, 0]
    for n in range(4):
        for k in range(64):
            quo = Fraction(W[n, k]) / Fraction(scale[n, k // 32])
            assert abs(quo - (int(code[n, k]) - 8)) <= Fraction(1, 2) or abs(quo) > 7
    back = oracle.w4_weight(oracle.w4_pack(code), scale)
    assert np.abs(back - W).max() <= 0.51 * scale.max()
    z = rng.integers(0, 16, scale.shape)
    assert np.array_equal(oracle.w4_weight(oracle.w4_pack(code), scale, z)[1, :32], (code[1, :32] - z[1, 0]) * scale[1, 0])


def test_e4m3_rounding_matches_the_format():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()
    every = np.unique(every[np.isfinite(every)])
    assert every[-1] == 448 and np.array_equal(oracle.e4m3_round(every), every)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.uniform(-448, 448, 500), rng.standard_normal(500) * 0.02])
    near = every[np.abs(every[None] - x[:, None]).argmin(1)]
    assert np.array_equal(oracle.e4m3_round(x), near)
    mid = (every[:-1] + every[1:]) / 2
    t = torch.from_numpy(mid.astype(np.float32)).to(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(oracle.e4m3_round(mid), t)  # ties to even


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_oracle_is_a_rotation(interleaved):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 2, 10))
    f = np.array([1.0, 0.3, 0.01], dtype=np.float32)
    pos = np.array([[0, 5, -7], [1, 2, 3]])
    axis = [0, 1, 0]
    y = oracle.rope(x, pos, f, axis, interleaved)
    assert np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose(oracle.rope(y, pos, f, axis, interleaved, inverse=True), x)
    lo, hi = (2, 3) if interleaved else (1, 4)
    z = (x[2, 1, lo] + 1j * x[2, 1, hi]) * np.exp(1j * 3 * float(f[1]))
    assert np.allclose([y[2, 1, lo], y[2, 1, hi]], [z.real, z.imag])


# ---------------------------------------------------------------------------
# the kernels' steps, restated
# ---------------------------------------------------------------------------
def turns_per_position(f):
    """The kernel's steps: the 24-bit significand times 64 bits of 1 / 2 pi, shifted, modulo 2^64."""
    u = int(np.float32(f).view(np.uint32))
    x = (u >> 23) & 255
    m = (u & 0x7fffff) | (0x800000 if x else 0)
    e = (x if x else 1) - 150 - 2
    lo, hi, mod = m * 0xa2f9836e4e441529 % 2 ** 64, m * 0xa2f9836e4e441529 >> 64, 2 ** 64
    if e >= 0:
        t = (lo << e) % mod if e < 64 else 0
    elif e > -64:
        t = (lo >> -e) | ((hi << (64 + e)) % mod)
    else:
        t = hi >> (-e - 64) if e > -128 else 0
    return (mod - t) % mod if u >> 31 else t


def test_fixed_point_turns_hold_for_every_position():
    """position * frac(f / 2 pi) modulo one turn in 64-bit fixed point, against exact arithmetic: the fraction is off by
    one unit of 2^-64 for its shift and f * 2^-64 for the bits of 1 / 2 pi, so 2^31 positions are off by 2^-24 turns at
    most up to f = 256."""
    rng = np.random.default_rng(3)
    inv2pi = Fraction("0.159154943091895335768883763372514362034459645740456448747667344058896797634226535")
    for f in [1.0, 0.5, 1e-4, 0.731, 6.0, 2e-7, 1e-12, 1e-40, -0.25, 255.0, 6.2831855] + list(rng.uniform(0, 1, 20)):
        f = float(np.float32(f))
        F = turns_per_position(f)
        for p in [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1048575] + list(rng.integers(-2 ** 31, 2 ** 31, 20)):
            got = Fraction((int(p) * F) % 2 ** 64, 2 ** 64)
            want = (int(p) * Fraction(f) * inv2pi) % 1
            off = abs(got - want)
            assert min(off, 1 - off) <= Fraction(1, 2 ** 24), (f, p)


def find_slot(i, n_seqs, cu):
    """The kernel's search, lane by lane: the number of entries of cu[1:] that are <= i, and the begin offset of that
    sequence as the kernel gets it. Every index it reads is checked."""
    lo, n, rounds = 0, n_seqs, 0
    while n > 128:
        step = (n + 31) // 32
        c = 0
        for lane in range(32):
            at = min(lo + (lane + 1) * step, lo + n)
            assert 0 <= at <= n_seqs
            le = cu[at] <= i
            c += bool(le and lo + (lane + 1) * step <= lo + n + step - 1)
        done = min(c * step, n)
        lo += done
        n = 0 if done == n else min(step - 1, n - done)
        rounds += 1
        assert rounds < 8
    c, begin = 0, {}
    for j in range(4):
        if j and 32 * j >= n:
            continue
        for lane in range(32):
            mine = min(lo + 32 * j + lane, n_seqs - 1)
            assert 0 <= mine < n_seqs
            begin[j, lane] = cu[mine]
            c += bool(32 * j + lane < n and cu[mine + 1] <= i)
    b = lo + c
    if b >= n_seqs:
        return b, None
    if c < 32 * ((max(n, 1) + 31) // 32):
        j = max([0] + [j for j in (1, 2, 3) if c >= 32 * j and 32 * j < n])
        return b, begin[j, c & 31]
    return b, cu[b]


@pytest.mark.parametrize("n_seqs", [1, 2, 31, 32, 33, 64, 100, 127, 128, 129, 200, 1024, 1025, 5000])
def test_sequence_search(n_seqs):
    rng = np.random.default_rng(n_seqs)
    for kind in range(3):
        n = rng.integers(0, 4, n_seqs) if kind else np.ones(n_seqs, dtype=int)
        cu = np.concatenate([[rng.integers(0, 3) if kind == 2 else 0], n]).cumsum()
        for i in rng.integers(0, cu[-1] + 3, 12):
            want = int(np.searchsorted(cu[1:], i, side="right"))
            b, first = find_slot(i, n_seqs, cu)
            assert b == want and (b == n_seqs or first == cu[b])
    # offsets out of order: some index in range, and an end
    junk = rng.integers(-5, 50, n_seqs + 1)
    for i in (0, 10, 60):
        assert 0 <= find_slot(i, n_seqs, junk)[0] <= n_seqs


def test_codes_next_to_a_border():
    """The kernel's fp32 steps against the exact quotient, on rows whose values lie on and next to borders: the two
    roundings from either side, and the exact step where they differ."""
    f32 = np.float32

    def fma(a, b, c):  # one rounding; exact in Fraction
        return f32(float(Fraction(float(a)) * Fraction(float(b)) + Fraction(float(c))))

    def nearest_even(fr):
        lo = fr.numerator // fr.denominator
        d = fr - lo
        return lo + 1 if d > Fraction(1, 2) or (d == Fraction(1, 2) and lo % 2) else lo

    rng = np.random.default_rng(9)
    shift = f32(12582912.0)
    exact = 0
    for _ in range(300):
        amax = f32(round16("bf16")(abs(rng.standard_normal()) + 0.01))
        s = f32(amax * f32(f32(1.0) / f32(127.0)))
        inv = f32(f32(1.0) / s)
        up, dn = f32(inv * f32(1 + 2.0 ** -21)), f32(inv * f32(1 - 2.0 ** -21))
        for c in rng.integers(-127, 127, 6):
            for x in {float(round16("bf16")((c + 0.5) * float(s))), float(amax) / 2, float(amax), float(c) * 0.01}:
                x = f32(x if abs(x) <= amax else amax)
                r, q = fma(x, up, shift) - shift, fma(x, dn, shift) - shift
                if r != q:
                    exact += 1
                    d = fma(-(r + q), f32(0.5) * s, x)
                    takes_up = int(r) % 2 == 0 if d == 0 else (d > 0) == (x > 0)
                    r = r if takes_up else q
                assert int(r) == nearest_even(Fraction(float(x)) / Fraction(float(s)))
    assert exact > 20


# ---------------------------------------------------------------------------
# what a graph keeps
# ---------------------------------------------------------------------------
class FakeLibrary:
    """Every call succeeds; a capture ends with a graph handle."""
    calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            if name == "fl_capture_end":
                args[1]._obj.value = 1
            return 64 if name.endswith("workspace_size") else 0
        return call


class FakeOperators:
    """Stands in for the extension module: makes what is not given, and a workspace."""

    @staticmethod
    def _new():
        return torch.zeros(8)

    def w4_quantize(self, W, group, q, scales, stream):
        return q if q is not None else self._new(), scales if scales is not None else self._new()

    def w4_gemm(self, *a):
        return a[7] if a[7] is not None else self._new(), None if a[10] is not None else self._new()

    def w4_swiglu_ffn(self, *a):
        return a[6] if a[6] is not None else self._new(), None if a[8] is not None else self._new()

    def rope(self, q, k, pos, f, sections, inter, inverse, oq, ok, stream):
        return oq if oq is not None else self._new(), ok if ok is not None else self._new()


def test_graph_keeps_all_that_its_calls_made(monkeypatch):
    """Outputs and workspaces that calls under Graph.capture make for themselves live as long as the graph, the 16-bit
    functions' too, also those that only the next call saw; so do a layer and what was attached to it when it was issued.
    They are let go when the graph is closed, and calls outside a capture leave nothing behind."""
    import gc
    import weakref
    fake = FakeLibrary()
    monkeypatch.setattr(fl, "lib", lambda: fake)
    monkeypatch.setattr(fl, "_ops", FakeOperators())
    monkeypatch.setattr(fl, "_check_tensors", lambda *a, **k: None)
    monkeypatch.setattr(fl, "_stream", lambda s: 1)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    made = []

    def watched(f):
        def call(*a, **k):
            t = f(*a, **k)
            made.append(weakref.ref(t))
            return t
        return call
    x, W = torch.zeros((4, 8), dtype=torch.float16), torch.zeros((8, 8), dtype=torch.float16)
    layer = fl.DecoderLayer(x=x, Wg=W, Wk=W)
    attached = torch.zeros(3)
    layer.attached = (attached,)
    owned = [weakref.ref(attached), weakref.ref(layer)]
    del attached
    monkeypatch.setattr(torch, "empty", watched(torch.empty))
    monkeypatch.setattr(torch, "empty_like", watched(torch.empty_like))
    monkeypatch.setattr(FakeOperators, "_new", staticmethod(watched(FakeOperators._new)))

    def calls():
        fl.w4_gemm(fl.w4_gemm(x, None, None), None, None, out=x)
        fl.w4_swiglu_ffn(x, None, None, None, None)
        fl.w4_quantize(W)
        fl.rope(x, x, None, None)
        fl.gemm_epilogue(x, W)
        fl.norm_gemm(x, None, W)
        fl.norm_gemm_multi(x, None, [W, W])
        fl.input_bias_gemm(x, None, W)
        fl.rms_norm(x, None)
        fl.swiglu_ffn(x, None, W, W, W)
        fl.swiglu_ffn_noalloc(x, None, W, W, W)
    calls()
    count = len(made)
    gc.collect()
    assert count == 18 and not any(r() is not None for r in made)
    del made[:]
    graph = fl.Graph.capture(lambda: (calls(), layer.issue(0)))
    layer.attached = ()
    del layer
    gc.collect()
    assert len(made) == count and all(r() is not None for r in made + owned)
    graph.close()
    gc.collect()
    assert not any(r() is not None for r in made + owned)
    assert fl._captures == []


# ---------------------------------------------------------------------------
# host code compiled by itself
# ---------------------------------------------------------------------------
RESIDENT = r"""
#include "fl_resident.h"
#include <cstdio>
#define CHECK(X) if (!(X)) { std::printf("line %d: %s\n", __LINE__, #X); return 1; }
int main() {
    static fl::Resident<4, 8> r;
    int asked = 0, n = -1;
    auto says = [&](int value, int error) { return [&asked, value, error](int* out) { ++asked; *out = value; return error; }; };
    // one device's answer is not another's
    CHECK(r.get(0, 1, says(152, 0), &n) == 0 && n == 152 && asked == 1);
    CHECK(r.get(1, 1, says(132, 0), &n) == 0 && n == 132 && asked == 2);
    CHECK(r.get(0, 1, says(7, 0), &n) == 0 && n == 152 && asked == 2);
    CHECK(r.get(1, 1, says(7, 0), &n) == 0 && n == 132 && asked == 2);
    CHECK(r.get(3, 8, says(17, 0), &n) == 0 && n == 17 && asked == 3);
    // a failed query is handed on, and asked again
    CHECK(r.get(2, 4, says(9, 46), &n) == 46 && n == 0 && asked == 4);
    CHECK(r.get(2, 4, says(9, 2), &n) == 2 && n == 0 && asked == 5);
    CHECK(r.get(2, 4, says(30, 0), &n) == 0 && n == 30 && asked == 6);
    CHECK(r.get(2, 4, says(1, 2), &n) == 0 && n == 30 && asked == 6);
    // none resident is an answer
    CHECK(r.get(0, 8, says(0, 0), &n) == 0 && n == 0 && asked == 7);
    CHECK(r.get(0, 8, says(5, 0), &n) == 0 && n == 0 && asked == 7);
    return 0;
}
"""


def test_resident_counts_are_kept_by_device_and_only_when_known(tmp_path):
    import subprocess
    src = tmp_path / "resident.cpp"
    src.write_text(RESIDENT)
    exe = str(tmp_path / "resident")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", _build.CSRC, str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@no_gpu
def test_rope_takes_one_row_of_positions_for_every_axis(L):
    def call(**kw):
        return L.fl_rope(ctypes.byref(rope_desc(n_axes=3, axis_of=bytes([0, 1, 2, 0] * 8), **kw)), None)
    assert call(positions_stride=0) in PASSES                                  # expanded: a stride of 0
    assert call(positions_stride=10) in PASSES and call(positions_stride=11) in PASSES
    assert call(positions_stride=1) == INVALID and call(positions_stride=9) == INVALID and call(positions_stride=-10) == INVALID


# ---------------------------------------------------------------------------
# the build
# ---------------------------------------------------------------------------
@pytest.fixture
def toy_build(monkeypatch, tmp_path):
    """_build on a folder of its own, with compilers that note what they are asked for and leave a file."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "one.cu").write_text("")
    (tmp_path / "fl_torch.cpp").write_text("")
    out = tmp_path / "_build"
    for name, value in (("PKG", str(tmp_path)), ("CSRC", str(csrc)), ("BUILD", str(out)), ("INCLUDE", str(csrc)),
                        ("LIB", str(tmp_path / "libfusedlin.so")), ("BINDING", str(tmp_path / "_torch_binding.so")),
                        ("BINDING_SRC", str(tmp_path / "fl_torch.cpp")), ("STAMP", str(out / "fl_torch.stamp"))):
        monkeypatch.setattr(_build, name, value, raising=False)
    asked = []

    def run(cmd, **kw):
        made = cmd[cmd.index("-o") + 1]
        asked.append(made.replace(str(tmp_path), "").removesuffix(".tmp"))
        with open(made, "w") as f:
            f.write("x")

        class Result:
            returncode, stdout, stderr = 0, "", ""
        return Result
    monkeypatch.setattr(_build.subprocess, "run", run)

    def build():
        del asked[:]
        _build.build()
        return sorted(asked)
    return build


EVERYTHING = ["/_build/fl_torch.o", "/_build/one.o", "/_torch_binding.so", "/libfusedlin.so"]


def test_binding_is_rebuilt_when_torch_changes(toy_build, monkeypatch):
    assert toy_build() == EVERYTHING
    assert toy_build() == []
    monkeypatch.setattr(_build, "_torch", lambda: "another torch", raising=False)
    assert toy_build() == ["/_build/fl_torch.o", "/_torch_binding.so", "/libfusedlin.so"]
    assert toy_build() == []


def test_library_is_built_without_torch(toy_build, monkeypatch):
    import builtins
    import importlib.util
    find, imports = importlib.util.find_spec, builtins.__import__

    def no_torch(name, *a, **k):
        if name == "torch" or name.startswith("torch."):
            raise ImportError("no torch here")
        return imports(name, *a, **k)
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(builtins, "__import__", no_torch)
    assert toy_build() == ["/_build/one.o", "/libfusedlin.so"]
    assert toy_build() == []
    monkeypatch.undo()


# ---------------------------------------------------------------------------
# sizes whose products pass 32 bits
# ---------------------------------------------------------------------------
def test_rows_of_any_length_are_measured_in_64_bits(L):
    """Rows far too long for the decode kernel's shared memory go to the tile kernel, which wants its row scales, also
    where the bytes they would take are a small number modulo 2^32."""
    for M in (1, 2, 3, 8, 16, 24):
        for K in (1 << 26, 1 << 27, 1 << 28, 1 << 29, 1 << 30, (1 << 28) + 128, 0x7fff0000):
            assert fl.w4_gemm_workspace_size(M, K, True) >= 4 * M, (M, K)
            assert fl.w4_swiglu_ffn_workspace_size(M, K, 64) >= 2 * 64 * M + 4 * M, (M, K)


@no_gpu
def test_rows_next_to_2_31_are_refused(L):
    """Steps of 64 k and loads of 2048 run past a row's end before they are cut off: no sum of those may pass 2^31."""
    def gemm(K):
        return L.fl_w4_gemm(addr(0), addr(1), ctypes.byref(weight(group=32)), None, None, addr(4), 30, 8, K, 1e-6, 0, addr(5),
                            1 << 30, 0, None)

    def ffn(D, F):
        w = [weight(i, group=32) for i in (20, 22, 24)]
        return L.fl_w4_swiglu_ffn(addr(0), addr(1), *(ctypes.byref(v) for v in w), None, addr(4), 1, D, F, 1e-6, addr(6),
                                  1 << 35, 0, None)
    assert gemm(0x7fffffe0) == UNSUPPORTED and "too long" in fl.last_error()
    assert gemm(0x7ffff020) == UNSUPPORTED and "too long" in fl.last_error()
    assert gemm(0x7fff0000) in PASSES and "too long" not in fl.last_error()
    assert ffn(0x7fffffe0, 32) == UNSUPPORTED and "too" in fl.last_error()
    assert ffn(32, 0x7fffffe0) == UNSUPPORTED and "too" in fl.last_error()


def test_attach_cache_names_what_is_missing(monkeypatch):
    """Parts of a description that are left out or have other axes are a ValueError, before the library is called."""
    fake = FakeLibrary()
    monkeypatch.setattr(fl, "lib", lambda: fake)
    monkeypatch.setattr(fl, "_check_tensors", lambda *a, **k: None)
    x, W = torch.zeros((4, 64), dtype=torch.float16), torch.zeros((64, 64), dtype=torch.float16)
    layer = fl.DecoderLayer(x=x, Wg=W, Wk=W, q=x, k=x)
    f, pos, table, start = torch.ones(16), torch.zeros(4, dtype=torch.int32), torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    kc, ks = torch.zeros((8, 16, 2, 32), dtype=torch.int8), torch.zeros((8, 16, 2))
    full = dict(k_cache=kc, v_cache=kc, k_scale=ks, v_scale=ks, page_table=table, start=start)
    del fake.calls[:]
    layer.attach_cache(32, positions=pos, inv_freq=f, **full)
    assert fake.calls == ["fl_layer_attach_cache"]
    for bad in (dict(inv_freq=f), dict(inv_freq=f, positions=pos[0]), dict(inv_freq=f[None], positions=pos),
                *({**full, n: None} for n in ("v_cache", "k_scale", "v_scale", "page_table", "start")),
                {**full, "k_cache": kc[0]}, {**full, "page_table": table[0]}):
        with pytest.raises(ValueError):
            layer.attach_cache(32, **bad)
    assert fake.calls == ["fl_layer_attach_cache"]
