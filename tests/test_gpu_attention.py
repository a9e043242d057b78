"""Attention over prompts and over the paged cache, and the cache's page keeping, on the GPU against the float64 oracle
(needs an sm_103a GPU).

Bounds. u is the largest relative error of one rounding to the dtype (2^-8 bf16, 2^-11 fp16), w a row's normalised
weights, A = sum w |v|, size the largest sum |q| |k| scale / ln 2 of the row's scores.
  A score, in units of a factor of two, is off by 2^-20 size (fp32 sums of the products, the product with the scale and
  the difference to the maximum), so a weight is off by that times ln 2, and the sum that divides by as much: 2^-19 size
  together; the exponential and the fp32 sums add 2^-20.
  attention: the weights are rounded once to the dtype, below 2^-14 in fp16 by 2^-25 (they are 1 at least where the running
  maximum was set, so that their sum is 1 at least): |err| <= u |y| + (u + 2^-20 + 2^-19 size) A + n 2^-25 max |v|.
  kv_attend: weights times the value's scale are rounded to 11 bits in both types, or by 2^-25 of the largest one; the
  logarithm of the scale, of 2^-19 at most for scales between 2^-30 and 2^10, is one more term:
  |err| <= u |y| + (2^-11 + 2^-18 + 2^-19 size) A + n 2^-25 top max(w vs).
  The roundings are independent: the mean square is u^2 y^2 + u_w^2 sum (w v)^2 at most, of which a uniformly spread rounding
  reaches a third; the root of the mean over the tensor is tested with the bound itself, plus the fp32 terms.
Codes moved and counts of pages are equal.
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
FMT = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}


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


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().float().cpu().double().numpy()


def sums(n):
    return [0] + [int(x) for x in np.cumsum(n)]


def check(got, ref, u, uw, extra, floor, what=""):
    """extra: relative fp32 terms; floor: absolute, per row and head."""
    g, y = f64(got) if isinstance(got, torch.Tensor) else got, ref["out"]
    assert np.isfinite(g).all(), what
    err = np.abs(g - y)
    fp = extra + 2.0 ** -19 * ref["size"][..., None]
    bound = u * np.abs(y) + (uw + fp) * ref["mag"] + floor[..., None] + 2.0 ** -25 * (u == U["f16"])
    assert (err <= bound).all(), f"{what}: {np.nanmax(err / np.maximum(bound, 1e-300))} times the bound"
    rms = np.sqrt((err ** 2).mean())
    most = np.sqrt((u * u * y ** 2 + uw * uw * ref["sq"]).mean()) + (fp * ref["mag"] + floor[..., None]).mean() + 2.0 ** -25
    assert rms <= most, f"{what}: rms {rms} above {most}"


# ---------------------------------------------------------------------------
# attention over 16-bit keys and values
# ---------------------------------------------------------------------------
def attention_case(dt, hq, hkv, D, lq, lk, is_causal, seed, out=None, scale=None):
    rng = gen(40, seed)
    T, S = sum(lq), sum(lk)
    q, k, v = (put(rng.standard_normal((n, h, D)), dt) for n, h in ((T, hq), (S, hkv), (S, hkv)))
    cu_q, cu_k = sums(lq), sums(lk)
    got = fl.attention(q, k, v, cu_q=ints(cu_q), cu_k=ints(cu_k), causal=is_causal, out=out, scale=scale)
    fl.device_status()
    ref = oracle.attention(f64(q), f64(k), f64(v), cu_q, cu_k, is_causal, scale or D ** -0.5)
    floor = np.zeros((T, hq)) if dt == "bf16" else np.full((T, hq), max(lk + [0]) * 2.0 ** -25 * (float(v.abs().max()) if S else 0))
    return got, ref, (q, k, v, cu_q, cu_k, floor)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,D,lq,lk", [
    (1, 1, 64, [1], [1]),
    (1, 1, 128, [1], [1]),
    (2, 1, 64, [37], [37]),
    (2, 2, 128, [128], [128]),
    (3, 1, 128, [129], [129]),
    (4, 2, 64, [256], [256]),
    (2, 1, 128, [257], [257]),
    (1, 1, 128, [600], [600]),
    (1, 1, 64, [1100], [1100]),
    (4, 1, 80, [5, 0, 131, 1, 260], [5, 0, 131, 1, 260]),
    (2, 2, 96, [64, 300], [700, 301]),
    (6, 2, 8, [33, 2], [40, 129]),
    (1, 1, 72, [200, 10, 0, 3], [90, 4, 7, 0]),
    (2, 1, 128, [1, 1, 1], [1, 128, 513]),
    (1, 1, 120, [140] * 35, [140] * 35),
])
@pytest.mark.parametrize("is_causal", [True, False])
def test_attention(dt, hq, hkv, D, lq, lk, is_causal):
    got, ref, (*_, floor) = attention_case(dt, hq, hkv, D, lq, lk, is_causal, sum(lq) + D)
    check(got, ref, U[dt], U[dt], 2.0 ** -20, floor, f"{lq} {lk}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,D,lq,lk", [
    (2, 1, 64, [1], [4096]),
    (1, 1, 128, [130], [2100]),
    (2, 2, 96, [300], [5000]),
    (3, 1, 128, [7, 0, 200], [3000, 9, 4100]),
    (4, 4, 64, [257, 1], [2000, 3]),
    (32, 8, 128, [9], [1030]),
])
@pytest.mark.parametrize("is_causal", [True, False])
def test_attention_few_rows_over_many_keys(dt, hq, hkv, D, lq, lk, is_causal):
    """The keys are split over clusters, of sequences that have many and of ones that have few."""
    got, ref, (*_, floor) = attention_case(dt, hq, hkv, D, lq, lk, is_causal, sum(lk) + D)
    check(got, ref, U[dt], U[dt], 2.0 ** -20, floor, f"{lq} {lk}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_split_keys_that_are_not_finite(D, bad):
    rng = gen(66, D)
    n, m = 200, 2500
    q, k, v = (put(rng.standard_normal((x, 1, D)), "bf16") for x in (n, m, m))
    clean = fl.attention(q, k, v)
    at = m - 90                                    # seen by rows 110 and up
    v[at, 0, 3] = bad
    got = fl.attention(q, k, v)
    fl.device_status()
    hit = got[110:, 0, 3]
    assert torch.equal(got[:110], clean[:110]) and torch.equal(got[..., 4:], clean[..., 4:])
    assert (torch.isnan(hit) if bad != bad else hit == bad).all()
    # rows without keys beside split ones
    got = fl.attention(q, k, v, cu_q=ints([0, 150, 200]), cu_k=ints([0, 2400, 2400]))
    assert (got[150:] == 0).all() and torch.isfinite(got[:150]).all()
    fl.device_status()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_large_scores(dt):
    """Scores of some hundreds in both directions, the largest of a row coming late: the running maximum moves often."""
    rng = gen(41)
    T, D = 700, 64
    q = rng.standard_normal((T, 2, D))
    k = rng.standard_normal((T, 1, D)) * np.linspace(0.2, 12, T)[:, None, None]
    q, k, v = put(q, dt), put(k, dt), put(rng.standard_normal((T, 1, D)), dt)
    got = fl.attention(q, k, v, causal=True, scale=1.0)
    fl.device_status()
    ref = oracle.attention(f64(q), f64(k), f64(v), [0, T], [0, T], True, 1.0)
    floor = np.full((T, 2), 0 if dt == "bf16" else T * 2.0 ** -25 * 5)
    check(got, ref, U[dt], U[dt], 2.0 ** -20, floor)


def test_attention_one_sequence_without_offsets():
    rng = gen(42)
    q, k, v = (put(rng.standard_normal((300, h, 128)), "bf16") for h in (4, 2, 2))
    cu = ints([0, 300])
    a = fl.attention(q, k, v)
    assert torch.equal(a, fl.attention(q, k, v, cu_q=cu)) and torch.equal(a, fl.attention(q, k, v, cu_q=cu, cu_k=cu))
    b = fl.attention(q[:100].contiguous(), k, v)      # the last 100 rows' positions
    assert torch.equal(b, fl.attention(q[:100].contiguous(), k, v, cu_q=ints([0, 100]), cu_k=cu))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_strided_and_rows_behind_the_last_sequence(dt):
    """q, k and v as column ranges of a stacked projection, out a column range of a wider matrix; rows in front of the first
    and behind the last sequence stay as they were."""
    rng = gen(43)
    T, hq, hkv, D = 420, 6, 2, 64
    qkv = put(rng.standard_normal((T, (hq + 2 * hkv) * D)), dt)
    q = qkv[:, :hq * D].unflatten(1, (hq, D))
    k, v = (qkv[:, (hq + i * hkv) * D:(hq + (i + 1) * hkv) * D].unflatten(1, (hkv, D)) for i in (0, 1))
    wide = torch.full((T, hq * D + 24), 7.0, dtype=DT[dt], device="cuda")
    out = wide[:, 8:8 + hq * D].unflatten(1, (hq, D))
    cu = [3, 3, 150, 411]
    got = fl.attention(q, k, v, cu_q=ints(cu), out=out)
    fl.device_status()
    assert got is out
    w = f64(wide)
    assert (w[:, :8] == 7).all() and (w[:, 8 + hq * D:] == 7).all() and (w[:3] == 7).all() and (w[411:] == 7).all()
    ref = oracle.attention(f64(q), f64(k), f64(v), cu, cu, True, D ** -0.5)
    ref = {n: x[3:411] for n, x in ref.items()}
    floor = np.full((408, hq), 0 if dt == "bf16" else 261 * 2.0 ** -25 * 5)
    check(out[3:411], ref, U[dt], U[dt], 2.0 ** -20, floor)
    # heads in front of rows: [heads, rows, D] in memory
    qh, kh, vh = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    oh = torch.full((hq, T, D), 7.0, dtype=DT[dt], device="cuda").transpose(0, 1)
    fl.attention(qh, kh, vh, cu_q=ints(cu), out=oh)
    assert torch.equal(oh, out.contiguous())


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_rows_without_keys(dt):
    got, ref, _ = attention_case(dt, 2, 1, 64, [200, 150, 20], [60, 0, 3], True, 44)
    g = f64(got)
    assert (g[:140] == 0).all() and (g[200:350] == 0).all() and (g[350:367] == 0).all()
    assert (g[140:200] != 0).any(-1).all() and (g[367:] != 0).any(-1).all()
    got, ref, _ = attention_case(dt, 2, 1, 128, [5, 3], [0, 4], False, 45)
    assert (f64(got)[:5] == 0).all() and (f64(got)[5:] != 0).any(-1).all()
    q = put(gen(46).standard_normal((9, 2, 64)), dt)
    none = torch.empty((0, 1, 64), dtype=DT[dt], device="cuda")
    assert (f64(fl.attention(q, none, none)) == 0).all()
    assert fl.attention(q[:0], none, none).shape == (0, 2, 64)
    fl.device_status()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_what_is_not_seen_does_not_reach_a_row(dt, D, bad):
    """Values and keys that are not finite, in another sequence, behind the last key and in front of a causal row's border."""
    rng = gen(47, D)
    lq = lk = [130, 300]
    cu = sums(lq)
    q, k, v = (put(rng.standard_normal((cu[-1] + 40, h, D)), dt) for h in (2, 1, 1))
    at = 130 + 211
    v[cu[-1]:], k[cu[-1]:], q[cu[-1]:] = bad, bad, bad
    out = torch.zeros_like(q)
    clean = fl.attention(q, k, v, cu_q=ints(cu), out=out.clone())
    assert torch.isfinite(clean[:cu[-1]]).all()
    v[at, 0, 5] = bad
    got = fl.attention(q, k, v, cu_q=ints(cu), out=out.clone())
    fl.device_status()
    same = got == clean
    assert same[:at].all() and same[..., :5].all() and same[..., 6:].all()
    hit = got[at:cu[-1], :, 5]
    assert (torch.isnan(hit) if bad != bad else hit == bad).all()
    v[at + 3, 0, 5] = -bad                          # inf and -inf: a NaN from there on
    got = fl.attention(q, k, v, cu_q=ints(cu), out=out.clone())
    assert torch.isnan(got[at + 3:cu[-1], :, 5]).all() and (got[:at] == clean[:at]).all()
    # a key that is not finite makes NaN of the rows that see it, and of no others
    v[at, 0, 5] = v[at + 3, 0, 5] = 0
    clean = fl.attention(q, k, v, cu_q=ints(cu), out=out.clone())
    k[at, 0, 7] = float("nan")
    got = fl.attention(q, k, v, cu_q=ints(cu), out=out.clone())
    assert torch.isnan(got[at:cu[-1]]).all() and torch.equal(got[:at], clean[:at])
    # so does a row of q, of itself alone
    k[at, 0, 7] = 0
    clean = fl.attention(q, k, v, cu_q=ints(cu), out=out.clone())
    q[200, 1, 3] = bad
    got = fl.attention(q, k, v, cu_q=ints(cu), out=out.clone())
    rest = torch.ones(cu[-1], 2, dtype=torch.bool, device="cuda")
    rest[200, 1] = False
    assert torch.isnan(got[200, 1]).all() and torch.equal(got[:cu[-1]][rest], clean[:cu[-1]][rest])
    fl.device_status()


def test_attention_offsets_out_of_range_stay_inside():
    """Offsets past the row counts, negative or falling, are taken as the nearest that is possible."""
    q = put(gen(48).standard_normal((50, 1, 64)), "f16")
    out = torch.full_like(q, 7.0)
    fl.attention(q, q, q, cu_q=ints([-5, 20, 10, 900]), out=out)
    fl.device_status()
    want = torch.full_like(q, 7.0)
    fl.attention(q, q, q, cu_q=ints([0, 20, 20, 20]), out=want)
    fl.attention(q, q, q, cu_q=ints([10, 50, 50, 50]), out=want)
    assert torch.equal(out[20:], want[20:])
    fl.device_status()


def test_attention_streams_graphs_and_repeated_calls():
    rng = gen(49)
    cu = ints([0, 70, 333])
    q, k, v = (put(rng.standard_normal((333, h, 128)), "bf16") for h in (8, 2, 2))
    want = fl.attention(q, k, v, cu_q=cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a = fl.attention(q, k, v, cu_q=cu)
    b = fl.attention(q, k, v, cu_q=cu, stream=s)
    s.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    out = torch.zeros_like(q)
    with torch.cuda.stream(s):
        graph = fl.Graph.capture(lambda: fl.attention(q, k, v, cu_q=cu, out=out))
        q.copy_(q.flip(0))
        graph.launch()
        again = fl.attention(q, k, v, cu_q=cu)
        cu.copy_(ints([0, 200, 300]))
        out2 = out.clone()
        graph.launch()
    s.synchronize()
    assert torch.equal(out2, again) and not torch.equal(out2, want)
    assert torch.equal(out[:300], fl.attention(q, k, v, cu_q=cu)[:300]) and torch.equal(out[300:], out2[300:])
    fl.device_status()


# ---------------------------------------------------------------------------
# attention over the cache
# ---------------------------------------------------------------------------
class Paged:
    """A cache with random codes, pages in random order, for sequences of `lens` positions."""

    def __init__(self, rng, lens, H, D, page, fmt, spare=3, scales=(0.004, 0.03)):
        need = [-(-n // page) for n in lens]
        self.page, self.H, self.D, self.fmt = page, H, D, fmt
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), max(need + [1]) + 1), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        code, top = FMT[fmt]
        shape = (self.pages, page, H, D)
        c = np.clip(rng.standard_normal((2, *shape)) * top / 4, -top, top)
        c = np.rint(c) if fmt == "int8" else oracle.e4m3_round(c)
        s = np.exp(rng.uniform(np.log(scales[0]), np.log(scales[1]), (2, *shape[:3]))).astype(np.float32)
        if fmt == "e4m3":
            s = s / np.float32(4)
        self.code, self.scale = c, s
        self.k, self.v = (torch.from_numpy(x).to(torch.float32).to(code).cuda() for x in c)
        self.ks, self.vs = (put(x) for x in s)

    def tensors(self):
        return self.k, self.v, self.ks, self.vs

    def values(self):
        """Of each sequence: k, v, which positions have a page."""
        out = []
        for row in self.table:
            there = np.repeat((row >= 0) & (row < self.pages), self.page)
            at = np.clip(row, 0, self.pages - 1)
            kv = [(self.code[w][at] * self.scale[w][at].astype(np.float64)[..., None]).reshape(-1, self.H, self.D) for w in (0, 1)]
            out.append((*kv, there))
        return out


def attend_case(rng, dt, cache, hq, n_rows, start, tree=None, cu=None, q=None, out=None, scale=None, pad=0):
    rows = sum(n_rows)
    q = put(rng.standard_normal((rows + pad, hq, cache.D)), dt) if q is None else q
    cu_rows = sums(n_rows)
    got = fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints(start), cu_rows=ints(cu_rows) if cu is None else cu,
                       tree=None if tree is None else put(tree), out=out, scale=scale)
    vals = cache.values()
    ref = oracle.kv_attend(f64(q)[:rows], [x[0] for x in vals], [x[1] for x in vals], [x[2] for x in vals], cu_rows, start,
                           tree, scale or cache.D ** -0.5)
    return got, ref, q


def attend_check(got, ref, dt, cache, n_rows, start, what=""):
    n = max(a + b for a, b in zip(n_rows, start))
    top = FMT[cache.fmt][1]
    floor = n * 2.0 ** -25 * top * cache.scale[1].max() * ref["top"]
    check(got, ref, U[dt], 2.0 ** -11, 2.0 ** -18, floor, what)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("H,group,D,page,n_rows,start", [
    (1, 1, 64, 16, [1], [0]),
    (1, 1, 128, 16, [1], [1]),
    (2, 4, 128, 16, [1, 1, 1], [0, 15, 16]),
    (1, 3, 80, 7, [1, 1, 0, 1], [127, 128, 9, 300]),
    (2, 1, 8, 64, [1, 2], [40, 0]),
    (1, 4, 256, 32, [1, 3], [260, 77]),
    (1, 16, 128, 16, [1, 2], [513, 100]),
    (2, 4, 128, 16, [7, 1, 0, 12], [100, 700, 5, 0]),
    (1, 4, 96, 16, [40], [333]),
    (1, 2, 200, 16, [20], [129]),
    (1, 1, 24, 16, [70, 1], [3, 90]),
    (3, 1, 128, 64, [1], [4000]),
    (1, 8, 64, 16, [9], [2100]),
    (1, 20, 128, 16, [3], [1000]),
    (2, 2, 64, 7, [1, 3], [200, 61]),
    (1, 4, 48, 1, [2], [40]),
    (2, 4, 64, 6, [5], [600]),
    (1, 2, 256, 3, [2], [100]),
])
def test_kv_attend(dt, fmt, H, group, D, page, n_rows, start):
    rng = gen(50, H, group, D, page, sum(start))
    cache = Paged(rng, [a + b for a, b in zip(n_rows, start)], H, D, page, fmt)
    for kind in ("causal", "tree"):
        tree = None
        if kind == "tree":
            tree = rng.random((sum(n_rows), max(n_rows) + 1)) < 0.5
        got, ref, _ = attend_case(rng, dt, cache, H * group, n_rows, start, tree)
        fl.device_status()
        attend_check(got, ref, dt, cache, n_rows, start, kind)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("H,group,D,page,n_rows,start", [
    (1, 4, 128, 16, [48], [0]),
    (1, 4, 128, 16, [48, 33], [100, 5]),
    (2, 4, 64, 16, [64, 64], [700, 129]),
    (1, 1, 96, 7, [129, 40], [300, 3]),
    (2, 2, 128, 48, [70, 0, 9, 130], [5000, 3, 1, 0]),
    (1, 3, 80, 64, [100], [2000]),
    (1, 1, 16, 16, [300], [64]),
    (8, 4, 128, 16, [40, 40], [300, 2000]),
    (1, 4, 64, 9, [50], [1500]),
    (1, 4, 64, 6, [50], [1500]),
    (1, 4, 128, 1, [40], [1100]),
])
def test_kv_attend_many_rows(dt, fmt, H, group, D, page, n_rows, start):
    rng = gen(67, H, group, D, page, sum(start))
    cache = Paged(rng, [a + b for a, b in zip(n_rows, start)], H, D, page, fmt)
    for kind in ("causal", "tree"):
        tree = None
        if kind == "tree":
            tree = rng.random((sum(n_rows), max(n_rows) - 1)) < 0.3
        got, ref, q = attend_case(rng, dt, cache, H * group, n_rows, start, tree)
        fl.device_status()
        attend_check(got, ref, dt, cache, n_rows, start, kind)
        again = fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints(start), cu_rows=ints(sums(n_rows)),
                             tree=None if tree is None else put(tree))
        assert torch.equal(again, got)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_kv_attend_many_rows_what_is_not_seen(fmt, D):
    """Junk in unused places, drafts that hold no number, rows that see nothing, positions without a page, rows behind
    the last sequence, one row of q that is not finite: each stays where it belongs."""
    rng = gen(68, D)
    n_rows, start = [40, 50], [137, 0]
    cache = Paged(rng, [177, 50], 1, D, 16, fmt)
    tree = rng.random((95, 50)) < 0.4
    tree[:, 7] = False
    tree[3, 7] = tree[60, 7] = True
    tree[45] = False                                # sees nothing: its context is empty
    q = put(rng.standard_normal((95, 4, D)), "f16")
    out = torch.full_like(q, 7.0)
    clean, ref, _ = attend_case(rng, "f16", cache, 4, n_rows, start, tree, q=q, out=out)
    clean = clean.clone()
    assert (clean[90:] == 7).all() and (clean[45] == 0).all() and torch.isfinite(clean[:90]).all()
    attend_check(clean[:90], ref, "f16", cache, n_rows, start)
    used = np.zeros((cache.pages, 16), dtype=bool)
    for b, n in ((0, 177), (1, 50)):
        for p in range(n):
            used[cache.table[b, p // 16], p % 16] = True
    junk = torch.from_numpy(~used).cuda()
    for t in (cache.ks, cache.vs):
        t[junk] = float("nan")
    for t in (cache.k, cache.v):
        t.view(torch.uint8)[junk] = 0x7f            # a NaN in e4m3
    args = (ints(cache.table), ints(start))
    got = fl.kv_attend(q, *cache.tensors(), *args, cu_rows=ints(sums(n_rows)), tree=put(tree), out=out)
    fl.device_status()
    assert torch.equal(got, clean)
    # draft 7 of each sequence holds no number: rows 3 and 60 see it, no others
    for b, pos in ((0, 144), (1, 7)):
        page, at = int(cache.table[b, pos // 16]), pos % 16
        for t in (cache.k, cache.v):
            t.view(torch.uint8)[page, at] = 0
        for t in (cache.ks, cache.vs):
            t[page, at] = float("nan")
    got = fl.kv_attend(q, *cache.tensors(), *args, cu_rows=ints(sums(n_rows)), tree=put(tree), out=out)
    rest = torch.ones(95, dtype=torch.bool, device="cuda")
    rest[3] = rest[60] = False
    assert torch.isnan(got[3]).all() and torch.isnan(got[60]).all() and torch.equal(got[rest], clean[rest])
    q[20, 2, 1] = float("inf")
    got = fl.kv_attend(q, *cache.tensors(), *args, cu_rows=ints(sums(n_rows)), tree=put(tree), out=out)
    assert torch.isnan(got[20, 2]).any() and torch.equal(got[20, 1], clean[20, 1])
    rest[20] = False
    assert torch.equal(got[rest], clean[rest])
    fl.device_status()
    # a page that is not there
    cache = Paged(rng, [177, 50], 1, D, 16, fmt)
    cache.table[0, 4] = -1
    got, ref, _ = attend_case(rng, "bf16", cache, 4, n_rows, start)
    with pytest.raises(fl.FusedLinError):
        fl.device_status()
    attend_check(got, ref, "bf16", cache, n_rows, start)


def test_kv_attend_many_rows_of_any_scale():
    """Rows of bf16 far outside fp16's range, values whose scales lie 2^18 apart, scores that grow towards the end."""
    rng = gen(69)
    n_rows, start = [60], [900]
    cache = Paged(rng, [960], 1, 128, 16, "int8")
    cache.scale[1] = np.where(rng.random(cache.scale[1].shape) < 0.5, 2.0 ** -6, 2.0 ** -24).astype(np.float32)
    order = np.empty(cache.pages * 16)
    for p in range(60 * 16):
        order[cache.table[0, p // 16] * 16 + p % 16] = 0.001 * 1.005 ** p
    cache.scale[0] = order.reshape(cache.pages, 16, 1).astype(np.float32)
    cache.ks, cache.vs = put(cache.scale[0]), put(cache.scale[1])
    for size in (2.0 ** -50, 2.0 ** 40):
        q = put(rng.standard_normal((60, 1, 128)) * size * np.exp2(rng.integers(-6, 6, (60, 1, 1))), "bf16")
        got, ref, _ = attend_case(rng, "bf16", cache, 1, n_rows, start, q=q, scale=0.08 / size)
        fl.device_status()
        vals = cache.values()[0]
        floor = np.zeros((60, 1))
        for i in range(60):
            x = vals[0][:901 + i, 0] @ f64(q)[i, 0] * 0.08 / size
            w = np.exp(x - x.max())
            vs = cache.scale[1][cache.table[0][:60]].reshape(-1)[:len(w)]
            floor[i, 0] = len(w) * 2.0 ** -25 * 127 * (w / w.sum() * vs).max()
        check(got, ref, U["bf16"], 2.0 ** -11, 2.0 ** -18, floor, f"{size}")


def test_kv_attend_decode_without_offsets():
    rng = gen(51)
    start = [5, 1000, 0, 64]
    cache = Paged(rng, [n + 1 for n in start], 2, 128, 16, "int8")
    got, ref, q = attend_case(rng, "bf16", cache, 8, [1] * 4, start)
    alone = fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints(start))
    assert torch.equal(got, alone)
    # fewer and more rows than sequences: the first sequences' rows, and rows that belong to none
    out = torch.full((6, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q6 = torch.cat((q, q[:2]))
    fl.kv_attend(q6, *cache.tensors(), ints(cache.table), ints(start), out=out)
    assert torch.equal(out[:4], got) and (out[4:] == 7).all()
    two = fl.kv_attend(q[:2].contiguous(), *cache.tensors(), ints(cache.table), ints(start))
    assert torch.equal(two, got[:2])
    fl.device_status()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_kv_attend_split_contexts_of_uneven_lengths(dt, fmt):
    """Contexts long enough to be read by many CTAs beside short ones; the answer is the same in every run."""
    rng = gen(52)
    start, n_rows = [9000, 3, 517, 0, 2600], [5, 1, 9, 2, 33]
    cache = Paged(rng, [a + b for a, b in zip(n_rows, start)], 2, 64, 16, fmt)
    got, ref, q = attend_case(rng, dt, cache, 4, n_rows, start)
    fl.device_status()
    attend_check(got, ref, dt, cache, n_rows, start)
    for _ in range(3):
        again = fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints(start), cu_rows=ints(sums(n_rows)))
        assert torch.equal(again, got)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_kv_attend_values_of_very_different_scales(dt):
    """Rows of v whose scales lie 2^30 apart, and the largest score where the values are smallest: the weights that are rounded
    carry the scale, so the answer keeps its digits."""
    rng = gen(53)
    cache = Paged(rng, [600], 1, 64, 16, "int8")
    q = put(rng.standard_normal((2, 4, 64)), dt)
    big = rng.random(cache.scale[1].shape) < 0.5
    cache.scale[1] = np.where(big, 2.0 ** -6, 2.0 ** -24).astype(np.float32)
    cache.scale[0] = np.where(big, 2.0 ** -10, 2.0 ** -5).astype(np.float32)   # small values: large scores
    cache.ks, cache.vs = put(cache.scale[0]), put(cache.scale[1])
    got, ref, _ = attend_case(rng, dt, cache, 4, [2], [598], q=q, scale=0.25)
    fl.device_status()
    floor = np.zeros((2, 4))
    vals = cache.values()[0]
    for i in range(2):
        for h in range(4):
            x = vals[0][:598 + i + 1, 0] @ f64(q)[i, h] * 0.25
            w = np.exp(x - x.max())
            vs = cache.scale[1][cache.table[0]].reshape(-1)[:len(w)]
            floor[i, h] = len(w) * 2.0 ** -25 * 127 * (w / w.sum() * vs).max()
    check(got, ref, U[dt], 2.0 ** -11, 2.0 ** -18, floor)


def test_kv_attend_bf16_rows_of_any_size():
    """bf16 rows of q far outside fp16's range: each row is multiplied as fp16 times a power of two."""
    rng = gen(54)
    cache = Paged(rng, [200], 1, 128, 16, "int8")
    for size in (2.0 ** -60, 2.0 ** -20, 2.0 ** 20, 2.0 ** 60):
        q = put(rng.standard_normal((1, 2, 128)) * size, "bf16")
        got, ref, _ = attend_case(rng, "bf16", cache, 2, [1], [199], q=q, scale=1.0 / size / 11)
        attend_check(got, ref, "bf16", cache, [1], [199])
    fl.device_status()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_kv_attend_rows_that_see_nothing(dt):
    rng = gen(55)
    n_rows, start = [4, 3], [0, 0]
    cache = Paged(rng, [4, 3], 2, 64, 16, "e4m3")
    tree = np.ones((7, 4), dtype=bool)
    tree[1] = False
    tree[5] = False
    tree[0, 1:] = False
    got, ref, q = attend_case(rng, dt, cache, 4, n_rows, start, tree)
    g = f64(got)
    assert (g[1] == 0).all() and (g[5] == 0).all() and (g[0] != 0).any() and (g[4] != 0).any()
    attend_check(got, ref, dt, cache, n_rows, start)
    none = fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints(start), cu_rows=ints(sums(n_rows)),
                        tree=torch.zeros((7, 0), dtype=torch.bool, device="cuda"))
    assert (none == 0).all()
    fl.device_status()
    # new rows at negative positions are seen by nobody
    got = fl.kv_attend(q[:4].contiguous(), *cache.tensors(), ints(cache.table), ints([-2, -9]), cu_rows=ints([0, 4, 4]))
    g = f64(got)
    assert (g[:2] == 0).all() and (g[2:] != 0).any(-1).all()
    fl.device_status()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_kv_attend_what_is_not_seen_does_not_reach_a_row(fmt, D):
    """Codes and scales that are not finite in pages that no row may see, behind the last position, and in drafts that a row
    does not see."""
    rng = gen(56, D)
    n_rows, start = [3, 2], [37, 200]
    cache = Paged(rng, [40, 202], 1, D, 16, fmt)
    tree = np.array([[1, 0, 0], [0, 1, 0], [0, 1, 1], [1, 0, 0], [1, 1, 0]], dtype=bool)
    q = put(rng.standard_normal((5, 2, D)), "f16")
    clean, ref, _ = attend_case(rng, "f16", cache, 2, n_rows, start, tree, q=q)
    used = np.zeros((cache.pages, 16), dtype=bool)
    for b, n in ((0, 40), (1, 202)):
        for p in range(n):
            used[cache.table[b, p // 16], p % 16] = True
    junk = torch.from_numpy(~used).cuda()
    for t in (cache.ks, cache.vs):
        t[junk] = float("nan")
    for t in (cache.k, cache.v):
        t.view(torch.uint8)[junk] = 0x7f            # a NaN in e4m3
    got = fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints(start), cu_rows=ints(sums(n_rows)), tree=put(tree))
    assert torch.equal(got, clean)
    fl.device_status()
    # draft 1 of the first sequence holds no number: rows 1 and 2 see it, row 0 does not
    page, at = cache.table[0, 38 // 16], 38 % 16
    for t in (cache.k, cache.v):
        t.view(torch.uint8)[int(page), at] = 0
    for t in (cache.ks, cache.vs):
        keep = t[int(page), at].clone()
        t[int(page), at] = float("nan")
        got = fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints(start), cu_rows=ints(sums(n_rows)), tree=put(tree))
        assert torch.isnan(got[1:3]).all() and torch.equal(got[0], clean[0]) and torch.equal(got[3:], clean[3:])
        t[int(page), at] = keep
    q[3, 0, 1] = float("nan")
    cache.k.view(torch.uint8)[int(page), at] = torch.from_numpy(cache.code[0][int(page), at].astype(np.float32)).to(
        FMT[fmt][0]).view(torch.uint8).cuda()
    cache.v.view(torch.uint8)[int(page), at] = torch.from_numpy(cache.code[1][int(page), at].astype(np.float32)).to(
        FMT[fmt][0]).view(torch.uint8).cuda()
    got = fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints(start), cu_rows=ints(sums(n_rows)), tree=put(tree))
    assert torch.isnan(got[3, 0]).all() and torch.equal(got[3, 1], clean[3, 1]) and torch.equal(got[:3], clean[:3])
    fl.device_status()


def test_kv_attend_positions_without_a_page():
    rng = gen(57)
    n_rows, start = [2, 1, 1], [300, 40, 10]
    cache = Paged(rng, [302, 41, 11], 2, 64, 16, "int8")
    cache.table[0, 3] = cache.pages
    cache.table[0, 7] = -1
    cache.table[1, 0] = 1 << 30
    got, ref, _ = attend_case(rng, "f16", cache, 2, n_rows, start)
    with pytest.raises(fl.FusedLinError) as e:
        fl.device_status()
    assert e.value.status == 7
    fl.device_status()
    attend_check(got, ref, "f16", cache, n_rows, start)
    # past the table
    short = ints(cache.table[:, :2])
    q = put(rng.standard_normal((4, 2, 64)), "f16")
    fl.kv_attend(q, *cache.tensors(), short, ints(start), cu_rows=ints(sums(n_rows)))
    with pytest.raises(fl.FusedLinError):
        fl.device_status()
    fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints([2, 3, 4]), cu_rows=ints([0, 1, 1, 2]))
    with pytest.raises(fl.FusedLinError):   # sequence 1 has no rows, sequence 0 and 2 have their pages
        cache.table[2, 0] = -7
        fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints([2, 3, 4]), cu_rows=ints([0, 1, 1, 2]))
        fl.device_status()


def test_kv_attend_strided_tables_rows_and_outputs():
    rng = gen(58)
    n_rows, start = [3, 2], [50, 170]
    cache = Paged(rng, [53, 172], 2, 64, 16, "int8")
    got, ref, q = attend_case(rng, "bf16", cache, 6, n_rows, start)
    wide = put(rng.standard_normal((9, 6 * 64 + 64)), "bf16")
    wq = wide[1:6, 32:32 + 384].unflatten(1, (6, 64))
    wq.copy_(q)
    table = torch.full((2, cache.table.shape[1] + 5), 1 << 20, dtype=torch.int32, device="cuda")
    table[:, 2:2 + cache.table.shape[1]] = ints(cache.table)
    buf = torch.full((6, 7, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf.transpose(0, 1)[:5, :, 8:72]
    tree = torch.zeros((5, 9), dtype=torch.bool, device="cuda")
    for i, n in enumerate((1, 2, 3, 1, 2)):
        tree[i, 4:4 + n] = True
    r = fl.kv_attend(wq, *cache.tensors(), table[:, 2:2 + cache.table.shape[1]], ints(start), cu_rows=ints(sums(n_rows)),
                     tree=tree[:, 4:7], out=out)
    fl.device_status()
    assert r is out and torch.equal(out, got)
    assert (buf[..., :8] == 7).all() and (buf[..., 72:] == 7).all() and (buf[:, 5:] == 7).all()


def test_kv_attend_workspace_streams_and_graphs():
    """Two captured graphs with a workspace each, replayed side by side from other lengths than they were captured with."""
    rng = gen(59)
    start = [3000, 10]
    cache = Paged(rng, [3010, 2000], 2, 128, 16, "e4m3")
    table, st = ints(cache.table), ints(start)
    qs = [put(rng.standard_normal((2, 8, 128)), "bf16") for _ in range(2)]
    want = [fl.kv_attend(q, *cache.tensors(), table, st) for q in qs]
    need = fl.kv_attend_workspace_size(qs[0], cache.k, table)
    assert need > 0
    for fill in (0, 0xff):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(fl.kv_attend(qs[0], *cache.tensors(), table, st, workspace=ws), want[0])
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [torch.zeros_like(q) for q in qs]
    graphs = []
    torch.cuda.synchronize()
    for q, s, o in zip(qs, streams, outs):
        with torch.cuda.stream(s):
            graphs.append(fl.Graph.capture(lambda: fl.kv_attend(q, *cache.tensors(), table, st, out=o)))
    st.copy_(ints([700, 1999]))
    torch.cuda.synchronize()
    junk = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")  # memory the graphs would have lost
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.launch()
    torch.cuda.synchronize()
    for q, o, w in zip(qs, outs, want):
        assert torch.equal(o, fl.kv_attend(q, *cache.tensors(), table, st)) and not torch.equal(o, w)
    assert (junk == 0xff).all()
    fl.device_status()


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def random_tables(rng, B, per, pages, share=0.2):
    """Consistent tables and counts, some pages shared by several entries."""
    table = np.full((B, per), -1, dtype=np.int32)
    order = list(rng.permutation(pages))
    for b in range(B):
        n = int(rng.integers(0, per + 1))
        for j in range(n):
            if b and rng.random() < share and (table[:b] >= 0).any():
                other = table[:b][table[:b] >= 0]
                table[b, j] = other[rng.integers(len(other))]
            elif order:
                table[b, j] = order.pop()
    refs = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    return table, refs


@pytest.mark.parametrize("B,per,pages,page", [(1, 1, 1, 16), (1, 9, 30, 16), (3, 300, 700, 1), (7, 16, 130, 16), (61, 40, 900, 7),
                                              (256, 65, 9000, 64), (300, 3, 2000, 16), (2, 5000, 12000, 4), (40, 7, 60, 16),
                                              (20, 20, 2049, 16), (600, 9, 700, 16), (9, 600, 70000, 16), (3, 40, 600000, 16)])
def test_kv_resize(B, per, pages, page):
    rng = gen(60, B, per)
    table, refs = random_tables(rng, B, per, pages)
    t, r = ints(table), ints(refs)
    for k in range(4):
        lengths = rng.integers(-3, per * page + 1, B)
        if k == 1:
            lengths[:] = 0
        if k == 2:
            lengths[rng.random(B) < 0.5] = 0
        fl.kv_resize(t, r, ints(lengths), page)
        table, refs, fine = oracle.kv_resize(table, refs, lengths, page)
        if fine:
            fl.device_status()
        else:
            with pytest.raises(fl.FusedLinError):
                fl.device_status()
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs), k
    assert (refs == np.bincount(table[table >= 0], minlength=pages)).all()


def test_kv_resize_too_long_strided_and_foreign_entries():
    """Lengths past the table, entries that are no pages, a table inside a larger one, which keeps its other columns."""
    wide = torch.full((3, 10), 5, dtype=torch.int32, device="cuda")
    t = wide[:, 2:6]
    t.copy_(ints([[1, 99, -5, -1], [-1, -1, -1, -1], [3, 2, 20, -7]]))
    refs = ints([0, 1, 1, 1] + [0] * 16)
    table = t.cpu().numpy().copy()
    fl.kv_resize(t, refs, ints([49, 1000, 17]), 16)
    with pytest.raises(fl.FusedLinError):
        fl.device_status()
    want, want_refs, fine = oracle.kv_resize(table, np.array([0, 1, 1, 1] + [0] * 16), [49, 1000, 17], 16)
    assert not fine and np.array_equal(t.cpu().numpy(), want) and np.array_equal(refs.cpu().numpy(), want_refs)
    assert (wide[:, :2] == 5).all() and (wide[:, 6:] == 5).all()
    fl.device_status()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("H,D,page,lens,each,spare", [(1, 64, 16, [1], 1, 1), (2, 80, 7, [20, 21, 0], 3, 12), (3, 24, 16, [300, 45], 4, 9),
                                                      (8, 128, 64, [150, 64, 700], 7, 40), (2, 64, 16, [33, 50], 5, 4)])
def test_kv_fork(fmt, H, D, page, lens, each, spare):
    rng = gen(61, H, D, page)
    P = len(lens)
    cache = Paged(rng, lens + [0] * (P * each), H, D, page, fmt, spare=spare)
    refs = np.bincount(cache.table[cache.table >= 0], minlength=cache.pages).astype(np.int32)
    parents = np.repeat(np.arange(P), each)
    children = P + rng.permutation(P * each)
    lengths = np.repeat(lens, each)
    lengths[::2] = lengths[::2] * 2 // 3
    t, r = ints(cache.table), ints(refs)
    table = cache.table
    host = [x.view(torch.uint8).cpu().numpy().copy() for x in (cache.k, cache.v)] + [x.cpu().numpy().copy() for x in (cache.ks, cache.vs)]
    for _ in range(2):                               # a second call releases what the first gave
        fl.kv_fork(*cache.tensors(), t, r, ints(parents), ints(children), ints(lengths))
        table, refs, copies, fine = oracle.kv_fork(table, refs, parents, children, lengths, page)
        for a, b, n in copies:
            for x in host:
                x[b, :n] = x[a, :n]
        if fine:
            fl.device_status()
        else:
            with pytest.raises(fl.FusedLinError):
                fl.device_status()
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
        for x, y in zip((cache.k, cache.v, cache.ks, cache.vs), host):
            assert np.array_equal((x if x.dtype == torch.float32 else x.view(torch.uint8)).cpu().numpy(), y)
        lengths = lengths[::-1].copy()
        lengths = np.minimum(lengths, np.repeat(lens, each))


def test_kv_fork_bad_sequences_and_missing_pages():
    rng = gen(62)
    cache = Paged(rng, [40, 0, 0, 0], 1, 64, 16, "int8")
    cache.table[0, 1] = -1
    refs = np.bincount(cache.table[cache.table >= 0], minlength=cache.pages).astype(np.int32)
    for parents, children, lengths in (([0, 0], [1, 9], [40, 40]), ([-1, 0], [1, 2], [5, 16]), ([0], [3], [20]), ([0], [2], [9999])):
        t, r = ints(cache.table), ints(refs)
        fl.kv_fork(*cache.tensors(), t, r, ints(parents), ints(children), ints(lengths))
        with pytest.raises(fl.FusedLinError):
            fl.device_status()
        want, want_refs, _, fine = oracle.kv_fork(cache.table, refs, parents, children, lengths, 16)
        assert not fine and np.array_equal(t.cpu().numpy(), want) and np.array_equal(r.cpu().numpy(), want_refs)
    fl.kv_fork(*cache.tensors(), t, r, ints([]), ints([]), ints([]))
    fl.device_status()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("H,D,page,B,drafts,most", [(1, 64, 16, 1, 1, 1), (2, 128, 16, 3, 20, 20), (5, 24, 7, 4, 64, 17), (3, 8, 5, 2, 30, 9),
                                                    (8, 128, 64, 9, 64, 40), (1, 256, 16, 2, 200, 130), (40, 128, 16, 2, 12, 6)])
def test_kv_compact(fmt, H, D, page, B, drafts, most):
    rng = gen(63, H, D, page, drafts)
    start = rng.integers(0, 100, B)
    start[0] = 0
    cache = Paged(rng, [int(s) + drafts for s in start], H, D, page, fmt)
    acc = np.full((B, most), -1, dtype=np.int32)
    for b in range(B):
        n = int(rng.integers(0, min(most, drafts) + 1)) if b else min(most, drafts)
        acc[b, :n] = np.sort(rng.choice(drafts, n, replace=False))
        if b == B - 1 and n < most:
            acc[b, n + 1:] = 3                       # behind the end: not read
    host = [x.view(torch.uint8).cpu().numpy().copy() for x in (cache.k, cache.v)] + [x.cpu().numpy().copy() for x in (cache.ks, cache.vs)]
    fl.kv_compact(*cache.tensors(), ints(cache.table), ints(start), ints(acc))
    fl.device_status()
    moves, fine = oracle.kv_compact(cache.table, cache.pages, start, acc, page)
    assert fine
    for src, dst in moves:
        for x in host:
            x[dst] = x[src]
    for x, y in zip(cache.tensors(), host):
        assert np.array_equal((x if x.dtype == torch.float32 else x.view(torch.uint8)).cpu().numpy(), y)


def test_kv_compact_rows_without_a_page():
    rng = gen(64)
    cache = Paged(rng, [50, 60], 2, 64, 16, "int8")
    table = cache.table.copy()
    table[0, 2] = -1
    acc, start = [[0, 2, 20, 90], [1, 4, -1, 7]], [20, 30]
    host = [cache.k.cpu().numpy().copy(), cache.ks.cpu().numpy().copy()]
    fl.kv_compact(*cache.tensors(), ints(table), ints(start), ints(acc))
    with pytest.raises(fl.FusedLinError) as e:
        fl.device_status()
    assert e.value.status == 7
    moves, fine = oracle.kv_compact(table, cache.pages, start, np.array(acc), 16)
    assert not fine and moves
    for src, dst in moves:
        for x in host:
            x[dst] = x[src]
    assert np.array_equal(cache.k.cpu().numpy(), host[0]) and np.array_equal(cache.ks.cpu().numpy(), host[1])
    fl.kv_compact(*cache.tensors(), ints(table), ints([0, 0]), ints([[1, 1], [-1, 5]])[:, :0].contiguous())
    fl.device_status()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("B,H,hq,D,page,rows,spread", [(300, 2, 4, 64, 16, 1, 3), (700, 1, 3, 128, 16, 3, 2), (1100, 1, 4, 64, 64, 9, 1)])
def test_kv_attend_many_sequences(fmt, B, H, hq, D, page, rows, spread):
    """More sequences than a CTA has threads, a few of them long, so that some are split; some without rows."""
    rng = gen(71, B, H, hq)
    n_rows = rng.integers(max(0, rows - spread), rows + spread + 1, B).tolist()
    start = rng.integers(0, 40, B)
    start[::97] = rng.integers(1000, 1500, len(start[::97]))
    start = start.tolist()
    cache = Paged(rng, [a + b for a, b in zip(n_rows, start)], H, D, page, fmt)
    got, ref, q = attend_case(rng, "bf16", cache, hq, n_rows, start)
    fl.device_status()
    attend_check(got, ref, "bf16", cache, n_rows, start)
    again = fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints(start), cu_rows=ints(sums(n_rows)))
    assert torch.equal(again, got)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group,n", [(1, 1), (4, 12)])
def test_cache_of_more_bytes_than_32_bits_count(fmt, group, n):
    """The last pages of a cache of more than 2^32 bytes of k, and of v, answer as the first ones of a small cache do: rows
    written, attended, forked and moved."""
    rng = gen(72, group, n)
    H, D, page, per, B = 8, 128, 64, 20, 3
    pages = (1 << 32) // (page * H * D) + 200
    start = [1150, 64, 100]
    answers = []
    for n_pages, first in ((100, 0), (pages, pages - 100)):
        code = FMT[fmt][0]
        cache = [torch.zeros((n_pages, page, H, D), dtype=torch.int8, device="cuda").view(code) for _ in "kv"]
        cache += [torch.ones((n_pages, page, H), device="cuda") for _ in "kv"]
        assert n_pages == 100 or cache[0].numel() > 1 << 32
        r = gen(73, group, n)
        refs = torch.ones(n_pages, dtype=torch.int32, device="cuda")
        refs[first:first + 100] = 0
        table = torch.full((B, per), -1, dtype=torch.int32, device="cuda")
        total = [s + n for s in start]
        fl.kv_resize(table, refs, ints(total[:2] + [0]), page)
        k, v = (put(r.standard_normal((sum(total[:2]), H, D)), "bf16") for _ in "kv")
        fl.kv_write(k, v, *cache, table, ints([0, 0, 0]), cu_rows=ints(sums(total[:2] + [0])))
        fl.kv_fork(*cache, table, refs, ints([0]), ints([2]), ints([start[2]]))
        fl.kv_resize(table, refs, ints(total), page)
        k, v = (put(r.standard_normal((n, H, D)), "bf16") for _ in "kv")
        fl.kv_write(k, v, *cache, table, ints([0, 0, start[2]]), cu_rows=ints([0, 0, 0, n]))
        q = put(r.standard_normal((B * n, H * group, D)), "bf16")
        cu = ints([0, n, 2 * n, 3 * n])
        out = [fl.kv_attend(q, *cache, table, ints(start), cu_rows=cu)]
        if n > 1:
            fl.kv_compact(*cache, table, ints(start), ints([[1, 3, 7], [0, 11, -1], [-1, 0, 0]]))
            out.append(fl.kv_attend(q, *cache, table, ints(start), cu_rows=cu))
        back = [torch.empty((sum(total), H, D), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        fl.kv_read(*cache, table, ints(sums(total)), out_k=back[0], out_v=back[1])
        fl.device_status()
        answers.append((table - first * (table >= 0), refs[first:first + 100].clone(), *out, *back))
        del cache
    for a, b in zip(*answers):
        assert torch.equal(a, b)
    assert not torch.equal(answers[0][2], torch.zeros_like(answers[0][2]))


def test_attention_strides_past_32_bits():
    """Rows and heads whose places lie more than 2^32 bytes apart."""
    rng = gen(74)
    big = torch.empty((300, 1 << 23), dtype=torch.bfloat16, device="cuda")
    assert big.numel() * 2 > 1 << 32
    views = [big[:, i * 1024:i * 1024 + 256].unflatten(1, (2, 128)) for i in range(4)]
    q, k, v = (put(rng.standard_normal((300, 2, 128)), "bf16") for _ in "qkv")
    for x, y in zip(views, (q, k, v)):
        x.copy_(y)
    for cu in (None, ints([0, 17, 290])):
        want, out = torch.full_like(q, 7.0), views[3]
        out.fill_(7.0)
        fl.attention(q, k, v, cu_q=cu, out=want)
        fl.attention(*views[:3], cu_q=cu, out=out)
        fl.device_status()
        assert torch.equal(out, want)


def test_calls_without_overlapped_launches():
    """The same answers when a kernel starts only once the one before it has ended."""
    rng = gen(75)
    q = put(rng.standard_normal((40, 4, 64)), "f16")
    kv = put(rng.standard_normal((5000, 1, 64)), "f16")
    start = [5000, 30]
    cache = Paged(rng, [5020, 50], 2, 64, 16, "int8")
    x = put(rng.standard_normal((40, 4, 64)), "f16")

    def calls():
        refs = ints(np.bincount(cache.table[cache.table >= 0], minlength=cache.pages))
        table = ints(cache.table)
        a = fl.attention(q, kv, kv)
        b = fl.kv_attend(x, *cache.tensors(), table, ints(start), cu_rows=ints([0, 20, 40]))
        fl.kv_resize(table, refs, ints([100, 70]), 16)
        return a, b, table, refs

    want = calls()
    fl.set_option("pdl", 0)
    try:
        got = calls()
    finally:
        fl.set_option("pdl", 1)
    fl.device_status()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# a step as it is used
# ---------------------------------------------------------------------------
def test_speculative_step_in_one_graph():
    """Pages taken, drafts rotated and written, their tree verified, accepted rows moved, pages given back: captured once,
    replayed for two steps, and the cache that is left attended by a plain decode step, against the oracle."""
    rng = gen(65)
    H, hq, D, page, per, pages, B, n = 2, 8, 64, 16, 12, 40, 3, 9
    k_cache, v_cache = (torch.zeros((pages, page, H, D), dtype=torch.int8, device="cuda") for _ in "kv")
    k_scale, v_scale = (torch.full((pages, page, H), float("nan"), device="cuda") for _ in "kv")
    cache = (k_cache, v_cache, k_scale, v_scale)
    table, refs = torch.full((B, per), -1, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    length = ints([0, 0, 0])
    # prompts: attended on their 16-bit keys, then cached
    lens = [33, 5, 60]
    cu = ints(sums(lens))
    q, k, v = (put(rng.standard_normal((sum(lens), h, D)), "bf16") for h in (hq, H, H))
    out = fl.attention(q, k, v, cu_q=cu)
    ref = oracle.attention(f64(q), f64(k), f64(v), sums(lens), sums(lens), True, D ** -0.5)
    check(out, ref, U["bf16"], U["bf16"], 2.0 ** -20, np.zeros((sum(lens), hq)))
    fl.kv_resize(table, refs, ints(lens), page)
    fl.kv_write(k, v, *cache, table, length, cu_rows=cu)
    length += ints(lens)
    # one drafted step as a graph
    inv_freq = torch.ones(D // 2, device="cuda") * 0.01
    qd, kd, vd = (torch.zeros((B * n, h, D), dtype=torch.bfloat16, device="cuda") for h in (hq, H, H))
    pos = torch.zeros(B * n, dtype=torch.int32, device="cuda")
    cu_d = ints([0, n, 2 * n, 3 * n])
    tree = torch.zeros((B * n, n), dtype=torch.bool, device="cuda")
    accepted = torch.full((B, 5), -1, dtype=torch.int32, device="cuda")
    room, kept = ints([0] * B), ints([0] * B)
    o = torch.zeros_like(qd)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def step():
        fl.kv_resize(table, refs, room, page)
        fl.rope(qd, kd, pos, inv_freq, out_q=qd, out_k=kd)
        fl.kv_write(kd, vd, *cache, table, length, cu_rows=cu_d)
        fl.kv_attend(qd, *cache, table, length, cu_rows=cu_d, tree=tree, out=o)
        fl.kv_compact(*cache, table, length, accepted)
        fl.kv_resize(table, refs, kept, page)

    with torch.cuda.stream(s):
        graph = fl.Graph.capture(step)
    host_k = [oracle_rows(f64(k)[sums(lens)[b]:sums(lens)[b + 1]]) for b in range(B)]
    host_v = [oracle_rows(f64(v)[sums(lens)[b]:sums(lens)[b + 1]]) for b in range(B)]
    at = list(lens)
    for turn in range(2):
        qn, kn, vn = (put(rng.standard_normal((B * n, h, D)), "bf16") for h in (hq, H, H))
        sees = np.zeros((B * n, n), dtype=bool)
        parent = np.array([-1] + [int(rng.integers(0, i)) for i in range(1, n)])
        for b in range(B):
            for i in range(n):
                j = i
                while j >= 0:
                    sees[b * n + i, j] = True
                    j = parent[j]
        acc = []
        for b in range(B):                              # a path from the root
            path, j = [], int(rng.integers(1, n))
            while j >= 0:
                path.append(j)
                j = parent[j]
            acc.append((path[::-1] + [-1] * 5)[:5])
        keep = [sum(x >= 0 for x in a) for a in acc]
        acc = np.array(acc)
        depth = sees.sum(1) - 1
        with torch.cuda.stream(s):
            qd.copy_(qn), kd.copy_(kn), vd.copy_(vn)
            pos.copy_(ints(np.repeat(at, n) + depth))
            tree.copy_(put(sees)), accepted.copy_(ints(acc))
            room.copy_(length + n), kept.copy_(length + ints(keep))
            graph.launch()
            qr, kr = f64(qd), f64(kd)
            length.copy_(kept)
        fl.device_status(s)
        ks, vs = [], []
        for b in range(B):
            ks.append(np.concatenate((host_k[b], oracle_rows(kr[b * n:(b + 1) * n]))))
            vs.append(np.concatenate((host_v[b], oracle_rows(f64(vn)[b * n:(b + 1) * n]))))
        ref = oracle.kv_attend(qr, ks, vs, [np.ones(len(x), bool) for x in ks], [0, n, 2 * n, 3 * n], at, sees, D ** -0.5)
        # (scales of rows of unit variance: 0.02 to 0.04)
        floor = 200 * 2.0 ** -25 * 127 * 0.06 * ref["top"]
        check(o, ref, U["bf16"], 2.0 ** -11, 2.0 ** -18, floor, f"turn {turn}")
        for b in range(B):
            rows = [at[b] + a for a in acc[b] if a >= 0]
            host_k[b], host_v[b] = (np.concatenate((x[b][:at[b]], x[b][rows])) for x in (ks, vs))
            at[b] += keep[b]
        held = (table >= 0).sum(1).tolist()
        assert held == [-(-a // page) for a in at] and int(refs.sum()) == sum(held) and int(refs.max()) == 1
    # what is left, seen by one more row of each; and by a forked sequence's row
    table2 = torch.cat((table, torch.full((1, per), -1, dtype=torch.int32, device="cuda")))
    fl.kv_fork(*cache, table2, refs, ints([2]), ints([3]), ints([at[2]]))
    q1 = put(rng.standard_normal((4, hq, D)), "bf16")
    q1[3] = q1[2]
    k1, v1 = (put(rng.standard_normal((4, H, D)), "bf16") for _ in "kv")
    start = ints(at + [at[2]])
    fl.kv_resize(table2, refs, start + 1, page)
    fl.kv_write(k1, v1, *cache, table2, start)
    got = fl.kv_attend(q1, *cache, table2, start)
    fl.device_status()
    src = [0, 1, 2, 2]
    ks, vs = ([np.concatenate((h[b], oracle_rows(f64(x)[i:i + 1]))) for i, b in enumerate(src)] for h, x in ((host_k, k1), (host_v, v1)))
    ref = oracle.kv_attend(f64(q1), ks, vs, [np.ones(len(x), bool) for x in ks], [0, 1, 2, 3, 4], at + [at[2]], None, D ** -0.5)
    check(got, ref, U["bf16"], 2.0 ** -11, 2.0 ** -18, 200 * 2.0 ** -25 * 127 * 0.06 * ref["top"])


def oracle_rows(x):
    """Rows as the int8 cache holds them."""
    code, scale = oracle.kv_quantize(x, "int8")
    return code * scale[..., None]
