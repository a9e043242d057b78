"""Cases of the operators of a decoder layer served from 4-bit weights and an 8-bit cache.

w4_quantize   a 16-bit weight [N, K] to 4-bit codes with one scale per group of K
w4_gemm       act(RMSNorm(x) W^T + bias) (+ residual) on such a weight, from one row to a prompt
w4_ffn        the SwiGLU block on three such weights
rope          rotary positions of q and k, with one or several position axes
kv_write      k and v rows quantised to 8 bits into a paged cache
kv_read       rows of that cache as 16-bit k and v

Sizes are those of the library's own workloads (D = 1024, 2048, 4096, F = 2816, 11008, k/v width 1024, heads of
128 channels) and ragged ones around them.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
CACHES = {"int8": (torch.int8, 127.0), "fp8": (torch.float8_e4m3fn, 448.0)}
EPS = 1e-6
TINY = 2.0 ** -126  # the smallest scale of a cache row


def listed():
    return [
        # one weight matrix of the smallest model of the decode sweep, quantised once when it is loaded
        {"name": "w4_quantize bf16 1024x1024 g32", "op": "w4_quantize", "dtype": "bf16", "N": 1024, "K": 1024, "group": 32},
        # the largest matrix of the FFN configuration
        {"name": "w4_quantize f16 11008x4096 g128", "op": "w4_quantize", "dtype": "f16", "N": 11008, "K": 4096, "group": 128},
        # the smallest call: one token through one 1024-wide projection behind its norm
        {"name": "w4_gemm bf16 1x1024x1024", "op": "w4_gemm", "dtype": "bf16", "M": 1, "N": 1024, "K": 1024, "group": 128,
         "zeros": False, "norm": True, "act": "none", "bias": False, "residual": False},
        # a short prompt through the stacked q, k and v projection, asymmetric weights
        {"name": "w4_gemm f16 333x6144x4096 zeros", "op": "w4_gemm", "dtype": "f16", "M": 333, "N": 6144, "K": 4096,
         "group": 64, "zeros": True, "norm": True, "act": "none", "bias": True, "residual": False},
        # a decode step of three sequences through the FFN block
        {"name": "w4_ffn bf16 3x4096x11008", "op": "w4_ffn", "dtype": "bf16", "M": 3, "D": 4096, "F": 11008, "group": 128,
         "zeros": False},
        # a long prompt through the FFN block
        {"name": "w4_ffn bf16 2048x4096x11008", "op": "w4_ffn", "dtype": "bf16", "M": 2048, "D": 4096, "F": 11008,
         "group": 128, "zeros": False},
        # a decode step of seven sequences far into their contexts, one position axis
        {"name": "rope bf16 7 rows", "op": "rope", "dtype": "bf16", "rows": 7, "hq": 32, "hkv": 8, "D": 128, "R": 128,
         "axes": 1, "far": True, "interleaved": False, "inverse": False},
        # a prompt of text, image and video tokens: time, height and width axes
        {"name": "rope f16 4099 rows 3 axes", "op": "rope", "dtype": "f16", "rows": 4099, "hq": 32, "hkv": 8, "D": 128,
         "R": 128, "axes": 3, "far": False, "interleaved": False, "inverse": False},
        # a decode step: one new token of each of 61 sequences
        {"name": "kv_write int8 bf16 61x1", "op": "kv_write", "dtype": "bf16", "cache": "int8", "seqs": 61, "rows": 61,
         "H": 8, "D": 128, "page": 16, "context": 150, "pad": 0},
        # three prompts appended at once, k and v being column ranges of the stacked projection's output
        {"name": "kv_write fp8 f16 3 prompts", "op": "kv_write", "dtype": "f16", "cache": "fp8", "seqs": 3, "rows": 4099,
         "H": 8, "D": 128, "page": 64, "context": 700, "pad": 13},
        # the context of one short conversation for an attention kernel that takes 16-bit k and v
        {"name": "kv_read fp8 bf16 1x37", "op": "kv_read", "dtype": "bf16", "cache": "fp8", "seqs": 1, "rows": 37, "H": 8,
         "D": 128, "page": 16, "context": 0, "pad": 0},
        # a batch of long contexts
        {"name": "kv_read int8 f16 16 long", "op": "kv_read", "dtype": "f16", "cache": "int8", "seqs": 16, "rows": 60001,
         "H": 8, "D": 128, "page": 64, "context": 0, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w4_quantize", "w4_gemm", "w4_gemm", "w4_ffn", "rope", "kv_write", "kv_read"])
    c = {"op": op, "dtype": rng.choice(["f16", "bf16"])}
    if op == "w4_quantize":
        c["group"] = rng.choice([32, 64, 128])
        c["N"] = 8 * _log(rng, 8, 1300)
        c["K"] = c["group"] * max(1, _log(rng, 256, 4096) // c["group"])
    elif op == "w4_gemm":
        c["group"] = rng.choice([32, 64, 128])
        c["M"] = _log(rng, 1, 2048)
        c["N"] = 8 * _log(rng, 32, 1376)
        c["K"] = c["group"] * max(1, _log(rng, 256, 8192) // c["group"])
        c.update(zeros=rng.random() < 0.5, norm=rng.random() < 0.5, act=rng.choice(["none", "gelu", "silu", "relu"]),
                 bias=rng.random() < 0.5, residual=rng.random() < 0.5)
        if c["act"] != "none":
            c["residual"] = False
    elif op == "w4_ffn":
        c["group"] = rng.choice([32, 64, 128])
        c["M"] = _log(rng, 1, 1024)
        c["D"] = 128 * _log(rng, 4, 32)
        c["F"] = 128 * _log(rng, 8, 86)
        c["zeros"] = rng.random() < 0.5
    elif op == "rope":
        c["rows"] = _log(rng, 1, 4000)
        c["D"] = rng.choice([64, 96, 128])
        c["R"] = rng.choice([c["D"], c["D"] // 2])
        c["hkv"] = rng.choice([1, 2, 4, 8])
        c["hq"] = c["hkv"] * rng.choice([1, 3, 4])
        c.update(axes=rng.choice([1, 2, 3]), far=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                 inverse=rng.random() < 0.3)
    else:
        c["cache"] = rng.choice(["int8", "fp8"])
        c["rows"] = _log(rng, 1, 4000 if op == "kv_write" else 40000)
        c["seqs"] = min(c["rows"], _log(rng, 1, 64))
        if op == "kv_write" and rng.random() < 0.3:
            c["rows"] = c["seqs"]
        c["H"] = rng.choice([1, 2, 5, 8])
        c["D"] = rng.choice([64, 80, 128])
        c["page"] = rng.choice([16, 32, 64])
        c["context"] = _log(rng, 1, 1000) if op == "kv_write" else 0
        c["pad"] = rng.choice([0, 0, 5])
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _weight4(g, N, K, group, zeros, dtype):
    """Codes two to a byte (the even k in the low half), group scales, zero points or None, of a weight of variance 1/K."""
    code = (_randn(g, N, K) * 2.6 + 8.0).round_().clamp_(0, 15).to(torch.uint8)
    q = code[:, 0::2] | (code[:, 1::2] << 4)
    s = ((1.0 + 0.15 * _randn(g, N, K // group)).clamp_(0.4, 1.8) / (2.6 * math.sqrt(K))).to(dtype)
    z = torch.randint(6, 11, (N, K // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return q.contiguous(), s, z


def _rows(g, M, K, dtype):
    """Activations with a few channels that are much larger than the rest."""
    x = _randn(g, M, K)
    x[:, torch.randint(0, K, (max(1, K // 512),), generator=g, device="cuda")] *= 12.0
    return x.to(dtype)


def _spread(g, seqs, rows):
    """Row offsets of `seqs` sequences over `rows` rows, each with one row at least where there are enough."""
    if rows == seqs:
        n = torch.ones(seqs, device="cuda")
    else:
        w = torch.rand(seqs, generator=g, device="cuda") + 0.05
        n = 1 + torch.floor(w / w.sum() * (rows - seqs))
        n[0] += rows - n.sum()
    cu = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    cu[1:] = n.cumsum(0).to(torch.int32)
    return cu


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    dt = DTYPES[c["dtype"]]
    op = c["op"]
    s = {"case": c}
    if op == "w4_quantize":
        s["W"] = (_randn(g, c["N"], c["K"]) / math.sqrt(c["K"])).to(dt)
    elif op == "w4_gemm":
        M, N, K = c["M"], c["N"], c["K"]
        s["x"] = _rows(g, M, K, dt)
        s["q"], s["scales"], s["zeros"] = _weight4(g, N, K, c["group"], c["zeros"], dt)
        s["gamma"] = (1.0 + 0.1 * _randn(g, K)).to(dt) if c["norm"] else None
        s["bias"] = (0.1 * _randn(g, N)).to(dt) if c["bias"] else None
        s["residual"] = _randn(g, M, N).to(dt) if c["residual"] else None
    elif op == "w4_ffn":
        M, D, F = c["M"], c["D"], c["F"]
        s["x"] = _rows(g, M, D, dt)
        s["gamma"] = (1.0 + 0.1 * _randn(g, D)).to(dt)
        s["Wg"] = _weight4(g, F, D, c["group"], c["zeros"], dt)
        s["Wu"] = _weight4(g, F, D, c["group"], c["zeros"], dt)
        s["Wd"] = _weight4(g, D, F, c["group"], c["zeros"], dt)
    elif op == "rope":
        T, hq, hkv, D, R, A = c["rows"], c["hq"], c["hkv"], c["D"], c["R"], c["axes"]
        # q and k as the stacked projection leaves them, side by side in one row (v behind them)
        qkv = _randn(g, T, (hq + 2 * hkv) * D).to(dt)
        s["q"] = qkv[:, :hq * D].unflatten(1, (hq, D))
        s["k"] = qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
        base = 10000.0 if not c["far"] else 500000.0
        s["inv_freq"] = base ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        s["inv_freq"] = s["inv_freq"].float()
        if c["far"]:
            pos = torch.randint(0, 1 << 20, (A, T), generator=g, device="cuda")
        else:
            pos = torch.arange(T, device="cuda")[None, :] + torch.randint(0, 90, (A, T), generator=g, device="cuda")
        s["positions"] = pos.to(torch.int32)
        n = R // 2
        s["sections"] = [n - (A - 1) * (n * 3 // 8)] + [n * 3 // 8] * (A - 1)
    else:
        B, T, H, D, page = c["seqs"], c["rows"], c["H"], c["D"], c["page"]
        cu = _spread(g, B, T)
        start = torch.randint(0, c["context"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        # a pool of pages in random order; a sequence's table row ends with -1 where it has no page
        pages = B + -(-(T + B * c["context"]) // page)
        need = (start + cu[1:] - cu[:-1] + page - 1) // page
        first = need.cumsum(0) - need
        j = torch.arange(-(-(T + c["context"]) // page), device="cuda")
        order = torch.randperm(pages, generator=g, device="cuda")
        table = order[(first[:, None] + j).clamp(max=pages - 1)]
        s["page_table"] = torch.where(j < need[:, None], table, -1).to(torch.int32)
        s["cu_rows"] = cu
        s["start"] = start
        code, top = CACHES[c["cache"]]
        shape = (pages, page, H, D)
        for n in "kv":
            s[n + "_cache"] = (_randn(g, *shape) * top / 4).clamp_(-top, top).to(code)
            s[n + "_scale"] = 0.01 + 0.02 * torch.rand(shape[:3], generator=g, device="cuda")
        if op == "kv_write":
            # k and v side by side in the rows of the stacked projection, q in front of them
            qkv = _randn(g, T + c["pad"], 6 * H * D).to(dt)
            s["k"] = qkv[:, 4 * H * D:5 * H * D].unflatten(1, (H, D))
            s["v"] = qkv[:, 5 * H * D:].unflatten(1, (H, D))
        else:
            s["out_k"] = torch.zeros(T + c["pad"], H, D, dtype=dt, device="cuda")
            s["out_v"] = torch.zeros(T + c["pad"], H, D, dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_weight(q, scales, zeros):
    N, K = q.shape[0], q.shape[1] * 2
    code = torch.stack((q & 15, q >> 4), 2).reshape(N, scales.shape[1], -1).float()
    z = 8.0 if zeros is None else zeros.float()[:, :, None]
    return ((code - z) * scales.float()[:, :, None]).reshape(N, K)


def _plain_norm(x, gamma):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * gamma.float()


def _plain_act(y, act):
    if act == "gelu":
        return 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    if act == "silu":
        return y / (1.0 + torch.exp(-y))
    return torch.clamp(y, min=0.0) if act == "relu" else y


def _plain_rotate(x, cos, sin, R, interleaved):
    out = x.float()
    if interleaved:
        a, b = out[..., 0:R:2], out[..., 1:R:2]
        rot = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = out[..., :R // 2], out[..., R // 2:R]
        rot = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((rot, out[..., R:]), -1).to(x.dtype)


def _plain_slots(s, rows):
    """Page and place in the page of each of the first `rows` rows."""
    i = torch.arange(rows, device="cuda")
    cu = s["cu_rows"].long()
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    p = s["start"].long()[b] + i - cu[b]
    size = s["k_cache"].shape[1]
    return s["page_table"].long()[b, p // size], p % size


def _plain_codes(x, code, top):
    x = x.float()
    scale = torch.clamp(x.abs().amax(-1) / top, min=TINY)
    y = x.double() / scale.double()[..., None]  # in 64 bits: values next to a border between two codes
    if code == torch.int8:
        return y.round().clamp(-127, 127).to(code), scale
    # e4m3: three bits behind the leading one, from 2^-6 up
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
    return ((y / step).round() * step).clamp(-448, 448).to(code), scale


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import gemm_epilogue_tma_gb300 as fl
        if op == "w4_quantize":
            return fl.w4_quantize(s["W"], group=c["group"])
        if op == "w4_gemm":
            return fl.w4_gemm(s["x"], s["q"], s["scales"], zeros=s["zeros"], gamma=s["gamma"], bias=s["bias"],
                              residual=s["residual"], eps=EPS, act=c["act"])
        if op == "w4_ffn":
            return fl.w4_swiglu_ffn(s["x"], s["gamma"], s["Wg"], s["Wu"], s["Wd"], eps=EPS)
        if op == "rope":
            return fl.rope(s["q"], s["k"], s["positions"], s["inv_freq"], sections=s["sections"],
                           interleaved=c["interleaved"], inverse=c["inverse"])
        if op == "kv_write":
            fl.kv_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"],
                        s["start"], cu_rows=s["cu_rows"])
            return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
        return fl.kv_read(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"], s["cu_rows"],
                          start=s["start"], out_k=s["out_k"], out_v=s["out_v"])
    if op == "w4_quantize":
        W = s["W"]
        w = W.float().unflatten(1, (-1, c["group"]))
        least = 2.0 ** -24 if W.dtype == torch.float16 else 2.0 ** -133
        scales = torch.clamp(w.abs().amax(2) / 7.0, min=least).to(W.dtype)
        code = (w / scales.float()[:, :, None]).round().clamp(-7, 7).add(8.0).to(torch.uint8).flatten(1)
        return code[:, 0::2] | (code[:, 1::2] << 4), scales
    if op == "w4_gemm":
        x = s["x"].float() if s["gamma"] is None else _plain_norm(s["x"], s["gamma"])
        y = x @ _plain_weight(s["q"], s["scales"], s["zeros"]).t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        y = _plain_act(y, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(s["x"].dtype)
    if op == "w4_ffn":
        x = _plain_norm(s["x"], s["gamma"])
        h = _plain_act(x @ _plain_weight(*s["Wg"]).t(), "silu") * (x @ _plain_weight(*s["Wu"]).t())
        return (h @ _plain_weight(*s["Wd"]).t() + s["x"].float()).to(s["x"].dtype)
    if op == "rope":
        axis = torch.cat([s["positions"][a:a + 1].expand(n, -1) for a, n in enumerate(s["sections"])])
        angle = axis.t().double() * s["inv_freq"].double()  # in 64 bits: angles of far positions
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
        if c["inverse"]:
            sin = -sin
        return tuple(_plain_rotate(t, cos, sin, c["R"], c["interleaved"]) for t in (s["q"], s["k"]))
    page, at = _plain_slots(s, c["rows"])
    if op == "kv_write":
        code, top = CACHES[c["cache"]]
        for n in "kv":
            q, scale = _plain_codes(s[n][:c["rows"]], code, top)
            # (by bytes: not every torch version indexes 8-bit floats)
            s[n + "_cache"].view(torch.uint8)[page, at] = q.view(torch.uint8)
            s[n + "_scale"][page, at] = scale
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    for n in "kv":
        got = s[n + "_cache"].view(torch.uint8)[page, at].view(s[n + "_cache"].dtype).float()
        s["out_" + n][:c["rows"]] = (got * s[n + "_scale"][page, at][..., None]).to(s["out_" + n].dtype)
    return s["out_k"], s["out_v"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _w4_bytes(N, K, group, zeros):
    return N * K / 2 + N * (K // group) * (3 if zeros else 2)


def work(case):
    c = case
    op = c["op"]
    if op == "w4_quantize":
        n = c["N"] * c["K"]
        return {"bytes": 2 * n + n / 2 + 2 * n / c["group"], "flops": 3 * n}
    if op == "w4_gemm":
        M, N, K = c["M"], c["N"], c["K"]
        b = 2 * M * K + 2 * M * N * (2 if c["residual"] else 1) + _w4_bytes(N, K, c["group"], c["zeros"])
        return {"bytes": b + (2 * K if c["norm"] else 0) + (2 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    if op == "w4_ffn":
        M, D, F = c["M"], c["D"], c["F"]
        w = 2 * _w4_bytes(F, D, c["group"], c["zeros"]) + _w4_bytes(D, F, c["group"], c["zeros"])
        return {"bytes": 4 * M * D + 2 * D + w, "flops": 6 * M * D * F}
    if op == "rope":
        n = c["rows"] * (c["hq"] + c["hkv"])
        return {"bytes": 4 * n * c["D"] + 4 * c["rows"] * c["axes"] + 2 * c["R"], "flops": 3 * n * c["R"]}
    n = 2 * c["rows"] * c["H"]
    index = 4 * (2 * c["seqs"] + 1) + 4 * (c["rows"] // c["page"] + c["seqs"])
    return {"bytes": n * (3 * c["D"] + 4) + index, "flops": (3 if op == "kv_write" else 1) * n * c["D"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_weight(w):
    q, scales, zeros = w
    N, G = scales.shape
    even, odd = (q % 16).double(), torch.div(q, 16, rounding_mode="floor").double()
    W = torch.empty(N, q.shape[1] * 2, dtype=torch.float64, device="cuda")
    W[:, 0::2] = even
    W[:, 1::2] = odd
    z = torch.full((N, G), 8.0, dtype=torch.float64, device="cuda") if zeros is None else zeros.double()
    each = W.shape[1] // G
    return (W - z.repeat_interleave(each, 1)) * scales.double().repeat_interleave(each, 1)


def _exact_norm(x, gamma):
    x = x.double()
    return x / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + EPS) * gamma.double()


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    op = c["op"]
    if op == "w4_quantize":
        W = s["W"].double().reshape(c["N"], -1, c["group"])
        least = 2.0 ** -24 if s["W"].dtype == torch.float16 else 2.0 ** -133
        scale = (W.abs().max(dim=2).values / 7).clamp_min(least).to(s["W"].dtype).double()
        code = 8 + torch.round(W / scale.unsqueeze(2)).clamp(-7, 7).reshape(c["N"], c["K"])
        return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8), scale
    if op == "w4_gemm":
        x = s["x"].double() if s["gamma"] is None else _exact_norm(s["x"], s["gamma"])
        y = torch.matmul(x, _exact_weight((s["q"], s["scales"], s["zeros"])).T)
        if s["bias"] is not None:
            y += s["bias"].double()
        if c["act"] == "gelu":
            y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
        elif c["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif c["act"] == "relu":
            y = torch.where(y > 0, y, torch.zeros_like(y))
        return y if s["residual"] is None else y + s["residual"].double()
    if op == "w4_ffn":
        x = _exact_norm(s["x"], s["gamma"])
        gate, up = (torch.matmul(x, _exact_weight(s[n]).T) for n in ("Wg", "Wu"))
        return torch.matmul(gate * torch.sigmoid(gate) * up, _exact_weight(s["Wd"]).T) + s["x"].double()
    if op == "rope":
        n, sign = c["R"] // 2, -1.0 if c["inverse"] else 1.0
        of_pair = torch.tensor([a for a, m in enumerate(s["sections"]) for _ in range(m)], device="cuda")
        angle = sign * s["positions"].double().index_select(0, of_pair).T * s["inv_freq"].double()
        turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
        outs = []
        for t in (s["q"], s["k"]):
            y = t.double().clone()
            lo = torch.arange(n, device="cuda") * (2 if c["interleaved"] else 1)
            hi = lo + (1 if c["interleaved"] else n)
            z = torch.complex(y[..., lo], y[..., hi]) * turn
            y[..., lo], y[..., hi] = z.real, z.imag
            outs.append(y)
        return tuple(outs)
    B, size = c["seqs"], c["page"]
    cu, start = s["cu_rows"].tolist(), s["start"].tolist()
    slot = torch.cat([s["page_table"][b].long()[p // size] * size + p % size for b in range(B)
                      for p in [torch.arange(start[b], start[b] + cu[b + 1] - cu[b], device="cuda")]])
    if op == "kv_write":
        # the codes' own values are whole numbers, or 8-bit floats: what is left to compare is the scales
        outs = [None, None]
        for n in "kv":
            scale = s[n + "_scale"].double().reshape(-1, c["H"])
            scale[slot] = (s[n][:c["rows"]].double().abs().max(dim=2).values / CACHES[c["cache"]][1]).clamp_min(TINY)
            outs.append(scale.reshape(s[n + "_scale"].shape))
        return tuple(outs)
    outs = []
    for n in "kv":
        flat = s[n + "_cache"].float().double().reshape(-1, c["H"], c["D"])
        out = torch.zeros(c["rows"] + c["pad"], c["H"], c["D"], dtype=torch.float64, device="cuda")
        out[:c["rows"]] = flat[slot] * s[n + "_scale"].double().reshape(-1, c["H"])[slot].unsqueeze(2)
        outs.append(out)
    return tuple(outs)
