"""The operators of a draft layer in 8 bits as work to be measured: the norm that ends in 8 bits, the
matrix product with its epilogue, and keys that are rotated on their way into the 4-bit cache.

8-bit rows.  A row y stands as codes c (e4m3, four bits of exponent and three of mantissa) and one scale
s in fp32:  s = max(max |y| / 448, 2^-100),  c = y / s rounded to the nearest e4m3 value (ties to even);
the row's values are s c.

norm     h = x + residual (or x);  y = w h / sqrt(mean(h^2) + eps), and h itself where a residual was
         added; y in bf16 or as an 8-bit row.  Without the norm y = x: rows quantised as they are.
linear   y = act(s_x s_w (x w^T) + bias) + residual for bf16 operands (no scales) or 8-bit rows x and w;
         act: none, silu, gelu, or swiglu, where w's rows are gates, then as many ups, and
         act = silu(gate) up.
rotary   rows of k and v go into the paged 4-bit cache (groups of 32 dims, m = lo rounded down and
         s = (hi - m) / 15 rounded up to fp16, c = (x - m) / s rounded), the keys turned on the way: pair
         (j, j + D / 2) of a head by position * theta^(-2 j / D), rounded to bf16 as the cache's keys
         are; the queries of the same rows are turned too.  Positions are the cache's own, or given.
"""
import math
import types

import numpy as np
import torch

own = False

GROUP = 32      # dims of one scale of the cache
PAGE = 64
LEAST = 2.0 ** -100
TOP = 448.0     # the largest e4m3 value


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one token of one request before its MLP (hidden 4096): the latency of a call
        dict(name="norm_single", op="norm", rows=1, cols=4096, norm=True, residual=True, out="e4m3"),
        # one step of 64 requests with 8-node trees
        dict(name="norm_step", op="norm", rows=512, cols=4096, norm=True, residual=True, out="e4m3"),
        # two prompts of 8191 tokens at hidden 8192, for a product in bf16
        dict(name="norm_prompt", op="norm", rows=16382, cols=8192, norm=True, residual=True, out="bf16"),
        # the MLP's inner rows of 32 trees of 65 nodes (inter 14336) before the down projection
        dict(name="norm_inner", op="norm", rows=2080, cols=14336, norm=False, residual=False, out="e4m3"),
        # a single token's output projection and the residual's addition
        dict(name="linear_single", op="linear", rows=1, k=4096, m=4096, kind="e4m3", bias=False, act="none",
             residual=True, out="bf16"),
        # the gate and up projections of one 60-node tree and its root (hidden 4096, inter 11008)
        dict(name="linear_tree", op="linear", rows=61, k=4096, m=11008, kind="e4m3", bias=False, act="swiglu",
             residual=False, out="bf16"),
        # 32 trees of 65 nodes: gate and up projections with inter 14336
        dict(name="linear_groups", op="linear", rows=2080, k=4096, m=14336, kind="e4m3", bias=False,
             act="swiglu", residual=False, out="bf16"),
        # the down projection of a prompt's 8192 tokens, with the residual
        dict(name="linear_prompt", op="linear", rows=8192, k=14336, m=4096, kind="e4m3", bias=False, act="none",
             residual=True, out="bf16"),
        # a decoding head's residual block x + silu(W x + b) over the nodes of 64 small trees
        dict(name="linear_block", op="linear", rows=512, k=4096, m=4096, kind="bf16", bias=True, act="silu",
             residual=True, out="bf16"),
        # odd everything: rows, depth and width that no tile divides, fp32 out
        dict(name="linear_odd", op="linear", rows=77, k=1001, m=777, kind="bf16", bias=True, act="gelu",
             residual=True, out="f32"),
        # one new token of 64 requests: their queries turned, keys and values to the cache
        dict(name="rotary_step", op="rotary", batch=64, heads=32, kv_heads=8, head_dim=128, rows=1, slots=1,
             select=False, len_min=900, len_max=1100, page=64),
        # four prompts' keys, values and queries at once
        dict(name="rotary_fill", op="rotary", batch=4, heads=32, kv_heads=8, head_dim=128, rows=8191,
             slots=8191, select=False, len_min=0, len_max=0, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    most = {op: {"bytes": 0.0, "flops": 0.0} for op in ("norm", "linear", "rotary")}
    for c in listed():
        w = work(c)
        most[c["op"]] = {k: max(v, w[k]) for k, v in most[c["op"]].items()}
    while True:
        op = rng.choice(["norm", "linear", "linear", "rotary"])
        c = dict(op=op)
        if op == "norm":
            c.update(rows=_log(rng, 1, 16384), cols=_log(rng, 64, 16384), norm=rng.random() < 0.75,
                     residual=rng.random() < 0.6, out=rng.choice(["e4m3", "e4m3", "bf16"]))
            c["cols"] = c["cols"] if rng.random() < 0.3 else max(64, c["cols"] // 64 * 64)
            if not c["norm"]:
                c.update(residual=False, out="e4m3")
        elif op == "linear":
            c.update(rows=_log(rng, 1, 8192), k=_log(rng, 64, 14336), m=_log(rng, 64, 14336),
                     kind=rng.choice(["e4m3", "e4m3", "bf16"]), bias=rng.random() < 0.4,
                     act=rng.choice(["none", "silu", "gelu", "swiglu"]), residual=rng.random() < 0.5,
                     out=rng.choice(["bf16", "bf16", "f32"]))
            if rng.random() < 0.7:  # most models' widths; the others are odd
                c.update(k=max(64, c["k"] // 64 * 64), m=max(64, c["m"] // 64 * 64))
        else:
            c.update(batch=_log(rng, 1, 64), kv_heads=rng.choice([1, 2, 4, 8, 32]),
                     head_dim=rng.choice([64, 128, 128, 32, 96]), page=rng.choice([16, 32, 64, 128]),
                     rows=_log(rng, 1, 8191), len_min=0, len_max=_log(rng, 1, 2000), select=rng.random() < 0.3)
            c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 8])
            c["rows"] = min(c["rows"], 65) if c["select"] else c["rows"]
            c["slots"] = rng.randint(1, c["rows"]) if c["select"] else c["rows"]
            if c["heads"] > 64 or c["batch"] * (c["len_max"] + c["slots"]) * c["kv_heads"] * c["head_dim"] > 3e8:
                continue
        w = work(c)
        if w["bytes"] <= most[op]["bytes"] and w["flops"] <= most[op]["flops"]:
            return c


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _gen(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _states(gen, rows, cols):
    """Hidden states as a residual stream holds them: normal, each row at a level of its own, a few
    channels some ten times as large."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    level = torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
    wide = 1 + 19 * (torch.rand(cols, generator=gen, device="cuda") < 0.002).float()
    return x * level * wide


def _padded(t, step):
    """The same values in rows that start a multiple of `step` elements apart."""
    rows, cols = t.shape
    ld = -(-cols // step) * step
    if ld == cols:
        return t
    wide = torch.zeros(rows, ld, dtype=t.dtype, device=t.device)
    wide[:, :cols] = t
    return wide[:, :cols]


def _lengths(case):
    """Cached positions of each request before the call: spread over len_min .. len_max."""
    lo, hi, n = case["len_min"], case["len_max"], case["batch"]
    return [hi if n == 1 else lo + ((i * 7919 + 3) % n) * (hi - lo) // (n - 1) for i in range(n)]


def _counts(case):
    """Rows that the call adds to each request."""
    n, s = case["batch"], case["slots"]
    return [s - (i * 5 % (s if case["select"] else (s + 1) // 2)) for i in range(n)]


def _inputs(case, seed):
    gen, s = _gen(seed), types.SimpleNamespace(case=dict(case))
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    if case["op"] == "norm":
        n, c = case["rows"], case["cols"]
        s.x = _padded(_states(gen, n, c).to(torch.bfloat16), 8)
        s.residual = _padded(_states(gen, n, c).to(torch.bfloat16), 8) if case["residual"] else None
        s.weight = (1 + 0.2 * rand(c)).to(torch.bfloat16) if case["norm"] else None
    elif case["op"] == "linear":
        n, k, m = case["rows"], case["k"], case["m"]
        both = 2 * m if case["act"] == "swiglu" else m
        x, w = _states(gen, n, k), rand(both, k) * (k ** -0.5)
        s.x_scale = s.w_scale = None
        if case["kind"] == "e4m3":
            s.x_scale, s.w_scale = (t.abs().amax(1).div(TOP).clamp(min=LEAST) for t in (x, w))
            x, w = (t.div(sc[:, None]).to(torch.float8_e4m3fn) for t, sc in ((x, s.x_scale), (w, s.w_scale)))
            s.x, s.w = (_padded(t.view(torch.uint8), 16).view(torch.float8_e4m3fn) for t in (x, w))
        else:
            s.x, s.w = (_padded(t.to(torch.bfloat16), 8) for t in (x, w))
        s.bias = (0.2 * rand(both)).to(torch.bfloat16) if case["bias"] else None
        s.residual = _padded(_states(gen, n, m).to(torch.bfloat16), 8) if case["residual"] else None
    else:
        b, n, hk, d, page = (case[k] for k in ("batch", "rows", "kv_heads", "head_dim", "page"))
        s.mp = max(1, -(-(max(_lengths(case)) + case["slots"]) // page))
        s.np = b * s.mp + 3
        s.table = torch.randperm(s.np, generator=gen, device="cuda")[:b * s.mp].reshape(b, s.mp).to(torch.int32)
        s.lengths = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        s.count = torch.tensor(_counts(case), dtype=torch.int32, device="cuda")
        # one projection's rows: queries, keys, values
        qkv = rand(b, n, (case["heads"] + 2 * hk), d)
        qkv[:, :, case["heads"]:] += rand(2 * hk, d)
        qkv = (0.8 * qkv).to(torch.bfloat16)
        s.q, s.k, s.v = qkv.split([case["heads"], hk, hk], 2)
        s.select = s.positions = None
        if case["select"]:
            # the accepted nodes of each tree in ascending order, -1 behind the path, and every node's
            # position: the request's length plus its depth
            pick = torch.rand(b, n, generator=gen, device="cuda")
            pick[:, 0] = -1
            j = torch.arange(case["slots"], device="cuda")
            live = j < s.count[:, None]
            pick = torch.where(live, pick.argsort(1)[:, :case["slots"]], n).sort(1).values
            s.select = torch.where(live, pick, -1).to(torch.int32)
            depth = torch.arange(n, device="cuda") * (0.3 + 0.7 * torch.rand(b, 1, generator=gen, device="cuda"))
            s.positions = (s.lengths[:, None] + depth.long()).to(torch.int32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "linear" and own:
        from eagle_speculative_decoding_draft_gb300 import linear_workspace
        s.workspace = linear_workspace(s.w, case["rows"])
    if case["op"] == "rotary":
        b, hk, d, page = case["batch"], case["kv_heads"], case["head_dim"], case["page"]
        s.k_out = torch.zeros(b, case["slots"], hk, d, dtype=torch.bfloat16, device="cuda")
        s.v_out = torch.zeros_like(s.k_out)
        if own:
            from eagle_speculative_decoding_draft_gb300 import KV4Cache
            s.cache = KV4Cache(batch=b, kv_heads=hk, head_dim=d, num_pages=s.np, max_pages=s.mp, page_size=page,
                               device=torch.device("cuda"))
            s.cache.table.copy_(s.table)
            s.cache.lengths.copy_(s.lengths)
        else:
            s.pool = {}
            for name in ("k", "v"):
                s.pool[name] = (torch.zeros(s.np + 1, page, hk, d // 2, dtype=torch.uint8, device="cuda"),
                                torch.zeros(s.np + 1, page, hk, d // GROUP, 2, dtype=torch.float16, device="cuda"))
    return s


THETA, EPS = 10000.0, 1e-5


# ------------------------------------------------------------------------------------------------
# the plain form
# ------------------------------------------------------------------------------------------------
def _plain_norm(s):
    case = s.case
    h = s.x.float()
    if s.residual is not None:
        h = h + s.residual.float()
    y = h
    if case["norm"]:
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s.weight.float()
    total = h.to(torch.bfloat16) if s.residual is not None else None
    if case["out"] == "bf16":
        return {"y": y.to(torch.bfloat16), "total": total}
    scale = (y.abs().amax(1) / TOP).clamp(min=LEAST)
    return {"y": (y / scale[:, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn), "scale": scale, "total": total}


def _plain_linear(s):
    y = torch.matmul(s.x.float(), s.w.float().t())
    if s.x_scale is not None:
        y = y * (s.x_scale[:, None] * s.w_scale)
    if s.bias is not None:
        y = y + s.bias.float()
    act = s.case["act"]
    if act == "silu":
        y = y / (1 + torch.exp(-y))
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif act == "swiglu":
        g, u = y.chunk(2, 1)
        y = g / (1 + torch.exp(-g)) * u
    if s.residual is not None:
        y = y + s.residual.float()
    return y if s.case["out"] == "f32" else y.to(torch.bfloat16)


def _turn(x, pos):
    """Rows [b][n][heads][d] turned at positions [b][n], in bf16."""
    half = x.shape[-1] // 2
    freq = THETA ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    ang = pos.double()[:, :, None, None] * freq
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    a, c = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * cos - c * sin, c * cos + a * sin], -1).to(torch.bfloat16)


def _half_down(x):
    h = x.half()
    bits = h.view(torch.int16)
    down = torch.where(h > 0, bits - 1, torch.where(h < 0, bits + 1, torch.full_like(bits, -32767)))
    return torch.where(h.float() > x, down.view(torch.float16), h)


def _half_up(x):
    h = x.half()
    return torch.where(h.float() < x, (h.view(torch.int16) + 1).view(torch.float16), h)  # x >= 0


def _quantise(x):
    """Codes [..., d] and parameters (s, m) [..., d / 32, 2] of bf16 rows [..., d]."""
    g = x.float().unflatten(-1, (-1, GROUP))
    m = _half_down(g.amin(-1))
    r = g.amax(-1) - m.float()
    st = _half_up(r / torch.full_like(r, 15.0))
    sf = st.float()[..., None]
    c = torch.where(sf > 0, torch.round((g - m.float()[..., None]) / torch.where(sf > 0, sf, 1.0)), 0.0)
    return c.clamp(0, 15).to(torch.uint8).flatten(-2), torch.stack([st, m], -1)


def _values(packed, par):
    c = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return (par[..., 1:].float() + par[..., :1].float() * c).flatten(-2)


def _plain_rotary(s):
    case, page = s.case, s.case["page"]
    rows = torch.arange(case["rows"], device="cuda")
    pos = s.positions if s.positions is not None else s.lengths[:, None] + rows
    q, k = _turn(s.q, pos), _turn(s.k, pos)
    j = torch.arange(case["slots"], device="cuda")
    live = j < s.count[:, None]
    at_pos = (s.lengths[:, None] + j).long()
    at = torch.where(live, s.table.gather(1, (at_pos // page).clamp(max=s.mp - 1)).long(), s.np)
    out = []
    for name, x in (("k", k), ("v", s.v)):
        if s.select is not None:
            i = s.select.clamp(min=0).long()[:, :, None, None]
            x = x.gather(1, i.expand(-1, -1, *x.shape[2:]))
        codes, par = _quantise(x[:, :case["slots"]])
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
        s.pool[name][0][at, at_pos % page] = codes
        s.pool[name][1][at, at_pos % page] = par
        got = _values(s.pool[name][0][at, at_pos % page], s.pool[name][1][at, at_pos % page])
        out.append(torch.where(live[..., None, None], got, 0.0).to(torch.bfloat16))
    return {"q": q, "k": out[0], "v": out[1], "lengths": s.lengths + s.count}


def run(s):
    case = s.case
    if own:
        import eagle_speculative_decoding_draft_gb300 as gb
        if case["op"] == "norm":
            to = torch.float8_e4m3fn if case["out"] == "e4m3" else torch.bfloat16
            if not case["norm"]:
                y, scale = gb.quantize_rows(s.x)
                return {"y": y, "scale": scale}
            y, scale, total = gb.rms_norm(s.x, s.weight, EPS, residual=s.residual, dtype=to)
            return {"y": y, "total": total} if scale is None else {"y": y, "scale": scale, "total": total}
        if case["op"] == "linear":
            return gb.linear(s.w, s.x, bias=s.bias, act=case["act"], residual=s.residual, w_scale=s.w_scale,
                             x_scale=s.x_scale, dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16,
                             workspace=s.workspace)
        q = s.cache.append_rotary(s.k, s.v, q=s.q, rope_theta=THETA, positions=s.positions, select=s.select,
                                  count=s.count, start=s.lengths)
        s.cache.read(start=s.lengths, out=(s.k_out, s.v_out))
        return {"q": q, "k": s.k_out, "v": s.v_out, "lengths": s.cache.lengths}
    return {"norm": _plain_norm, "linear": _plain_linear, "rotary": _plain_rotary}[case["op"]](s)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "norm":
        n, c = case["rows"], case["cols"]
        each = 2 + (4 if case["residual"] else 0) + (1 if case["out"] == "e4m3" else 2)  # x, residual and sum, y
        return {"bytes": n * c * each + (4 * n if case["out"] == "e4m3" else 0) + (2 * c if case["norm"] else 0),
                "flops": n * c * (8 if case["norm"] else 3)}
    if case["op"] == "linear":
        n, k, m = case["rows"], case["k"], case["m"]
        both = 2 * m if case["act"] == "swiglu" else m
        size = 1 if case["kind"] == "e4m3" else 2
        b = (n + both) * k * size + n * m * (4 if case["out"] == "f32" else 2)
        b += (4 * (n + both) if size == 1 else 0) + (2 * both if case["bias"] else 0) + (2 * n * m if case["residual"] else 0)
        return {"bytes": b, "flops": 2 * n * k * both}
    hk, d = case["kv_heads"], case["head_dim"]
    held = hk * (d // 2 + 4 * (d // GROUP)) * 2  # bytes of a cached token, keys and values
    rows = sum(_counts(case))
    every = case["batch"] * case["rows"] * case["heads"] * d
    # queries in and out; rows in, codes out; codes in, values out
    return {"bytes": 4 * every + rows * (2 * hk * d * 2 + 2 * held + 2 * hk * d * 2), "flops": 3 * every + rows * hk * d * 15}


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def _to_grid(x, bits, least, how):
    """x rounded to a multiple of its step: `bits` bits of mantissa, exponents from `least` on."""
    e = torch.frexp(x).exponent.clamp(min=least + 1).long()  # |x| in [2^(e-1), 2^e)
    step = ((e - 1 - bits + 1023) << 52).view(torch.float64)
    return how(x / step) * step


def _stands_for(x):
    """The values that cached rows of bf16 values stand for."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    low = _to_grid(g.min(-1, keepdim=True).values, 10, -14, torch.floor)
    step = _to_grid((g.max(-1, keepdim=True).values - low) / 15, 10, -14, torch.ceil)
    code = ((g - low) / step).nan_to_num(0.0).round().clamp(0, 15)
    return (low + step * code).reshape(x.shape)


def _turned(x, pos):
    """x [n][heads][d] in 64 bits as complex numbers (x_j + i x_{j + d/2}) times e^(i angle), on bf16's grid."""
    n, heads, d = x.shape
    power = torch.tensor([math.pow(THETA, -2.0 * j / d) for j in range(d // 2)], dtype=torch.float64, device="cuda")
    angle = torch.outer(pos.double(), power)
    z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    return _to_grid(torch.cat([z.real, z.imag], -1), 7, -126, torch.round)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "norm":
        h = s.x.double() + (s.residual.double() if case["residual"] else 0.0)
        y = h
        if case["norm"]:
            y = s.weight.double() * h / (h.pow(2).sum(1, keepdim=True) / case["cols"] + EPS).sqrt()
        out = {"total": h if case["residual"] else None}
        if case["out"] == "bf16":
            return {**out, "y": y}
        scale = torch.maximum(y.abs().max(1).values / TOP, torch.tensor(LEAST, dtype=torch.float64, device="cuda"))
        return {**out, "y": _to_grid(y / scale[:, None], 3, -6, torch.round), "scale": scale}
    if case["op"] == "linear":
        if work(case)["flops"] > 2e12:
            return None
        x, w = s.x.double(), s.w.double()
        if case["kind"] == "e4m3":
            x, w = x * s.x_scale.double()[:, None], w * s.w_scale.double()[:, None]
        z = x @ w.T
        if case["bias"]:
            z = z + s.bias.double()
        if case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        elif case["act"] == "swiglu":
            z = z[:, :case["m"]] * torch.sigmoid(z[:, :case["m"]]) * z[:, case["m"]:]
        return z + s.residual.double() if case["residual"] else z
    b, slots = case["batch"], case["slots"]
    q = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    k, v = (torch.zeros(b, slots, *s.k.shape[2:], dtype=torch.float64, device="cuda") for _ in "kv")
    lens, counts = _lengths(case), _counts(case)
    for i in range(b):
        pos = s.positions[i] if case["select"] else torch.arange(lens[i], lens[i] + case["rows"], device="cuda")
        q[i] = _turned(s.q[i].double(), pos)
        rows = s.select[i, :counts[i]].long() if case["select"] else torch.arange(counts[i], device="cuda")
        k[i, :counts[i]] = _stands_for(_turned(s.k[i].double(), pos)[rows])
        v[i, :counts[i]] = _stands_for(s.v[i, rows].double())
    return {"q": q, "k": k, "v": v, "lengths": torch.tensor(np.add(lens, counts), dtype=torch.int32, device="cuda")}
