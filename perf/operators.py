"""The 4-bit key/value cache of the draft engine as work to be measured: writing it, reading it back
and attending over it.

The cache.  Keys and values of a token are held per kv head in groups of 32 neighbouring head
dimensions.  With lo and hi the least and largest value of a group,
    m = lo rounded down to fp16,  s = (hi - m) / 15 rounded up to fp16,
    c = (x - m) / s rounded to the nearest whole number (ties to even) in 0..15  (0 where s = 0),
and the group stands for the values m + s c: 4 bits a value and 32 bits a group.  Tokens lie in pages
of `page` positions; table[b][i] names the page of positions i * page .. i * page + page - 1 of
request b, and lengths[b] says how many positions hold tokens.

write   rows of k and v go to positions start[b], start[b] + 1, ...: all rows in order, or the rows
        that `select` names (the accepted nodes of a verified tree); the lengths follow.
read    positions start[b] .. of every request, as the values that their codes stand for.
attend  o = softmax(q k^T / sqrt(head_dim)) v over the cached positions of the request and the new
        keys of its nodes: those that the node's mask row marks (a draft tree), or the node's own
        and the earlier ones (a prompt's next piece, a single token).  Query head h reads kv head
        h // (heads / kv_heads).
"""
import math
import types

import numpy as np
import torch

own = False

GROUP = 32


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # the smallest write: one decoding step of the engine's largest batch (64 requests, 32 kv
        # heads of 128); the nodes of the accepted paths, 1 to 6 of each 8-node tree, join the cache
        dict(name="write_step", op="write", batch=64, kv_heads=32, head_dim=128, page=64, rows=8,
             slots=6, select=True, len_min=900, len_max=1100, out="bf16"),
        # prompts of four requests, of different lengths, written at once
        dict(name="write_prompt", op="write", batch=4, kv_heads=8, head_dim=128, page=64, rows=8191,
             slots=8191, select=False, len_min=0, len_max=0, out="bf16"),
        # odd everything: head_dim 96, small pages, starts inside a page
        dict(name="write_odd", op="write", batch=7, kv_heads=3, head_dim=96, page=16, rows=301,
             slots=301, select=False, len_min=1, len_max=499, out="bf16"),
        # a ragged batch read back for a model that wants bf16 keys and values
        dict(name="read_ragged", op="read", batch=32, kv_heads=8, head_dim=128, page=64, len_min=1,
             len_max=2047, out="bf16"),
        # one long request read back in fp32
        dict(name="read_long", op="read", batch=1, kv_heads=8, head_dim=128, page=64, len_min=65536,
             len_max=65536, out="f32"),
        # one token of one request: the latency of a call (Llama-2-7B heads)
        dict(name="attend_single", op="attend", batch=1, heads=32, kv_heads=32, head_dim=128, page=64,
             nodes=1, mask="causal", len_min=1024, len_max=1024),
        # one draft tree over a 1024-token cache (the Vicuna-7B shape: 60 drafted nodes and the root)
        dict(name="attend_tree", op="attend", batch=1, heads=32, kv_heads=32, head_dim=128, page=64,
             nodes=61, mask="tree", len_min=1024, len_max=1024),
        # the largest batch of small trees (64 requests of 8 nodes, Llama-2-7B heads)
        dict(name="attend_step", op="attend", batch=64, heads=32, kv_heads=32, head_dim=128, page=64,
             nodes=8, mask="tree", len_min=1024, len_max=1024),
        # large trees under grouped heads (the Llama-3-8B shape: 32 requests of 65 nodes)
        dict(name="attend_groups", op="attend", batch=32, heads=32, kv_heads=8, head_dim=128, page=64,
             nodes=65, mask="tree", len_min=1024, len_max=1024),
        # single tokens of requests between short and very long, small pages (Llama-2-70B heads)
        dict(name="attend_ragged", op="attend", batch=16, heads=64, kv_heads=8, head_dim=128, page=16,
             nodes=1, mask="causal", len_min=1, len_max=65536),
        # odd sizes: head_dim 64, groups of 3, seven nodes, lengths from nothing to a few thousand
        dict(name="attend_odd", op="attend", batch=5, heads=12, kv_heads=4, head_dim=64, page=32,
             nodes=7, mask="tree", len_min=0, len_max=3001),
        # the next 2047 tokens of two prompts over what is cached of them
        dict(name="attend_prompt", op="attend", batch=2, heads=64, kv_heads=8, head_dim=128, page=64,
             nodes=2047, mask="causal", len_min=4000, len_max=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    most = {"bytes": 0.0, "flops": 0.0}
    for c in listed():
        w = work(c)
        most = {k: max(most[k], w[k]) for k in most}
    while True:
        op = rng.choice(["write", "read", "attend", "attend"])
        c = dict(op=op, kv_heads=rng.choice([1, 2, 4, 8, 32]), head_dim=rng.choice([64, 128, 128, 32, 96]),
                 page=rng.choice([16, 32, 64, 128]))
        if op == "write":
            c.update(batch=_log(rng, 1, 64), rows=_log(rng, 1, 8191), len_min=0, len_max=_log(rng, 1, 2000),
                     select=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
            c["rows"] = min(c["rows"], 65) if c["select"] else c["rows"]
            c["slots"] = rng.randint(1, c["rows"]) if c["select"] else c["rows"]
        elif op == "read":
            c.update(batch=_log(rng, 1, 64), len_max=_log(rng, 1, 65536), out=rng.choice(["bf16", "f32"]))
            c["len_min"] = rng.randint(0, c["len_max"])
        else:
            c.update(batch=_log(rng, 1, 64), heads=c["kv_heads"] * rng.choice([1, 2, 3, 4, 8]),
                     nodes=_log(rng, 1, 2047), mask=rng.choice(["tree", "causal"]),
                     len_max=_log(rng, 1, 65536))
            c["len_min"] = rng.randint(0, c["len_max"])
            c["nodes"] = min(c["nodes"], 300) if c["mask"] == "tree" else c["nodes"]
            if c["heads"] > 64:
                continue
            # the plain form lays out fp32 keys, values and scores
            kv = 3 * 4 * c["batch"] * (c["len_max"] + c["nodes"]) * c["kv_heads"] * c["head_dim"]
            sc = 4 * 4 * c["batch"] * c["heads"] * c["nodes"] * (c["len_max"] + c["nodes"])
            if kv + sc > 30e9:
                continue
        cap = c["batch"] * (c["len_max"] + c.get("rows", 0)) * c["kv_heads"] * c["head_dim"]
        if cap > 1.2e9:
            continue
        w = work(c)
        if w["bytes"] <= 0.5 * most["bytes"] and w["flops"] <= most["flops"]:
            return c


def _lengths(case):
    """Cached positions of each request: spread over len_min .. len_max, the same for every seed."""
    lo, hi = case["len_min"], case["len_max"]
    n = case["batch"]
    return [hi if n == 1 else lo + ((i * 7919 + 3) % n) * (hi - lo) // (n - 1) for i in range(n)]


def _counts(case):
    """Rows that a write adds to each request."""
    n, s = case["batch"], case["slots"]
    return [s - (i * 5 % (s if case["select"] else (s + 1) // 2)) for i in range(n)]


def _pages_a_request(case):
    most = max(_lengths(case)) + (case["slots"] if case["op"] == "write" else 0)
    return max(1, -(-most // case["page"]))


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _kv(gen, *shape):
    """Keys or values as projections give them: normal, some channels with an offset of their own,
    a few ten times as large."""
    x = torch.randn(*shape, generator=gen, device="cuda")
    heads, dim = shape[-2:]
    at = torch.randn(heads, dim, generator=gen, device="cuda")
    wide = 1 + 9 * (torch.rand(heads, dim, generator=gen, device="cuda") < 0.01).float()
    return (0.8 * (x + at) * wide).to(torch.bfloat16)


def _tree_masks(case, seed):
    """Ancestor masks of one random draft tree a request: bit j of row i is set where node j is i or
    an ancestor of i, 32 nodes a word."""
    rng = np.random.default_rng(seed)
    b, n = case["batch"], case["nodes"]
    see = np.zeros((b, n, n), dtype=bool)
    for i in range(n):
        if i:
            parent = rng.integers(max(0, i - 10), i, size=b)
            see[:, i] = see[np.arange(b), parent]
        see[:, i, i] = True
    words = -(-n // 32)
    bits = np.zeros((b, n, words * 32), dtype=np.uint32)
    bits[:, :, :n] = see
    packed = (bits.reshape(b, n, words, 32) << np.arange(32, dtype=np.uint32)).sum(-1, dtype=np.uint32)
    return torch.from_numpy(packed.view(np.int32)).cuda()


def _inputs(case, seed):
    """The seed's tensors: what both forms and the exact values start from."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = types.SimpleNamespace(case=dict(case))
    b, hk, d, page = case["batch"], case["kv_heads"], case["head_dim"], case["page"]
    s.mp = _pages_a_request(case)
    s.np = b * s.mp + 3
    s.table = torch.randperm(s.np, generator=gen, device="cuda")[:b * s.mp].reshape(b, s.mp).to(torch.int32)
    s.lengths = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if case["op"] == "write":
        s.k, s.v = _kv(gen, b, case["rows"], hk, d), _kv(gen, b, case["rows"], hk, d)
        s.count = torch.tensor(_counts(case), dtype=torch.int32, device="cuda")
        s.select = None
        if case["select"]:  # node 0, then other nodes in ascending order; -1 behind the path
            pick = torch.rand(b, case["rows"], generator=gen, device="cuda")
            pick[:, 0] = -1
            pick = pick.argsort(1)[:, :case["slots"]]
            j = torch.arange(case["slots"], device="cuda")
            pick = torch.where(j < s.count[:, None], pick, case["rows"]).sort(1).values
            s.select = torch.where(j < s.count[:, None], pick, -1).to(torch.int32)
    else:
        s.kc, s.vc = _kv(gen, b, s.mp * page, hk, d), _kv(gen, b, s.mp * page, hk, d)
    if case["op"] == "attend":
        n = case["nodes"]
        s.q = (1.5 * torch.randn(b, n, case["heads"], d, generator=gen, device="cuda")).to(torch.bfloat16)
        s.kn, s.vn = _kv(gen, b, n, hk, d), _kv(gen, b, n, hk, d)
        s.mask = _tree_masks(case, seed) if case["mask"] == "tree" else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    b, hk, d, page = case["batch"], case["kv_heads"], case["head_dim"], case["page"]
    out = {"bf16": torch.bfloat16, "f32": torch.float32, None: None}[case.get("out")]
    if case["op"] != "attend":
        rows = case["slots"] if case["op"] == "write" else max(_lengths(case))
        s.k_out = torch.zeros(b, rows, hk, d, dtype=out, device="cuda")
        s.v_out = torch.zeros_like(s.k_out)
    if own:
        from eagle_speculative_decoding_draft_gb300 import KV4Cache
        s.cache = KV4Cache(batch=b, kv_heads=hk, head_dim=d, num_pages=s.np, max_pages=s.mp, page_size=page,
                           device=torch.device("cuda"))
        s.cache.table.copy_(s.table)
        if case["op"] != "write":
            s.cache.append(s.kc, s.vc)
        s.cache.lengths.copy_(s.lengths)
    else:
        s.pool = {}
        for name in ("k", "v"):
            s.pool[name] = (torch.zeros(s.np + 1, page, hk, d // 2, dtype=torch.uint8, device="cuda"),
                            torch.zeros(s.np + 1, page, hk, d // GROUP, 2, dtype=torch.float16, device="cuda"))
        if case["op"] != "write":
            for name, x in (("k", s.kc), ("v", s.vc)):
                codes, par = _quantise(x)
                at = s.table.long()
                s.pool[name][0][at] = _pack(codes).reshape(b, s.mp, page, hk, d // 2)
                s.pool[name][1][at] = par.reshape(b, s.mp, page, hk, d // GROUP, 2)
    if case["op"] != "write":
        del s.kc, s.vc
    return s


# ------------------------------------------------------------------------------------------------
# the plain form
# ------------------------------------------------------------------------------------------------
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
    s = _half_up(r / torch.full_like(r, 15.0))  # by a tensor: by a number it would be a product with 1 / 15
    sf = s.float()[..., None]
    c = torch.where(sf > 0, torch.round((g - m.float()[..., None]) / torch.where(sf > 0, sf, 1.0)), 0.0)
    return c.clamp(0, 15).to(torch.uint8).flatten(-2), torch.stack([s, m], -1)


def _pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _values(packed, par):
    """What codes and parameters stand for, in fp32."""
    c = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return (par[..., 1:].float() + par[..., :1].float() * c).flatten(-2)


def _cached(s, name):
    """All positions of every request's pages, in fp32: [b][mp * page][hk][d]."""
    at = s.table.long()
    return _values(s.pool[name][0][at], s.pool[name][1][at]).flatten(1, 2)


def _plain_write(s):
    case, page = s.case, s.case["page"]
    j = torch.arange(case["slots"], device="cuda")
    live = j < s.count[:, None]
    pos = (s.lengths[:, None] + j).long()
    at = torch.where(live, s.table.gather(1, (pos // page).clamp(max=s.mp - 1)).long(), s.np)
    out = []
    for name, x in (("k", s.k), ("v", s.v)):
        if s.select is not None:
            i = s.select.clamp(min=0).long()[:, :, None, None]
            x = x.gather(1, i.expand(-1, -1, *x.shape[2:]))
        codes, par = _quantise(x[:, :case["slots"]])
        codes = _pack(codes)
        s.pool[name][0][at, pos % page] = codes
        s.pool[name][1][at, pos % page] = par
        out.append(torch.where(live[..., None, None], _values(codes, par), 0.0).to(s.k_out.dtype))
    return out[0], out[1], s.lengths + s.count


def _plain_read(s):
    rows = s.k_out.shape[1]
    live = (torch.arange(rows, device="cuda") < s.lengths[:, None])[..., None, None]
    return tuple(torch.where(live, _cached(s, name)[:, :rows], 0.0).to(s.k_out.dtype) for name in ("k", "v"))


def _sees(s, keys):
    """[b][n][keys]: which cached positions and new keys each node attends to."""
    b, n = s.q.shape[:2]
    t = torch.arange(keys - n, device="cuda")
    old = (t < s.lengths[:, None])[:, None].expand(b, n, keys - n)
    i = torch.arange(n, device="cuda")
    if s.mask is None:
        new = (i <= i[:, None]).expand(b, n, n)
    else:
        new = ((s.mask[:, :, i // 32] >> (i % 32)) & 1).bool()
    return torch.cat([old, new], -1)


def _plain_attend(s):
    b, n, h, d = s.q.shape
    hk = s.kn.shape[2]
    k = torch.cat([_cached(s, "k"), s.kn.float()], 1).permute(0, 2, 3, 1)
    v = torch.cat([_cached(s, "v"), s.vn.float()], 1).permute(0, 2, 1, 3)
    see = _sees(s, k.shape[-1])
    q = s.q.float().reshape(b, n, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    x = torch.matmul(q / math.sqrt(d), k).reshape(b, hk, h // hk, n, -1)
    x = x.masked_fill_(~see[:, None, None], -math.inf)
    p = (x - x.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).reshape(b, hk, h // hk, n, d)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, h, d).to(torch.bfloat16)


def run(s):
    op = s.case["op"]
    if own:
        if op == "write":
            s.cache.append(s.k, s.v, select=s.select, count=s.count, start=s.lengths)
            s.cache.read(start=s.lengths, out=(s.k_out, s.v_out))
            return s.k_out, s.v_out, s.cache.lengths
        if op == "read":
            return s.cache.read(out=(s.k_out, s.v_out))
        return s.cache.attention(s.q, s.kn, s.vn, mask=s.mask)
    if op == "write":
        return _plain_write(s)
    return _plain_read(s) if op == "read" else _plain_attend(s)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    b, hk, d = case["batch"], case["kv_heads"], case["head_dim"]
    held = hk * (d // 2 + 4 * (d // GROUP)) * 2  # bytes of a cached token, keys and values
    if case["op"] == "write":  # the rows in, the codes out; the codes in and their values out
        rows = sum(_counts(case))
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": rows * (hk * d * 2 * 2 + 2 * held + hk * d * 2 * size), "flops": rows * hk * d * 2 * 6}
    tokens = sum(_lengths(case))
    if case["op"] == "read":
        return {"bytes": tokens * (held + hk * d * 2 * (2 if case["out"] == "bf16" else 4)), "flops": tokens * hk * d * 4}
    n, h = case["nodes"], case["heads"]
    new = n * n if case["mask"] == "tree" else n * (n + 1) // 2
    pairs = n * tokens + b * new
    words = b * n * -(-n // 32) * 4 if case["mask"] == "tree" else 0
    return {"bytes": tokens * held + 2 * b * n * hk * d * 2 + 2 * b * n * h * d * 2 + words, "flops": 4 * h * d * pairs}


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def _to_half_grid(x, up):
    """x rounded to a multiple of its fp16 step, down or up."""
    e = torch.frexp(x).exponent.clamp(min=-13).long()  # |x| in [2^(e-1), 2^e)
    step = ((e - 11 + 1023) << 52).view(torch.float64)  # 2^(e - 11)
    return (torch.ceil(x / step) if up else torch.floor(x / step)) * step


def _stands_for(x):
    """The values that a cached bf16 row stands for, in 64 bits."""
    groups = x.double().reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    low = _to_half_grid(groups.min(-1, keepdim=True).values, up=False)
    step = _to_half_grid((groups.max(-1, keepdim=True).values - low) / 15, up=True)
    code = ((groups - low) / step).nan_to_num(0.0).round().clamp(0, 15)
    return (low + step * code).reshape(x.shape)


def exact(case, seed):
    s = _inputs(case, seed)
    lens = _lengths(case)
    if case["op"] == "write":
        kind = {"k": s.k, "v": s.v}
        out = [torch.zeros(case["batch"], case["slots"], *s.k.shape[2:], dtype=torch.float64, device="cuda") for _ in kind]
        for o, x in zip(out, kind.values()):
            for b, count in enumerate(_counts(case)):
                rows = s.select[b, :count].long() if case["select"] else torch.arange(count, device="cuda")
                o[b, :count] = _stands_for(x[b, rows])
        return out[0], out[1], s.lengths + s.count
    if case["op"] == "read":
        out = [torch.zeros(case["batch"], max(lens), *s.kc.shape[2:], dtype=torch.float64, device="cuda") for _ in "kv"]
        for o, x in zip(out, (s.kc, s.vc)):
            for b, t in enumerate(lens):
                o[b, :t] = _stands_for(x[b, :t])
        return tuple(out)
    if work(case)["flops"] > 2e12:
        return None
    b, n, h, d = s.q.shape
    hk = case["kv_heads"]
    out = torch.zeros(b, n, h, d, dtype=torch.float64, device="cuda")
    for i, t in enumerate(lens):
        keys = torch.cat([_stands_for(s.kc[i, :t]), s.kn[i].double()])
        values = torch.cat([_stands_for(s.vc[i, :t]), s.vn[i].double()])
        allowed = torch.ones(n, t + n, dtype=torch.bool, device="cuda")
        if s.mask is None:
            allowed[:, t:] = torch.ones(n, n, device="cuda").tril().bool()
        else:
            for j in range(n):
                allowed[:, t + j] = (s.mask[i, :, j // 32].long() >> (j % 32)) % 2 == 1
        for head in range(h):
            kv = head // (h // hk)
            z = s.q[i, :, head].double() @ keys[:, kv].T * d ** -0.5
            z = torch.where(allowed, z, torch.full_like(z, -math.inf))
            out[i, :, head] = torch.softmax(z, -1) @ values[:, kv]
    return out
