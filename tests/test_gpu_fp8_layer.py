"""The draft decoder layer in 8 bits over the 4-bit cache on the GPU: its operators one after the other, as a
caller would call them, and beside the bf16 layer."""
import numpy as np
import pytest
import torch

from decoder_ref import layer, random_tree, tree_mask
from test_gpu_kv4 import gen, i32, make_cache
from test_gpu_rotary import near

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-6


@pytest.fixture(scope="module")
def gb():
    assert torch.cuda.is_available()
    import eagle_speculative_decoding_draft_gb300 as pkg
    return pkg


def build(gb, B, n, h, H, Hk, D, I, P, seed):
    w, d = layer(B=B, n=n, P=max(P, 1), h=h, H=H, Hk=Hk, D=D, I=I, seed=seed, fan_in=True)
    w = {k: v.cuda() for k, v in w.items()}
    names = ("w_qkv", "w_o", "w_norm", "w_gu", "w_d")
    return w, gb.DecoderLayerFP8(*(w[k] for k in names), heads=H, kv_heads=Hk)


def filled(gb, w, B, Hk, D, P, room, seed):
    c = make_cache(B, Hk, D, P + room, 16, seed=seed)
    c.lengths.zero_()
    if P:
        lens = torch.randint(0, P + 1, (B,), generator=gen(seed), device="cuda", dtype=torch.int32)
        c.append(w["k_cache"], w["v_cache"], count=lens)
    return c


def by_hand(gb, w, cache, x, mask, H, Hk, D):
    """The layer as its operators, at position 0, where a rotation leaves everything as it is."""
    B, n, h = x.shape
    q = {k: gb.quantize_rows(w[k]) for k in ("w_qkv", "w_o", "w_gu", "w_d")}

    def product(rows8, name, **kw):
        return gb.linear(q[name][0], rows8[0], w_scale=q[name][1], x_scale=rows8[1], **kw)

    rows = x.reshape(B * n, h)
    qkv = product(gb.quantize_rows(rows), "w_qkv").reshape(B, n, H + 2 * Hk, D)
    qs, ks, vs = qkv.split([H, Hk, Hk], 2)
    o = cache.attention(qs, ks, vs, mask=mask).reshape(B * n, H * D)
    h1 = product(gb.quantize_rows(o), "w_o", residual=rows)
    r, scale, _ = gb.rms_norm(h1, w["w_norm"], EPS, dtype=E4M3)
    a = product((r, scale), "w_gu", act="swiglu")
    return product(gb.quantize_rows(a), "w_d", residual=h1).reshape(B, n, h), ks, vs


SHAPES = [
    # B, n, h, H, Hk, D, I, cached
    (1, 1, 64, 2, 1, 32, 48, 0),
    (3, 1, 512, 8, 2, 64, 1104, 100),
    (4, 4, 256, 4, 4, 128, 512, 40),
    (1, 61, 512, 4, 4, 128, 1376, 200),
    (5, 33, 384, 6, 3, 96, 1024, 70),
    (2, 300, 256, 4, 2, 64, 768, 500),
]


@pytest.mark.parametrize("B,n,h,H,Hk,D,I,P", SHAPES)
@pytest.mark.parametrize("tree", [False, True])
def test_the_layer_is_its_operators(gb, B, n, h, H, Hk, D, I, P, tree):
    w, lay = build(gb, B, n, h, H, Hk, D, I, P, seed=n + h)
    cache = filled(gb, w, B, Hk, D, P, n, seed=1)
    mask = None
    if tree:
        parents, _ = random_tree(n, 8, np.random.default_rng(n))
        mask = torch.from_numpy(tree_mask(parents).view(np.int32)).cuda().expand(B, -1, -1).contiguous()
    out, kn, vn = lay.kv4(w["x"], cache, i32(np.zeros((B, n))), mask=mask, new_kv=True)
    want, ks, vs = by_hand(gb, w, cache, w["x"], mask, H, Hk, D)
    assert torch.equal(kn, ks) and torch.equal(vn, vs)
    assert torch.equal(out, want)
    again = torch.full((lay.workspace_bytes(cache, B, n),), 0xff, dtype=torch.uint8, device="cuda")  # of any content
    assert torch.equal(lay.kv4(w["x"], cache, i32(np.zeros((B, n))), mask=mask, workspace=again), out)
    cache.status()


@pytest.mark.parametrize("B,n,h,H,Hk,D,I,P", SHAPES[1:])
def test_beside_the_bf16_layer(gb, B, n, h, H, Hk, D, I, P):
    """e4m3 rounds by 2^-5 to 2^-4 of a value at most, 0.026 in the mean square, so a product of two rounded
    operands is off by 0.036 of itself.  Keys, queries and values off by that move the attention's output by at
    most 0.09 with the output projection's own error; both factors of silu(g) u carry that and their own, the
    down projection adds 0.036: under a quarter of what the layer adds to x."""
    from eagle_speculative_decoding_draft_gb300.engine import DecoderLayer
    w, lay = build(gb, B, n, h, H, Hk, D, I, P, seed=7 + n)
    cache = filled(gb, w, B, Hk, D, P, n, seed=2)
    plain = DecoderLayer(*(w[k] for k in ("w_qkv", "w_o", "w_norm", "w_gu", "w_d")), heads=H, kv_heads=Hk)
    pos = cache.lengths[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
    got, kn, vn = lay.kv4(w["x"], cache, pos, new_kv=True)
    want = plain.kv4(w["x"], cache, pos)
    adds = (want.double() - w["x"].double()).norm()
    assert (got.double() - want.double()).norm() <= 0.25 * adds
    # the new keys are the projection's, turned
    q8, s8 = gb.quantize_rows(w["x"].reshape(B * n, h))
    wq, ws = gb.quantize_rows(w["w_qkv"])
    ks = gb.linear(wq, q8, w_scale=ws, x_scale=s8).reshape(B, n, H + 2 * Hk, D)[:, :, H:H + Hk]
    near(kn, ks, pos, 10000.0)
    cache.status()


def test_rounds_of_drafting_as_a_graph(gb):
    """Each round: the layer over the tree, the accepted nodes into the cache; captured once."""
    B, n, h, H, Hk, D, I = 3, 7, 256, 4, 2, 64, 512
    w, lay = build(gb, B, n, h, H, Hk, D, I, 30, seed=3)
    a, b = (filled(gb, w, B, Hk, D, 30, 64, seed=5) for _ in range(2))
    parents, depths = random_tree(n, 4, np.random.default_rng(4))
    mask = torch.from_numpy(tree_mask(parents).view(np.int32)).cuda().expand(B, -1, -1).contiguous()
    x, depth, sel = torch.empty_like(w["x"]), i32(depths), i32([[0, 2, -1], [0, -1, -1], [0, 1, 3]])
    cnt = i32([2, 1, 3])

    def step(c, ws=None):
        out, kn, vn = lay.kv4(x, c, c.lengths[:, None] + depth, mask=mask, new_kv=True, workspace=ws)
        c.append(kn, vn, select=sel, count=cnt)
        return out

    x.copy_(w["x"])
    start = b.lengths.clone()
    step(b), b.lengths.copy_(start)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(a)
    for i in range(6):
        x.copy_(torch.randn(x.shape, generator=gen(i), device="cuda"))
        graph.replay()
        assert torch.equal(out, step(b)), i
    assert torch.equal(a.lengths, b.lengths)
    a.status(), b.status()


def test_refusals_of_the_binding(gb):
    w, lay = build(gb, 2, 3, 64, 4, 2, 32, 48, 4, seed=0)
    c = make_cache(2, 2, 32, 32, 16)
    pos = i32(np.zeros((2, 3)))
    for kw, error in [(dict(x=w["x"][:1]), ValueError), (dict(x=w["x"].float()), TypeError), (dict(positions=pos[:, :2].contiguous()), ValueError),
                      (dict(mask=i32(np.zeros((2, 3, 2)))), ValueError), (dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")), ValueError),
                      (dict(out=torch.empty(2, 3, 32, dtype=BF16, device="cuda")), ValueError), (dict(cache=make_cache(2, 4, 32, 32, 16)), ValueError)]:
        with pytest.raises(error):
            lay.kv4(**{**dict(x=w["x"], cache=c, positions=pos), **kw})
    with pytest.raises(ValueError):
        gb.DecoderLayerFP8(w["w_qkv"], w["w_o"], w["w_norm"], w["w_gu"][:80], w["w_d"][:, :40].contiguous(), heads=4, kv_heads=2)


def test_a_new_layer_is_ready_on_any_stream(gb):
    """Constructed behind a queue of other work and called at once on another stream."""
    B, n, h, H, Hk, D, I = 2, 9, 256, 4, 2, 64, 512
    w, want_layer = build(gb, B, n, h, H, Hk, D, I, 20, 3)
    c = filled(gb, w, B, Hk, D, 20, n, 3)
    pos = c.lengths[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
    want = want_layer.kv4(w["x"], c, pos)
    names = ("w_qkv", "w_o", "w_norm", "w_gu", "w_d")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        trash = [torch.full((1 << 20,), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(8)]  # what the codes' memory holds
        del trash
        torch.cuda._sleep(100_000_000)
        made = gb.DecoderLayerFP8(*(w[k] for k in names), heads=H, kv_heads=Hk)
        got = made.kv4(w["x"], c, pos, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        torch.cuda.synchronize()
    c.status()
