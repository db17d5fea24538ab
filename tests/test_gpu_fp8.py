"""The norm that ends in 8 bits, rows quantised, and the product with its epilogue on the GPU, against
their formulas in 64 bits (fp8_ref.py, which derives the tolerances)."""
import math

import pytest
import torch

import fp8_ref as ref

pytestmark = pytest.mark.gpu

BF16, E4M3, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32


@pytest.fixture(scope="module")
def gb():
    assert torch.cuda.is_available()
    import eagle_speculative_decoding_draft_gb300 as pkg
    return pkg


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def wide(g, rows, cols, ld, scale=1.0, dtype=BF16):
    """A [rows][cols] view of wider rows whose rest is NaN: nothing may depend on it."""
    t = torch.full((rows, ld), math.nan, device="cuda").to(dtype)
    t[:, :cols] = (scale * torch.randn(rows, cols, generator=g, device="cuda")).to(dtype)
    return t[:, :cols]


def up(n, step):
    return -(-n // step) * step


# ------------------------------------------------------------------------------------------------
# rows
# ------------------------------------------------------------------------------------------------
ROWS = [(1, 1), (3, 7), (5, 8), (1, 64), (9, 100), (2, 257), (4, 1000), (130, 1024), (7, 1025), (513, 1536), (600, 4096),
        (1, 4096), (2, 8200), (3, 11008), (520, 8192), (1, 16384), (2, 16385), (3, 28672), (1, 32768)]
SUM = 40 * 2.0 ** -24  # a row's sum of squares: 64 additions a thread at most, ten steps after; halved by the root


@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(gb, rows, cols, residual):
    g = gen(rows + cols)
    x = wide(g, rows, cols, up(cols, 8) + 8 * (cols % 3), 3.0)
    r = wide(g, rows, cols, up(cols, 8), 2.0) if residual else None
    w = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(BF16)
    y, h = ref.norm(x, w, 1e-5, r)
    got, scale, total = gb.rms_norm(x, w, 1e-5, residual=r)
    assert scale is None and got.dtype is BF16
    assert ((got.double() - y).abs() <= ref.HALF_BF16 * y.abs() * (1 + SUM) + SUM * y.abs()).all()
    if residual:
        assert ((total.double() - h).abs() <= ref.HALF_BF16 * h.abs() + 2.0 ** -23 * (x.double().abs() + r.double().abs())).all()
    else:
        assert total is None
    codes, scale, total8 = gb.rms_norm(x, w, 1e-5, residual=r, dtype=E4M3)
    ref.check_rows8(codes, scale, y, SUM)
    if residual:
        assert torch.equal(total8, total)


@pytest.mark.parametrize("rows,cols", ROWS)
def test_quantize_rows(gb, rows, cols):
    x = wide(gen(rows * cols), rows, cols, up(cols, 8) + 8, 5.0)
    codes, scale = gb.quantize_rows(x)
    want = (x.float().abs().amax(1) / torch.full((rows,), 448.0, device="cuda")).clamp(min=ref.LEAST)
    assert torch.equal(scale, want)
    # the quotient in fp32, then the nearest e4m3 value: ties are decided by the quotient's last bit
    q, _ = ref.e4m3((x.float() / scale[:, None]).double())
    assert torch.equal(codes.double(), q)


def test_quantize_rows_ties_zeros_and_extremes(gb):
    x = torch.zeros(7, 24, device="cuda")
    x[1] = torch.tensor([448.0, 432, 440, 1.0625, 1.1875, -1.0625, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, -17, 27], device="cuda").repeat(2)
    x[2] = 2.0 ** -120          # below the least scale
    x[3, 3] = 1e38
    x[3, 4] = -3e38
    x[4] = torch.linspace(-1, 1, 24, device="cuda")
    x[4, 7] = math.nan
    x[5, 0] = math.inf
    x[6, 5] = -1e-35
    codes, scale = gb.quantize_rows(x.to(BF16))
    xd = x.to(BF16).float()
    for i in (0, 1, 2, 3, 6):
        want = max(float(torch.tensor(float(xd[i].abs().max()) / 448.0, dtype=F32)), ref.LEAST)
        assert float(scale[i]) == want, i
        q, _ = ref.e4m3((xd[i] / scale[i]).double())
        assert torch.equal(codes[i].double(), q), i
    for i in (4, 5):
        assert math.isnan(float(scale[i])) and torch.isnan(codes[i].float()).all()


def test_norm_of_rows_that_hold_nan_infinity_or_nothing(gb):
    x = torch.randn(5, 64, generator=gen(1), device="cuda").to(BF16)
    x[1, 3], x[2, 3], x[3] = math.nan, math.inf, 0.0
    w = torch.ones(64, device="cuda", dtype=BF16)
    codes, scale, _ = gb.rms_norm(x, w, 1e-5, dtype=E4M3)
    y, _, _ = gb.rms_norm(x, w, 1e-5)
    assert torch.isnan(scale[1:3]).all() and torch.isnan(codes[1:3].float()).all()
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 3])
    assert (codes[3].float() == 0).all() and float(scale[3]) == ref.LEAST and (y[3] == 0).all()
    alone, alone_scale, _ = gb.rms_norm(x[4:], w, 1e-5, dtype=E4M3)  # its neighbours have no influence
    assert torch.equal(alone.float(), codes[4:].float()) and torch.equal(alone_scale, scale[4:])


@pytest.mark.parametrize("rows,cols", [(3, 100), (5, 4096), (600, 4100)])
def test_rows_leave_what_lies_between_them(gb, rows, cols):
    """Outputs in wider rows, through the C ABI: the rest and a row behind the last keep what they hold; the
    sum may take the residual's place."""
    from eagle_speculative_decoding_draft_gb300 import _lib
    lib, g = _lib.load(), gen(3)
    x, r = wide(g, rows, cols, up(cols, 8)), wide(g, rows, cols, up(cols, 8) + 8)
    w = torch.ones(cols, device="cuda", dtype=BF16)
    want, scale, total = gb.rms_norm(x, w, 1e-5, residual=r, dtype=E4M3)
    ld = up(cols, 16) + 16
    y = torch.full((rows + 1, ld), 0x5a, dtype=torch.uint8, device="cuda")
    s = torch.full((rows + 1,), -1.0, device="cuda")
    assert lib.eagle_rms_norm(x.data_ptr(), x.stride(0), r.data_ptr(), r.stride(0), w.data_ptr(), 1e-5, rows, cols, r.data_ptr(),
                              r.stride(0), 2, y.data_ptr(), ld, s.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(y[:rows, :cols], want.view(torch.uint8)) and torch.equal(s[:rows], scale) and torch.equal(r, total)
    assert (y[:rows, cols:] == 0x5a).all() and (y[rows] == 0x5a).all() and float(s[rows]) == -1


# ------------------------------------------------------------------------------------------------
# products
# ------------------------------------------------------------------------------------------------
def operands(g, rows, M, K, kind, act, bias, residual, gb, pad=0):
    both = 2 * M if act == "swiglu" else M
    step = 16 if kind is E4M3 else 8
    x = wide(g, rows, K, up(K, 8) + 8 * pad, 2.0)
    w = wide(g, both, K, up(K, 8) + 8 * pad, K ** -0.5)
    w_scale = x_scale = None
    if kind is E4M3:
        (x, x_scale), (w, w_scale) = gb.quantize_rows(x), gb.quantize_rows(w)
        if K % step:  # what lies between the rows has no influence
            for t in (x, w):
                torch.as_strided(t.view(torch.uint8), (t.shape[0] - 1, t.stride(0) - K), (t.stride(0), 1), K).fill_(0x7f)
    b = (0.5 * torch.randn(both, generator=g, device="cuda")).to(BF16) if bias else None
    r = wide(g, rows, M, up(M, 8)) if residual else None
    return w, x, b, r, w_scale, x_scale


SHAPES = [
    # rows, M, K: up to 16 rows, up to 128 with K in 1 to 8 parts, more in chunks of 128, whole tiles of one pair or two;
    # odd everything
    (1, 4096, 4096), (1, 128, 64), (2, 1, 8), (7, 777, 1001), (15, 130, 72), (16, 2048, 8192), (16, 40000, 128),
    (17, 128, 4096), (31, 256, 8192), (33, 777, 1000), (61, 1000, 4096), (64, 8192, 512), (77, 777, 1001), (100, 64, 16),
    (255, 512, 520), (256, 4096, 1024), (257, 384, 2048), (300, 100, 333), (129, 700, 4097), (150, 300, 8192), (400, 4100, 1100), (1500, 4096, 256), (600, 2500, 640), (2080, 1024, 4096),
]
ACTS = [(None, False, False), ("silu", True, True), ("gelu", True, False), ("swiglu", False, True), (None, True, True), ("swiglu", True, False)]


@pytest.mark.parametrize("rows,M,K", SHAPES)
@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_linear(gb, rows, M, K, kind):
    g = gen(rows * 7 + M + K)
    for i, (act, bias, residual) in enumerate(ACTS):
        w, x, b, r, w_scale, x_scale = operands(g, rows, M, K, kind, act, bias, residual, gb, pad=i % 2)
        for dtype in (BF16, F32):
            y, tol = ref.linear(w, x, b, act, r, w_scale, x_scale, dtype)
            got = gb.linear(w, x, bias=b, act=act, residual=r, w_scale=w_scale, x_scale=x_scale, dtype=dtype)
            assert got.shape == (rows, M) and got.dtype is dtype
            off = (got.double() - y).abs() - tol
            assert (off <= 0).all(), (act, dtype, float(off.max()), int((off > 0).sum()))
            again = gb.linear(w, x, bias=b, act=act, residual=r, w_scale=w_scale, x_scale=x_scale, dtype=dtype)
            assert torch.equal(again, got)


@pytest.mark.parametrize("rows,M,K", [(300, 520, 16500), (1100, 5000, 4200), (700, 1300, 14336), (512, 4096, 9000), (512, 2048, 9000), (100, 300, 40000), (100, 20000, 4200)])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_long_sums_of_bf16_products_for_fp32_outputs(gb, rows, M, K, act):
    """Over 128 rows 2048 products at a time are summed by the tensor core, which adds 16 to what it has and
    truncates: 128 additions lose 2^-24 of the sum so far on average, 7.6e-6 of a segment's at most."""
    w, x, b, r, _, _ = operands(gen(K), rows, M, K, BF16, act, True, True, gb)
    y, tol = ref.linear(w, x, b, act, r, None, None, F32)
    got = gb.linear(w, x, bias=b, act=act, residual=r, dtype=F32)
    assert ((got.double() - y).abs() <= tol).all()
    if rows > 128 and act is None:
        z, _ = ref.linear(w, x, None, None, None, None, None, F32)
        assert (gb.linear(w, x, dtype=F32).double() - z).norm() <= 7.6e-6 * z.norm()
    assert torch.equal(gb.linear(w, x, bias=b, act=act, residual=r, dtype=F32), got)


@pytest.mark.parametrize("rows", [1, 16, 40, 300])
@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_linear_outputs_of_any_alignment_and_in_place_of_the_residual(gb, rows, kind, act):
    """Rows of Y that no bulk store can take, guard values around them, and Y in the residual's memory."""
    M, K, g = 200, 1100, gen(rows)
    w, x, b, r, w_scale, x_scale = operands(g, rows, M, K, kind, act, True, True, gb)
    want = gb.linear(w, x, bias=b, act=act, residual=r, w_scale=w_scale, x_scale=x_scale)
    ws = gb.linear_workspace(w, rows)
    for dtype in (BF16, F32):
        y, tol = ref.linear(w, x, b, act, r, w_scale, x_scale, dtype)
        for ld, at in ((M, 0), (M + 1, 1), (M + 8, 8), (208, 3), (209, 8)):
            room = torch.full((at + rows * ld + 5,), -7.0, device="cuda").to(dtype)
            out = torch.as_strided(room, (rows, M), (ld, 1), at)
            gb.linear(w, x, bias=b, act=act, residual=r, w_scale=w_scale, x_scale=x_scale, out=out, workspace=ws if ld % 2 else None)
            assert ((out.double() - y).abs() <= tol).all()
            out.fill_(-7.0)
            assert (room == -7.0).all()
    same = r.clone()
    assert gb.linear(w, x, bias=b, act=act, residual=same, w_scale=w_scale, x_scale=x_scale, out=same) is same
    assert torch.equal(same, want)


def test_linear_rows_do_not_depend_on_each_other(gb):
    """A NaN, an infinity or a NaN scale stays in its row."""
    w, x, b, r, ws, xs = operands(gen(5), 20, 256, 512, E4M3, None, True, False, gb)
    clean = gb.linear(w, x, bias=b, w_scale=ws, x_scale=xs)
    bad = xs.clone()
    bad[3] = math.nan
    got = gb.linear(w, x, bias=b, w_scale=ws, x_scale=bad)
    assert torch.isnan(got[3]).all()
    keep = torch.arange(20, device="cuda") != 3
    assert torch.equal(got[keep], clean[keep])
    wb, xb = torch.randn(256, 512, generator=gen(6), device="cuda").to(BF16), torch.randn(20, 512, generator=gen(7), device="cuda").to(BF16)
    clean = gb.linear(wb, xb, act="silu")
    xb[3, 9] = math.inf
    got = gb.linear(wb, xb, act="silu")
    assert torch.equal(got[keep], clean[keep]) and not torch.isfinite(got[3]).all()


def test_activations_far_from_zero(gb):
    """x is one-hot: the sums are the weights themselves."""
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 5.0, -5.0, 30.0, -30.0, 90.0, -90.0, 1e4, -1e4, 1e30, -1e30], device="cuda").to(BF16)
    w = torch.zeros(16, 8, device="cuda", dtype=BF16)
    w[:, 0] = z
    x = torch.zeros(1, 8, device="cuda", dtype=BF16)
    x[0, 0] = 1.0
    for act in ("silu", "gelu"):
        got = gb.linear(w, x, act=act, dtype=F32)[0].double()
        want = ref.activation(z.double(), act)
        assert torch.isfinite(got).all()
        # erfc's cancellation far below zero: gelu there is off by 2^-24 of z
        assert ((got - want).abs() <= 2.0 ** -19 * want.abs() + (2.0 ** -23 * z.double().abs() if act == "gelu" else 1e-35)).all(), act
    got = gb.linear(torch.cat([w, w]), x, act="swiglu", dtype=F32)[0].double()
    want = ref.activation(z.double(), "silu") * z.double()
    fine = want.abs() < 1e38
    assert ((got - want).abs()[fine] <= 2.0 ** -18 * want.abs()[fine] + 1e-35).all()


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_linear_workspace_serves_calls_of_changing_sizes(gb, kind):
    """Outputs that no bulk store takes, over 128 rows: whole tiles and tiles cut between workers, pairs, the
    second launch; the workspace of any content but for its first bytes."""
    ws = gb.linear_workspace(torch.empty(1, 1, device="cuda"), 1500)
    ws[4096:] = 0xff
    for i, (rows, M, K) in enumerate([(600, 4095, 256), (1500, 4096, 256), (200, 257, 8192), (257, 777, 1001), (600, 2501, 640), (129, 129, 5000)] * 2):
        act, bias, residual = ACTS[i % len(ACTS)]
        w, x, b, r, w_scale, x_scale = operands(gen(rows + M), rows, M, K, kind, act, bias, residual, gb)
        dtype = (BF16, F32)[i % 2]
        out = torch.empty(rows, M | 1, device="cuda", dtype=dtype)[:, :M]
        y, tol = ref.linear(w, x, b, act, r, w_scale, x_scale, dtype)
        gb.linear(w, x, bias=b, act=act, residual=r, w_scale=w_scale, x_scale=x_scale, workspace=ws, out=out)
        assert ((out.double() - y).abs() <= tol).all(), (rows, M, K)
        assert not ws[:4096].any()
        first = out.clone()
        gb.linear(w, x, bias=b, act=act, residual=r, w_scale=w_scale, x_scale=x_scale, workspace=ws, out=out)
        assert torch.equal(first, out)


def test_calls_are_captured_and_replayed(gb):
    """A draft layer's MLP as a graph, on another stream than the current one, replayed with new inputs."""
    g = gen(11)
    rows, h, inter = 24, 512, 1100
    gu, gus = gb.quantize_rows(wide(g, 2 * inter, h, h, h ** -0.5))
    dn, dns = gb.quantize_rows(wide(g, h, inter, up(inter, 8), inter ** -0.5))
    weight = (1 + 0.1 * torch.randn(h, generator=g, device="cuda")).to(BF16)
    x, r = wide(g, rows, h, h), wide(g, rows, h, h)
    ws = gb.linear_workspace(gu, rows)

    def mlp():
        y, ys, total = gb.rms_norm(x, weight, 1e-5, residual=r, dtype=E4M3)
        a, as_ = gb.quantize_rows(gb.linear(gu, y, act="swiglu", w_scale=gus, x_scale=ys, workspace=ws))
        return gb.linear(dn, a, residual=total, w_scale=dns, x_scale=as_, workspace=ws)

    mlp()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mlp()
    for seed in (1, 2):
        x.copy_(wide(gen(seed), rows, h, h))
        graph.replay()
        assert torch.equal(out, mlp())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q8, s8 = gb.quantize_rows(x, stream=side)
    got = gb.linear(gu, q8, act="swiglu", w_scale=gus, x_scale=s8, stream=side)
    side.synchronize()
    q, qs = gb.quantize_rows(x)
    assert torch.equal(got, gb.linear(gu, q, act="swiglu", w_scale=gus, x_scale=qs))


def test_nothing_to_do(gb):
    w = torch.randn(64, 32, device="cuda").to(BF16)
    assert gb.linear(w, torch.empty(0, 32, device="cuda", dtype=BF16)).shape == (0, 64)
    codes, scale = gb.quantize_rows(torch.empty(0, 32, device="cuda", dtype=BF16))
    assert codes.shape == (0, 32) and scale.shape == (0,)
    y, _, _ = gb.rms_norm(torch.empty(0, 32, device="cuda", dtype=BF16), torch.ones(32, device="cuda", dtype=BF16))
    assert y.shape == (0, 32)


def test_refusals_of_the_binding(gb):
    w, x = torch.randn(64, 32, device="cuda").to(BF16), torch.randn(4, 32, device="cuda").to(BF16)
    q, s = gb.quantize_rows(x)
    wq, wsc = gb.quantize_rows(w)
    for kw, error in [(dict(act="relu"), ValueError), (dict(bias=torch.zeros(63, device="cuda", dtype=BF16)), ValueError),
                      (dict(bias=torch.zeros(64, device="cuda")), TypeError), (dict(residual=torch.zeros(4, 63, device="cuda", dtype=BF16)), ValueError),
                      (dict(w_scale=wsc), ValueError), (dict(dtype=torch.float16), TypeError), (dict(out=torch.empty(4, 63, device="cuda", dtype=BF16)), ValueError),
                      (dict(workspace=torch.empty(16, device="cuda")), ValueError), (dict(bias=torch.zeros(64, dtype=BF16)), ValueError)]:
        with pytest.raises(error):
            gb.linear(w, x, **kw)
    with pytest.raises(TypeError):
        gb.linear(w, q)
    with pytest.raises(ValueError):
        gb.linear(wq, q)  # no scales
    with pytest.raises(ValueError):
        gb.linear(wq, q, w_scale=wsc, x_scale=s[:3])
    with pytest.raises(ValueError):
        gb.linear(w[:63], x, act="swiglu")
    with pytest.raises(ValueError):
        gb.linear(w, x[:, :16])
    with pytest.raises(ValueError):
        gb.linear(w.t(), w.t())
    with pytest.raises(ValueError):
        gb.quantize_rows(x.cpu())
    with pytest.raises(TypeError):
        gb.quantize_rows(x.float())
    with pytest.raises(TypeError):
        gb.rms_norm(x, torch.ones(32, device="cuda", dtype=BF16), dtype=F32)
    with pytest.raises(ValueError):
        gb.rms_norm(x, torch.ones(31, device="cuda", dtype=BF16))
    with pytest.raises(Exception, match="INVALID_ARG"):
        gb.linear(w, torch.cat([x] * 5), workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(Exception, match="INVALID_ARG"):
        gb.rms_norm(x, torch.ones(32, device="cuda", dtype=BF16), -1.0)
    with pytest.raises(Exception, match="UNSUPPORTED"):
        gb.quantize_rows(torch.zeros(1, 32776, device="cuda", dtype=BF16))


def test_the_short_and_the_long_way_are_the_same_call(gb, monkeypatch):
    """The compiled binding takes what is usual and declines the rest; without it every call goes through
    ctypes."""
    from eagle_speculative_decoding_draft_gb300 import _lib, fp8, kv4
    from test_gpu_kv4 import make_cache
    g = gen(21)
    x, r = wide(g, 20, 100, 112), wide(g, 20, 100, 104)
    weight = torch.ones(100, device="cuda", dtype=BF16)
    w, w_scale = gb.quantize_rows(wide(g, 64, 100, 104))
    qkv = torch.randn(2, 5, 8, 64, generator=g, device="cuda").to(BF16)

    def calls():
        codes, scale = gb.quantize_rows(x)
        y, ys, total = gb.rms_norm(x, weight, 1e-5, residual=r, dtype=E4M3)
        y2, none, h = gb.rms_norm(x, weight, 1e-5)
        assert none is None and h is None
        z = gb.linear(w, codes, act="swiglu", w_scale=w_scale, x_scale=scale, dtype=F32)
        out = torch.empty(20, 64, device="cuda", dtype=BF16)
        assert gb.linear(w, codes, w_scale=w_scale, x_scale=scale, out=out) is out
        c = make_cache(2, 2, 64, 32, 16, fill=0)
        q = c.append_rotary(qkv[:, :, 4:6], qkv[:, :, 6:], q=qkv[:, :, :4])
        assert c.append_rotary(qkv[:, :, 4:6], qkv[:, :, 6:]) is None
        back = c.read(out=(torch.zeros(2, 32, 2, 64, device="cuda"), torch.zeros(2, 32, 2, 64, device="cuda")))
        return [*back, codes.view(torch.uint8), scale, y.view(torch.uint8), ys, total, y2, z, out, q, c.pages, c.lengths]

    assert _lib.short.quantize_rows(x) is not NotImplemented
    one = calls()

    class Declines:
        def __getattr__(self, name):
            return lambda *args: NotImplemented

    for module in (fp8, kv4):
        monkeypatch.setattr(module, "short", Declines())
    for a, b in zip(one, calls()):
        assert a.dtype is b.dtype and a.stride() == b.stride() and torch.equal(a, b)
    for args in [(x.float(),), (x.cpu(),), (x[None],), (x.t(),), (None,)]:
        assert _lib.short.quantize_rows(*args) is NotImplemented


def test_scales_and_biases_that_start_anywhere(gb):
    """Vectors that are slices: aligned to their elements alone."""
    for rows in (5, 60, 300):
        w, x, b, r, w_scale, x_scale = operands(gen(rows), rows, 260, 512, E4M3, "swiglu", True, True, gb)
        want = gb.linear(w, x, bias=b, act="swiglu", residual=r, w_scale=w_scale, x_scale=x_scale)
        b, w_scale, x_scale = (torch.cat([t[:1], t])[1:] for t in (b, w_scale, x_scale))
        assert w_scale.data_ptr() % 16 == 4 and b.data_ptr() % 16 == 2
        assert torch.equal(gb.linear(w, x, bias=b, act="swiglu", residual=r, w_scale=w_scale, x_scale=x_scale), want)


def test_products_of_two_streams_at_once(gb):
    """Clusters, pairs and few rows side by side: each stream's results are those of a run by itself."""
    shapes = [(61, 2048, 4096, "swiglu"), (300, 1024, 8192, "silu"), (8, 4096, 2048, None), (120, 700, 5000, "gelu"), (1500, 2048, 1024, "swiglu")]
    work = []
    for i, (rows, M, K, act) in enumerate(shapes):
        w, x, b, r, ws, xs = operands(gen(i), rows, M, K, E4M3, act, True, True, gb)
        work.append(dict(w=w, x=x, bias=b, act=act, residual=r, w_scale=ws, x_scale=xs))
    want = [gb.linear(**c) for c in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    outs = {}
    for turn in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                for j in range(len(work)):
                    k = (j + i + turn) % len(work)
                    outs[i, turn, k] = gb.linear(**work[k])
    torch.cuda.synchronize()
    for (i, turn, k), out in outs.items():
        assert torch.equal(out, want[k]), (i, turn, k)


def test_offsets_beyond_32_bits(gb):
    """Rows whose elements lie over 2^31 places from the first."""
    n = 140000
    x = torch.zeros(n, 16384, device="cuda", dtype=BF16)
    x[-3:] = torch.randn(3, 16384, generator=gen(0), device="cuda").to(BF16)
    x[1] = x[-1]
    codes, scale = gb.quantize_rows(x)
    few, few_scale = gb.quantize_rows(x[-3:].clone())
    assert torch.equal(codes[-3:].view(torch.uint8), few.view(torch.uint8)) and torch.equal(scale[-3:], few_scale)
    assert not codes[2:-3].view(torch.uint8).any()
    del codes
    y, _, h = gb.rms_norm(x, torch.ones(16384, device="cuda", dtype=BF16), 1e-5, residual=x)
    few_y, _, few_h = gb.rms_norm(x[-3:].clone(), torch.ones(16384, device="cuda", dtype=BF16), 1e-5, residual=x[-3:].clone())
    assert torch.equal(y[-3:], few_y) and torch.equal(h[-3:], few_h)
    del x, y, h
    # a deep product, and a wide one with its residual
    x = torch.zeros(32768, 66000, device="cuda", dtype=BF16)
    x[-2:] = torch.randn(2, 66000, generator=gen(1), device="cuda").to(BF16)
    w = (torch.randn(64, 66000, generator=gen(2), device="cuda") / 256).to(BF16)
    got = gb.linear(w, x)
    y, tol = ref.linear(w, x[-2:], None, None, None, None, None, BF16)
    assert ((got[-2:].double() - y).abs() <= tol).all() and not got[:-2].any()
    del x
    w = (torch.randn(66000, 64, generator=gen(3), device="cuda") / 8).to(BF16)
    x = torch.randn(32768, 64, generator=gen(4), device="cuda").to(BF16)
    r = torch.zeros(32768, 66000, device="cuda", dtype=BF16)
    r[-2:] = 3.0
    for act in (None, "swiglu"):
        res = r if act is None else r[:, :33000]
        got = gb.linear(w, x, act=act, residual=res)
        for at in (slice(0, 2), slice(32766, 32768)):
            y, tol = ref.linear(w, x[at], None, act, res[at], None, None, BF16)
            assert ((got[at].double() - y).abs() <= tol).all(), (act, at)


@pytest.mark.parametrize("rows", [3, 40, 200])
def test_graphs_of_products_replayed_by_turns(gb, rows):
    """Two captured graphs of the same operands, other outputs, replayed on two streams."""
    w, x, b, r, ws, xs = operands(gen(rows), rows, 512, 2048, E4M3, "silu", True, True, gb)
    call = lambda: gb.linear(w, x, bias=b, act="silu", residual=r, w_scale=ws, x_scale=xs)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([call() for _ in range(3)])
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for some in outs:
        for o in some:
            assert torch.equal(o, want)
