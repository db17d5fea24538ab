"""More of the 8-bit operators on the GPU: products whose tiles follow each other closely, and what their
outputs keep of 64 bits (fp8_ref.py derives the tolerances)."""
import pytest
import torch

import fp8_ref as ref
from test_gpu_fp8 import BF16, E4M3, F32, gb, gen, operands, wide  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,M,K,act,residual", [
    (4096, 14336, 64, "swiglu", False), (4096, 14336, 128, "swiglu", False), (4096, 4095, 128, "swiglu", False),  # a copy a tile
    (4096, 14336, 128, "swiglu", True), (4096, 8192, 64, "silu", False), (4096, 8192, 128, None, True),           # with others'
])
@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_many_tiles_of_short_sums(gb, rows, M, K, act, residual, kind):
    """A tile's sums are ready as soon as the last tile's outputs are on their way: no output may leave with
    the next tile's values."""
    w, x, b, r, w_scale, x_scale = operands(gen(M + K), rows, M, K, kind, act, False, residual, gb)
    kw = dict(act=act, residual=r, w_scale=w_scale, x_scale=x_scale)
    ld = -(-M // 8) * 8
    outs = [torch.empty(rows, ld, device="cuda", dtype=BF16)[:, :M] for _ in range(3)]
    y, tol = ref.linear(w, x, None, act, r, w_scale, x_scale, BF16)
    got = gb.linear(w, x, **kw)
    assert ((got.double() - y).abs() <= tol).all()
    for i in range(60):
        out = outs[i % 3]
        out.fill_(float("nan"))
        gb.linear(w, x, out=out, **kw)
        assert torch.equal(out, got), i


def test_gated_products_without_a_residual_beside_others(gb):
    """On two streams at once, and as a graph that is replayed."""
    work = []
    for i, (rows, M, K) in enumerate([(3000, 7168, 128), (2080, 4096, 512), (1500, 14336, 64), (61, 4096, 1024)]):
        w, x, _, _, ws, xs = operands(gen(i), rows, M, K, E4M3, "swiglu", False, False, gb)
        work.append(dict(w=w, x=x, act="swiglu", w_scale=ws, x_scale=xs))
    want = [gb.linear(**c) for c in work]
    torch.cuda.synchronize()
    outs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs += [(k, gb.linear(**work[k])) for k in ((j + i + turn) % len(work) for j in range(len(work)))]
    torch.cuda.synchronize()
    for k, out in outs:
        assert torch.equal(out, want[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [gb.linear(**c) for c in work * 3]
    for _ in range(3):
        for out in outs:
            out.fill_(float("nan"))
        graph.replay()
        for i, out in enumerate(outs):
            assert torch.equal(out, want[i % len(work)]), i


# What an fp32 output may lose in a sum of products, norm-wise.  The tensor core truncates: an addition (of 16
# products, or 32 in 8 bits) loses half a step of the sum so far on average, 2^-24.5 of it, and a sum that grows as a
# random walk is 2/3 of the last on average.  bf16: 1024 products at a time, 64 additions: 64 x 2/3 x 2^-24.5 =
# 1.8e-6.  8 bits: 4096 at a time, 128 additions, but rows that reach 448 have products that are mostly multiples of
# the accumulator's step, which lose nothing: 2.2e-7 was measured of 4096 such products.  On top: the segments' sums,
# the scales and the output, 2^-24 each.
LOSS = {BF16: 2.5e-6, E4M3: 3e-7}


def check_loss(gb, rows, M, K, kind, odd=False, most=None):
    w, x, _, _, w_scale, x_scale = operands(gen(K + rows), rows, M, K, kind, None, False, False, gb)
    y, _ = ref.linear(w, x, None, None, None, w_scale, x_scale, F32)
    out = torch.empty(rows, M | 1, device="cuda")[:, :M] if odd else None
    got = gb.linear(w, x, w_scale=w_scale, x_scale=x_scale, dtype=F32, out=out)
    off = float((got.double() - y).norm() / y.norm())
    assert off <= (most or LOSS[kind]), off


@pytest.mark.parametrize("rows,M,K,odd", [(100, 20000, 14336, False), (128, 20001, 28672, True), (100, 20000, 40000, False), (61, 1300, 14336, True),
                                          (17, 4096, 8192, False), (300, 20000, 14336, True), (700, 1300, 14336, True), (40, 9728, 2100, False)])
@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_long_sums_of_17_to_128_rows(gb, rows, M, K, odd, kind):
    """All of K in a CTA or parts of it in a cluster; over 128 rows outputs that no bulk store takes."""
    if kind is E4M3 and K > 32768:
        pytest.skip("rows are quantised up to 32768 columns")
    check_loss(gb, rows, M, K, kind, odd)


@pytest.mark.parametrize("rows,M,K", [(700, 1300, 14336), (300, 20000, 14336), (2080, 4096, 8192), (1000, 20000, 4000), (512, 4096, 14336), (600, 4096, 40000),
                                      (400, 2052, 2304)])
@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_long_sums_of_many_rows(gb, rows, M, K, kind):
    """Whole tiles of a pair of CTAs, and of two that share K: up to 4096 bf16 products in one go (256 additions),
    else 2048 at a time (128); all 8-bit products, of which the losses measured (K 7e-11) are held with half on top."""
    if kind is E4M3 and K > 32768:
        pytest.skip("rows are quantised up to 32768 columns")
    check_loss(gb, rows, M, K, kind, most=(K / 16 if K <= 4096 else 256 if K <= 8192 else 128) * 2 / 3 * 2 ** -24.5 + 3 * 2 ** -24
               if kind is BF16 else 1e-10 * K + 2 ** -23)


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_large_products_with_a_workspace(gb, kind):
    """Over 1024 rows and more tiles of outputs than SMs, in rows that no bulk store takes: whole and cut tiles,
    one CTA and pairs, an odd number of tiles; the workspace of any content but for its first bytes, which are
    zero again behind every call, and the rest of the outputs' memory as it was."""
    ws = gb.linear_workspace(torch.empty(1, 1, device="cuda"), 2080)
    ws[4096:] = 0xff
    for i, (rows, M, K, act, residual) in enumerate([(1025, 19999, 256, None, True), (1100, 20001, 520, "silu", False), (2080, 9801, 640, "swiglu", False),
                                                     (1300, 39999, 128, "gelu", False), (1536, 19841, 4096, None, False)] * 2):
        w, x, b, r, w_scale, x_scale = operands(gen(rows + M), rows, M, K, kind, act, i % 2 == 0, residual, gb)
        dtype = (BF16, F32)[(i // 5) % 2]
        room = torch.full((rows, M + 2 - M % 2 + 1), -7.0, device="cuda").to(dtype)
        out = room[:, 1:M + 1]
        y, tol = ref.linear(w, x, b, act, r, w_scale, x_scale, dtype)
        kw = dict(bias=b, act=act, residual=r, w_scale=w_scale, x_scale=x_scale, workspace=ws, out=out)
        gb.linear(w, x, **kw)
        assert ((out.double() - y).abs() <= tol).all(), (rows, M, K)
        assert not ws[:4096].any()
        first = out.clone()
        gb.linear(w, x, **kw)
        assert torch.equal(first, out)
        out.fill_(-7.0)
        assert (room == -7.0).all()
        del y, tol, room, out, first


@pytest.mark.parametrize("rows,M,K", [(1, 1300, 14336), (16, 20000, 14336), (8, 20000, 40000), (9, 1300, 40000), (3, 8192, 4100), (16, 512, 28672), (5, 33000, 28673)])
@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_long_sums_of_few_rows(gb, rows, M, K, kind):
    """A warp's products, an eighth or a quarter of K, in segments where they are more than one."""
    if kind is E4M3 and K > 32768:
        pytest.skip("rows are quantised up to 32768 columns")
    check_loss(gb, rows, M, K, kind)
    if kind is BF16:  # with an epilogue, gates and their ups
        w, x, b, r, _, _ = operands(gen(M), rows, M, K, kind, "swiglu", True, True, gb)
        y, tol = ref.linear(w, x, b, "swiglu", r, None, None, F32)
        got = gb.linear(w, x, bias=b, act="swiglu", residual=r, dtype=F32)
        assert ((got.double() - y).abs() <= tol).all() and float((got.double() - y).norm() / y.norm()) <= 4 * LOSS[kind]


@pytest.mark.parametrize("eps", [1.4e-17, 1e-20, 1e-30, 1e-38, 1e-44])
@pytest.mark.parametrize("rows,cols", [(3, 64), (600, 4096)])
def test_norm_with_an_eps_near_nothing(gb, rows, cols, eps):
    """A row of zeros, or of weights of 0, is 0; tiny rows are what the formula says."""
    g = gen(cols)
    x = wide(g, rows, cols, cols)
    x[0] = 0
    x[1] *= 2.0 ** -100
    w = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(BF16)
    codes, scale, _ = gb.rms_norm(x, w, eps, dtype=E4M3)
    y, _ = ref.norm(x, w, float(torch.tensor(eps, dtype=F32)))
    # rows of 2^-100: their squares vanish in fp32, mean(h^2) of 2^-200 beside any eps but these matters nothing
    assert (codes[0].float() == 0).all() and float(scale[0]) == ref.LEAST
    assert torch.isfinite(scale).all() and torch.isfinite(codes.float()).all()
    ref.check_rows8(codes[2:], scale[2:], y[2:], 40 * 2.0 ** -24)
    ref.check_rows8(codes[1:2], scale[1:2], y[1:2], 2.0 ** -20)
    codes, scale, _ = gb.rms_norm(x, torch.zeros_like(w), eps, dtype=E4M3)
    assert (codes.float() == 0).all() and (scale == ref.LEAST).all()


@pytest.mark.parametrize("rows,cols", [(40, 64), (5, 1000), (600, 4096), (2, 16384), (1, 32768)])
def test_norm_gives_the_codes_of_quantize_rows(gb, rows, cols):
    """Rows of 1 and -1 have the norm 1, and so y = w h exactly: the codes and scales are those that
    quantize_rows gives y, ties of bf16 values over a bf16 maximum among them."""
    g = gen(cols)
    x = (torch.randint(0, 2, (rows, cols), generator=g, device="cuda") * 2 - 1).to(BF16)
    for seed in range(6):
        w = (1 + 0.3 * torch.randn(cols, generator=gen(seed), device="cuda")).to(BF16)
        codes, scale, _ = gb.rms_norm(x, w, 0.0, dtype=E4M3)
        want, want_scale = gb.quantize_rows(x * w)
        assert torch.equal(scale, want_scale) and torch.equal(codes.view(torch.uint8), want.view(torch.uint8))


def test_a_wait_that_ran_out_is_reported(gb):
    """Calls without a status word latch into the device's own.  Here a stalled attention call does it in their
    place: no product is made to fail."""
    from eagle_speculative_decoding_draft_gb300 import KV4Cache, _lib
    lib = _lib.load()
    w, x, _, _, ws, xs = operands(gen(1), 300, 256, 512, E4M3, None, False, False, gb)
    want = gb.linear(w, x, w_scale=ws, x_scale=xs)
    gb.linear_status()
    word = lib.eagle_linear_status_word()
    assert word
    work = gb.linear_workspace(w, 300)
    work[:4096] = 3  # tickets that a product given up in the middle has left
    c = KV4Cache(1, 2, 64, num_pages=4, max_pages=4, page_size=32)
    g = gen(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    c.append(r(1, 100, 2, 64), r(1, 100, 2, 64))
    q, k, v = r(1, 65, 8, 64), r(1, 65, 2, 64), r(1, 65, 2, 64)
    out, nbytes = torch.empty_like(q), c.attention_workspace_bytes(65, 8)
    scratch = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    assert lib.eagle_test_kv4_stall(c._ref, 1, 65, 8, q.data_ptr(), k.data_ptr(), v.data_ptr(), None, out.data_ptr(), scratch.data_ptr(), nbytes,
                                    5_000_000, 0, word, torch.cuda.current_stream().cuda_stream) == 0
    with pytest.raises(_lib.EagleError, match="TIMEOUT"):
        gb.linear_status(workspace=work)
    assert not work[:4096].any()
    side = torch.cuda.Stream()
    gb.linear_status(stream=side), gb.linear_status(device=0), gb.linear_status(device="cuda", workspace=work)
    assert torch.equal(gb.linear(w, x, w_scale=ws, x_scale=xs, workspace=work), want)
    gb.linear_status()
    with pytest.raises(ValueError):
        gb.linear_status(workspace=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        gb.linear_status(workspace=torch.zeros(4096, dtype=torch.uint8))


@pytest.mark.parametrize("rows", [1, 61, 300, 2080])
def test_the_first_call_of_a_process_may_be_captured(gb, rows):
    """What a call prepares once a device (attributes, occupancy, its status word) is allowed in a capture."""
    import subprocess
    import sys
    from pathlib import Path
    code = f"""
import torch
import eagle_speculative_decoding_draft_gb300 as gb
w, x = torch.randn(700, 512, device="cuda").bfloat16(), torch.randn({rows}, 512, device="cuda").bfloat16()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = gb.linear(w, x, dtype=torch.float32)
graph.replay()
gb.linear_status()
want = x.double() @ w.double().T
assert (y.double() - want).norm() <= 1e-5 * want.norm()
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parent.parent, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
