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
