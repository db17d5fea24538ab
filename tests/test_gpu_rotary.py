"""Keys turned on the way into the 4-bit cache, and the queries beside them: against the rotation in 64
bits, and against the plain write of keys turned beforehand."""
import math

import pytest
import torch

import fp8_ref as ref
from test_gpu_kv4 import gen, i32, make_cache

pytestmark = pytest.mark.gpu


def qkv(g, B, n, H, Hk, D):
    """One projection's rows, as views of it."""
    x = torch.randn(B, n, H + 2 * Hk, D, generator=g, device="cuda")
    x[:, :, H:] += torch.randn(2 * Hk, D, generator=g, device="cuda")
    return x.to(torch.bfloat16).split([H, Hk, Hk], 2)


def near(got, x, pos, theta):
    """Half a bf16 step, and of the fp32 arithmetic: the reduced angle to 2^-25 of pi, sine and cosine to
    2^-23, two products and a sum: 4 x 2^-23 of the pair's magnitudes; the frequencies, 2^-52 of themselves
    in either computation, by the position."""
    want, size = ref.turned(x, pos, float(torch.tensor(theta, dtype=torch.float32)))  # the call takes a float
    far = 2.0 ** -51 * pos.double().abs()[..., None, None]
    tol = ref.HALF_BF16 * want.abs() * (1 + 2.0 ** -8) + (4 * 2.0 ** -23 + far) * (1 + ref.HALF_BF16) * size
    assert ((got.double() - want).abs() <= tol).all(), float(((got.double() - want).abs() - tol).max())


CASES = [
    # B, H, Hk, D, rows, page, starts
    (1, 1, 1, 32, 1, 16, [0]),
    (2, 6, 3, 64, 5, 16, [0, 13]),
    (3, 2, 2, 96, 77, 32, [0, 31, 100]),
    (2, 32, 8, 128, 200, 64, [63, 1]),
    (64, 32, 32, 128, 1, 64, list(range(0, 640, 10))),
    (5, 18, 9, 32, 9, 128, [0, 5, 127, 128, 300]),
    (1, 64, 8, 128, 1500, 1024, [1]),
    (1, 17, 17, 64, 33, 16, [7]),
]


@pytest.mark.parametrize("B,H,Hk,D,rows,page,starts", CASES)
@pytest.mark.parametrize("given", [False, True])
def test_turned_and_written(B, H, Hk, D, rows, page, starts, given):
    g = gen(B * rows + D)
    q, k, v = qkv(g, B, rows, H, Hk, D)
    cap = max(starts) + rows
    a, b = make_cache(B, Hk, D, cap, page, seed=1), make_cache(B, Hk, D, cap, page, seed=1)
    start = i32(starts)
    pos = (torch.randint(-100, 1 << 20, (B, rows), generator=g, device="cuda", dtype=torch.int32) if given
           else start[:, None] + torch.arange(rows, device="cuda", dtype=torch.int32))
    theta = 500000.0 if given else 10000.0
    more = dict(rope_theta=theta, positions=pos if given else None, start=start)
    out = a.append_rotary(k, v, q=q, **more)
    near(out, q, pos, theta)
    # the queries' way gives the keys that the cache has to hold
    turned = b.append_rotary(k, v, q=k, **more)
    near(turned, k, pos, theta)
    b.pages.fill_(0xff)
    b.append(turned, v.contiguous(), start=start)
    assert torch.equal(a.pages, b.pages)
    assert a.lengths.tolist() == [s + rows for s in starts] == b.lengths.tolist()
    a.status(), b.status()


def test_far_positions_and_other_bases():
    """Angles do not lose bits with the position: whole turns are left out exactly."""
    q, k, v = qkv(gen(2), 1, 40, 4, 2, 128)
    pos = i32([[0, 1, -1, 1 << 30, (1 << 31) - 1, -(1 << 31), 123456789, 99999] * 5])
    for theta in (10000.0, 1e6, 1.0, 0.5, 3.0e38):
        c = make_cache(1, 2, 128, 40, 16)
        near(c.append_rotary(k, v, q=q, positions=pos, rope_theta=theta), q, pos, theta)
        c.status()


def test_selected_nodes_counts_and_starts():
    """A verified tree's accepted nodes at their own positions; requests with nothing; queries of all rows."""
    g = gen(9)
    q, k, v = qkv(g, 4, 8, 8, 2, 64)
    sel = i32([[0, 3, 7, -1], [0, -1, -1, -1], [0, 1, 2, 3], [5, 5, -1, 6]])
    cnt, start = i32([3, 0, 9, 4]), i32([10, 0, 30, 3])
    pos = start[:, None] + torch.tensor([0, 1, 1, 2, 2, 3, 3, 4], device="cuda", dtype=torch.int32)
    a, b, t = (make_cache(4, 2, 64, 64, 16, seed=4) for _ in range(3))
    out = a.append_rotary(k, v, q=q, positions=pos, select=sel, count=cnt, start=start)
    near(out, q, pos, 10000.0)
    turned = t.append_rotary(k, v, q=k, positions=pos)
    b.append(turned, v.contiguous(), select=sel, count=cnt, start=start)
    assert torch.equal(a.pages, b.pages) and torch.equal(a.lengths, b.lengths)
    assert a.lengths.tolist() == [13, 0, 34, 7]
    a.status(), b.status()


def test_behind_the_lengths_without_queries_and_in_place():
    g = gen(3)
    q, k, v = qkv(g, 2, 21, 4, 4, 128)
    a, b = make_cache(2, 4, 128, 64, 16), make_cache(2, 4, 128, 64, 16)
    for c in (a, b):
        c.lengths.copy_(i32([17, 2]))
    pos = i32([17, 2])[:, None] + torch.arange(21, device="cuda", dtype=torch.int32)
    qc = q.contiguous()
    assert a.append_rotary(k, v) is None
    want = b.append_rotary(k, v, q=q, positions=pos)
    assert torch.equal(a.pages, b.pages) and a.lengths.tolist() == [38, 23] == b.lengths.tolist()
    c = make_cache(2, 4, 128, 64, 16)
    c.lengths.copy_(i32([17, 2]))
    assert c.append_rotary(k, v, q=qc, out=qc) is qc
    assert torch.equal(qc, want) and torch.equal(c.pages, a.pages)


def test_bad_pages_and_full_caches_are_latched():
    from eagle_speculative_decoding_draft_gb300._lib import EagleError
    q, k, v = qkv(gen(4), 1, 20, 2, 1, 64)
    c = make_cache(1, 1, 64, 32, 16)
    before = c.pages.clone()
    c.table[0, 1] = -1
    out = c.append_rotary(k, v, q=q)
    assert int(c.lengths[0]) == 16
    near(out, q, torch.arange(20, device="cuda")[None], 10000.0)  # queries of rows that found no place
    with pytest.raises(EagleError):
        c.status()
    c.pages.copy_(before)
    c.append_rotary(k, v, start=i32([-1]))
    assert torch.equal(c.pages, before)
    with pytest.raises(EagleError):
        c.status()
    c = make_cache(1, 1, 64, 32, 16)
    c.append_rotary(k, v, start=i32([25]))
    assert int(c.lengths[0]) == 32
    with pytest.raises(EagleError):
        c.status()


def test_one_token_then_attention_as_a_graph():
    """The form of a decoding step: the new token joins the cache, its query attends over all of it;
    captured once, the lengths move on by themselves."""
    B, H, Hk, D = 3, 8, 2, 64
    g = gen(5)
    a, b = make_cache(B, Hk, D, 96, 16, seed=2), make_cache(B, Hk, D, 96, 16, seed=2)
    _, k0, v0 = qkv(g, B, 40, H, Hk, D)
    cnt = i32([40, 0, 13])
    for c in (a, b):
        c.append_rotary(k0, v0, count=cnt)
    x = torch.zeros(B, 1, H + 2 * Hk, D, device="cuda", dtype=torch.bfloat16)

    def step(c):
        q, k, v = x.split([H, Hk, Hk], 2)
        return c.attention(c.append_rotary(k, v, q=q))

    step(b), b.lengths.copy_(cnt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(a)
    for i in range(20):
        x.copy_(torch.cat(qkv(gen(i), B, 1, H, Hk, D), 2))
        graph.replay()
        assert torch.equal(out, step(b)), i
    assert a.lengths.tolist() == [60, 20, 33] == b.lengths.tolist()
    a.status(), b.status()


def test_refusals_of_the_binding():
    q, k, v = qkv(gen(4), 2, 5, 4, 2, 64)
    c = make_cache(2, 2, 64, 32, 16)
    with pytest.raises(ValueError):
        c.append_rotary(k, v, select=i32([[0], [0]]))
    with pytest.raises(ValueError):
        c.append_rotary(k, v, positions=i32([[0], [0]]))
    with pytest.raises(TypeError):
        c.append_rotary(k, v, positions=torch.zeros(2, 5, device="cuda"))
    with pytest.raises(ValueError):
        c.append_rotary(k, v, q=q[:, :4])
    with pytest.raises(TypeError):
        c.append_rotary(k, v, q=q.float())
    with pytest.raises(ValueError):
        c.append_rotary(k, v, out=torch.empty_like(q))
    with pytest.raises(ValueError):
        c.append_rotary(k, v, q=q, out=q)  # rows of a wider projection
    with pytest.raises(Exception, match="INVALID_ARG"):
        c.append_rotary(k, v, rope_theta=0.0)
    assert math.isfinite(float(c.attention(q.contiguous()).float().sum()))


@pytest.mark.parametrize("H,D,rows,most", [(32, 128, 4096, 8190), (8, 96, 4096, 8190), (16, 64, 4096, 131071), (64, 32, 4096, 1 << 30)])
def test_turned_values_are_those_of_fp32(H, D, rows, most):
    """Cosines and sines to the nearest fp32 value, two products and their sum rounded to fp32 each, then bf16:
    the same bits, but where a cosine or sine lies beside a tie.  The library misses the nearest in 2^-11.8 of
    them.  Such an entry moves a product by one fp32 step, and so one sum in 2^16 / 4 or less by a bf16 step:
    2^-25 of the values.  Up to 2^-20 of them may differ here, by one step (with tables and sums an fp32 step off
    2^-15 do)."""
    g = gen(H + D)
    q, k, v = qkv(g, 1, rows, H, 1, D)
    pos = torch.randint(0, most + 1, (1, rows), generator=g, device="cuda", dtype=torch.int32)
    c = make_cache(1, 1, D, rows, 64)
    got = c.append_rotary(k, v, q=q, positions=pos)
    c.status()
    # the angle as a fraction of a turn, by whole numbers: frequency in 2^-64 of a turn, as Python's floats have it
    turns = [math.pow(10000.0, -2.0 * j / D) / (2 * math.pi) for j in range(D // 2)]
    whole = [int(math.ldexp(t, 64)) % 2 ** 64 for t in turns]
    f = torch.tensor([w - 2 ** 64 if w >= 2 ** 63 else w for w in whole], dtype=torch.int64, device="cuda")
    ang = (pos.long()[..., None] * f).double() * (2 * math.pi / 2.0 ** 64)  # modulo a turn
    cos, sin = torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]
    a, b = q[..., :D // 2].float(), q[..., D // 2:].float()
    want = torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)
    other = got != want
    assert int(other.sum()) <= got.numel() * 2.0 ** -20, int(other.sum())
    assert ((got.double() - want.double()).abs() <= 2 * ref.HALF_BF16 * want.double().abs() + 2.0 ** -23 * 8).all()
