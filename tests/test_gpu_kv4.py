"""The 4-bit key/value cache on the GPU: writing, reading back and attention, against the definition
in 64 bits (kv4_ref.py, which also derives the tolerances)."""
import math

import numpy as np
import pytest
import torch

import kv4_ref as ref
from decoder_ref import layer, random_tree, reference_layer, tolerance, tree_mask

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available()
    return torch.device("cuda", 0)


def rows(g, *shape, scale=0.8):
    """Keys or values: normal, with an offset of each channel."""
    x = torch.randn(*shape, generator=g, device="cuda") + torch.randn(shape[-2:], generator=g, device="cuda")
    return (scale * x).to(torch.bfloat16)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make_cache(B, Hk, D, cap, page, seed=0, spare=2, fill=0xFF):
    """A cache whose pages lie in random order in a pool full of 0xFF (NaN parameters: nothing may
    depend on what no row was written to)."""
    from eagle_speculative_decoding_draft_gb300 import KV4Cache
    mp = max(1, -(-cap // page))
    c = KV4Cache(B, Hk, D, num_pages=B * mp + spare, max_pages=mp, page_size=page)
    c.pages.fill_(fill)
    perm = torch.randperm(B * mp + spare, generator=gen(seed), device="cuda")[:B * mp]
    c.table.copy_(perm.view(B, mp))
    return c


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------
# writing and reading back
# ------------------------------------------------------------------------------------------------
WRITES = [
    # B, Hk, D, page, rows, starts
    (1, 1, 32, 16, 1, [0]),
    (2, 3, 64, 16, 5, [0, 13]),
    (3, 2, 96, 32, 77, [0, 31, 100]),
    (2, 8, 128, 64, 200, [63, 1]),
    (5, 32, 128, 128, 9, [0, 5, 127, 128, 300]),
    (1, 1, 128, 1024, 1500, [1]),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", WRITES, ids=lambda c: "B%d_Hk%d_D%d_page%d_rows%d" % c[:5])
def test_rows_written_read_back_as_their_values(dev, case, dtype):
    B, Hk, D, page, n, starts = case
    g = gen(1)
    c = make_cache(B, Hk, D, max(starts) + n, page)
    k, v = rows(g, B, n, Hk, D), rows(g, B, n, Hk, D, scale=0.01)
    c.append(k, v, start=i32(starts))
    assert c.lengths.tolist() == [s + n for s in starts]
    gk, gv = c.read(start=i32(starts), rows=n, dtype=dtype)
    c.status()
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8 + 2.0 ** -24
    for got, x in ((gk, k), (gv, v)):
        want = ref.stands_for(x)
        assert torch.all((got.double() - want).abs() <= half * want.abs())
        step = ref.parts(x)[1].expand(-1, -1, -1, -1, 32).flatten(-2)
        assert torch.all((want - x.double()).abs() <= step / 2 * (1 + 1e-12))  # at most half a step from x


def test_writes_touch_their_positions_only_and_follow_the_lengths(dev):
    """Three writes one behind the other (the second of them empty for one request), then a rewrite
    from an earlier position: earlier rows keep their values, the lengths follow."""
    g = gen(2)
    B, Hk, D = 3, 2, 64
    c = make_cache(B, Hk, D, 200, 16)
    want = [torch.zeros(0, Hk, D, dtype=torch.bfloat16, device="cuda") for _ in range(B)]
    for counts in ([37, 1, 20], [5, 0, 64], [50, 3, 16]):
        k = rows(g, B, 64, Hk, D)
        c.append(k, k, count=i32(counts))
        want = [torch.cat([w, k[b, :m]]) for b, (w, m) in enumerate(zip(want, counts))]
    k = rows(g, B, 7, Hk, D)
    back = [30, 2, 99]
    c.append(k, k, start=i32(back))
    want = [torch.cat([w[:s], k[b]]) for b, (w, s) in enumerate(zip(want, back))]
    assert c.lengths.tolist() == [len(w) for w in want]
    got, _ = c.read(rows=200, dtype=torch.float32)
    c.status()
    for b in range(B):
        m = len(want[b])
        assert torch.equal(got[b, :m], ref.stands_for(want[b]).float())
        assert torch.all(got[b, m:] == 0)


def test_long_write_without_starts_sets_the_lengths_behind_all_blocks(dev):
    """Many blocks a request that all read their start from the lengths they end up changing."""
    g = gen(3)
    B, Hk, D, n = 2, 8, 128, 1000
    c = make_cache(B, Hk, D, 2100, 64)
    k, v = rows(g, B, n, Hk, D), rows(g, B, n, Hk, D)
    c.append(k, v)
    c.append(v, k, count=i32([1000, 17]))
    assert c.lengths.tolist() == [2000, 1017]
    gk, gv = c.read(rows=2100, dtype=torch.float32)
    for b, m in ((0, 1000), (1, 17)):
        assert torch.equal(gk[b, :1000 + m], ref.stands_for(torch.cat([k[b], v[b, :m]])).float())
        assert torch.equal(gv[b, :1000 + m], ref.stands_for(torch.cat([v[b], k[b, :m]])).float())


def test_selected_rows(dev):
    """Slots name their rows: padding is skipped, a row may come twice, a row that is not there
    latches an error and leaves its position."""
    from eagle_speculative_decoding_draft_gb300._lib import EagleError
    g = gen(4)
    B, n, Hk, D = 4, 9, 2, 128
    c = make_cache(B, Hk, D, 64, 16)
    first = rows(g, B, 20, Hk, D)
    c.append(first, first)
    k = rows(g, B, n, Hk, D)
    sel = [[0, 3, 7, -1, -1], [0, 0, 8, 1, 2], [-1, -1, -1, -1, -1], [4, -1, 5, -1, 6]]
    c.append(k, k, select=i32(sel), count=i32([5, 4, 5, 3]))
    c.status()
    assert c.lengths.tolist() == [23, 24, 20, 23]
    got, _ = c.read(rows=30, dtype=torch.float32)
    for b, take in enumerate([[0, 3, 7], [0, 0, 8, 1], [], [4, None, 5]]):
        assert torch.equal(got[b, :20], ref.stands_for(first[b]).float())
        for j, r in enumerate(take):
            if r is not None:
                assert torch.equal(got[b, 20 + j], ref.stands_for(k[b, r]).float())
    c.lengths.fill_(20)
    c.append(k, k, select=i32([[0, 9, 1]] + [[0, 1, 2]] * 3))
    with pytest.raises(EagleError, match="BOUNDS"):
        c.status()
    c.status()  # cleared


def test_groups_that_hold_no_numbers_or_only_one(dev):
    """NaN, infinities and magnitudes above 32768 make their own group NaN; constants, zeros, tiny and
    subnormal values, and wide ranges keep the error bound."""
    D = 128
    x = torch.zeros(12, 1, D, dtype=torch.float32, device="cuda")
    x[0, 0, 5] = math.nan
    x[1, 0, 40] = math.inf
    x[2, 0, 70] = -math.inf
    x[3, 0, 100] = 33000.0
    x[4] = 3.25
    x[5] = -1e-30
    x[6, 0] = torch.linspace(-32768, 32768, D)
    x[7, 0] = torch.linspace(0, 1e-6, D)
    x[8, 0] = torch.linspace(-1e-38, 1e-38, D)
    x[9, 0] = 1000 + torch.linspace(0, 8, D)
    x[10, 0, ::2] = -0.0
    x[11, 0] = torch.linspace(-2.0 ** -14, 2.0 ** -15, D)
    x = x.to(torch.bfloat16)[None]
    c = make_cache(1, 1, D, 12, 16)
    c.append(x, x)
    for got in c.read(rows=12, dtype=torch.float32):
        want = ref.stands_for(x)
        bad = torch.isnan(want)
        assert torch.equal(torch.isnan(got), bad) and int(bad.sum()) == 4 * 32
        assert torch.all((got.double() - want).abs()[~bad] <= 2.0 ** -24 * want.abs()[~bad])
        # each within half a step of x, and a step no larger than the range asks for
        step = ref.parts(x)[1].expand(-1, -1, -1, -1, 32).flatten(-2)
        assert torch.all(((got.double() - x.double()).abs() <= step / 2 * (1 + 1e-6) + 2.0 ** -24 * want.abs())[~bad])


def test_ties_go_to_the_even_code(dev):
    """Values half way between codes: steps of a power of two, from a least value of 0 and of -8 steps."""
    halves = torch.cat([torch.tensor([0.0, 15.0]), torch.arange(30) * 0.5]).cuda()
    x = torch.stack([(halves + low) * 2.0 ** e for low in (0.0, -8.0) for e in (-12, -3, 0, 5, 10)])
    k = x[:, None, None].to(torch.bfloat16)  # [groups][1][1][32]
    assert torch.equal(k[:, 0, 0].float(), x)
    c = make_cache(len(x), 1, 32, 16, 16)
    c.append(k, -k)
    got_k, got_v = c.read(rows=1, dtype=torch.float32)
    c.status()
    assert torch.equal(got_k, ref.stands_for(k).float()) and torch.equal(got_v, ref.stands_for(-k).float())
    step = (x.amax(1) - x.amin(1)) / 15
    assert torch.equal(got_k[:, 0, 0], x.amin(1)[:, None] + torch.round((x - x.amin(1)[:, None]) / step[:, None]) * step[:, None])


def test_bad_pages_and_positions_are_skipped_and_reported(dev):
    from eagle_speculative_decoding_draft_gb300._lib import EagleError
    g = gen(5)
    c = make_cache(3, 1, 32, 64, 16)
    k = rows(g, 3, 40, 1, 32)
    c.table[1, 1] = -1
    c.table[2, 0] = c.num_pages
    c.append(k, k, start=i32([40, 0, 0]))  # request 0: 40 .. 79 of 64
    with pytest.raises(EagleError, match="BOUNDS"):
        c.status()
    assert c.lengths.tolist() == [64, 40, 40]
    out = torch.full((3, 64, 1, 32), 7.0, device="cuda")
    got, _ = c.read(out=(out, out.clone()))
    with pytest.raises(EagleError, match="BOUNDS"):
        c.status()
    assert torch.equal(got[0, 40:], ref.stands_for(k[0, :24]).float())
    assert torch.equal(got[1, :16], ref.stands_for(k[1, :16]).float())
    assert torch.all(got[1, 16:32] == 7.0) and torch.all(got[1, 40:] == 7.0) and torch.all(got[2, :16] == 7.0)
    assert torch.equal(got[2, 16:40], ref.stands_for(k[2, 16:40]).float())
    before = c.lengths.clone()
    c.append(k, k, start=i32([-1, -5, -1]))
    with pytest.raises(EagleError, match="BOUNDS"):
        c.status()
    assert torch.equal(c.lengths, before)


@pytest.mark.parametrize("own_start", [False, True], ids=["behind", "start"])
def test_lengths_end_behind_the_last_written_slot(dev, own_start):
    """Trailing slots that name no row, lie behind the capacity or on no page are not written, and a length that
    counted them would make old bytes of the pool keys."""
    from eagle_speculative_decoding_draft_gb300._lib import EagleError
    g = gen(16)
    B, rows_n, cap, first = 8, 150, 160, [0, 3, 16, 20, 150, 157, 160, 0]
    c = make_cache(B, 1, 32, cap, 16)
    c.table[0, 1:] = -1           # one page: 16 of 150 rows
    c.table[1, 5:] = c.num_pages  # 80 positions
    c.table[2, :] = -1            # none
    c.table[3, 3] = -1            # a gap in front of what is written
    c.table[7, ::2] = -1          # every second page
    c.lengths.copy_(i32(first))
    k = rows(g, B, rows_n, 1, 32)
    c.append(k, k, start=i32(first) if own_start else None)
    with pytest.raises(EagleError, match="BOUNDS"):
        c.status()
    assert c.lengths.tolist() == [16, 80, 16, 160, 160, 160, 160, 150]
    # rows by name: -1 and rows that are not there behind the last one, slots behind the capacity
    c.lengths.copy_(i32(first))
    sel = torch.full((B, 70), -1, dtype=torch.int32, device="cuda")
    sel[0, 3] = 5                     # position 3 of the only page
    sel[0, 20] = 6                    # on no page
    sel[1, :] = torch.arange(70)      # 3 .. 72
    sel[1, 60:] = rows_n              # no such rows
    sel[2, 0] = 1                     # on no page: nothing is written
    sel[3, 30:34] = 1                 # 50 .. 53: in the gap
    sel[4, [0, 12]] = 1               # 150; 162 lies behind the capacity
    sel[5, [0, 2]] = 1                # 157, 159
    sel[6, 0] = 1                     # 160: behind it
    c.append(k, k, select=sel, start=i32(first) if own_start else None)
    with pytest.raises(EagleError, match="BOUNDS"):
        c.status()
    assert c.lengths.tolist() == [4, 63, 16, 20, 151, 160, 160, 0]


def test_pool_beyond_32_bits(dev):
    """Pages whose byte offsets pass 2^32, written, read and attended to."""
    from eagle_speculative_decoding_draft_gb300 import KV4Cache
    Hk, D, page = 8, 128, 64
    num = (1 << 32) // (Hk * 4 * 640 * 4) + 40
    c = KV4Cache(1, Hk, D, num_pages=num, max_pages=4, page_size=page)
    assert c.pages.numel() > 1 << 32
    c.table.copy_(i32([[num - 1, num - 3, 0, num - 2]]))
    g = gen(6)
    k, v = rows(g, 1, 250, Hk, D), rows(g, 1, 250, Hk, D)
    c.append(k, v)
    gk, gv = c.read(rows=250, dtype=torch.float32)
    assert torch.equal(gk, ref.stands_for(k).float()) and torch.equal(gv, ref.stands_for(v).float())
    q = rows(g, 1, 1, 16, D)
    o = c.attention(q)
    c.status()
    want, tol = ref.attend(q[0], k[0], v[0], None, None, torch.ones(1, 250, dtype=torch.bool, device="cuda"))
    assert torch.all((o[0].double() - want).abs() <= tol)


# ------------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------------
def build(case, seed=0, kscale=0.8, vscale=0.8, qscale=1.5):
    B, n, H, Hk, D, page, lens, kind = case
    g = gen(seed)
    cap = max(max(lens), 1)
    c = make_cache(B, Hk, D, cap, page, seed)
    kc, vc = rows(g, B, cap, Hk, D, scale=kscale), rows(g, B, cap, Hk, D, scale=vscale)
    c.append(kc, vc, count=i32(lens))  # nothing behind the lengths is ever written
    q = (qscale * torch.randn(B, n, H, D, generator=g, device="cuda")).to(torch.bfloat16)
    kn, vn = (rows(g, B, n, Hk, D, scale=kscale), rows(g, B, n, Hk, D, scale=vscale)) if kind != "cache" else (None, None)
    mask = None
    if kind == "tree":
        rng = np.random.default_rng(seed)
        mask = np.stack([tree_mask(random_tree(n, 8, rng)[0]) for _ in range(B)])
        mask = torch.from_numpy(mask.view(np.int32)).cuda()
    return c, kc, vc, q, kn, vn, mask


def check_attention(case, made, o):
    B, n, H, Hk, D, page, lens, kind = case
    c, kc, vc, q, kn, vn, mask = made
    assert o.shape == q.shape and o.dtype == torch.bfloat16
    for b in range(B):
        t = lens[b]
        see = ref.sees(n, t, None if mask is None else mask[b], "cuda")
        if kn is None:
            see = see[:, :t]
        want, tol = ref.attend(q[b], kc[b, :t], vc[b, :t], None if kn is None else kn[b], None if vn is None else vn[b], see)
        assert torch.equal(torch.isnan(o[b]), torch.isnan(want))
        err = torch.nan_to_num(o[b].double() - want).abs()
        assert torch.all(err <= tol), (b, float((err - tol).max()), float(err.max()))


ATTENTION = [
    # B, n, H, Hk, D, page, lengths, new keys
    (1, 1, 1, 1, 32, 16, [0], "causal"),            # a lone token and nothing cached
    (1, 1, 1, 1, 128, 16, [1], "cache"),            # one cached key and no new ones
    (2, 1, 4, 4, 128, 64, [0, 5], "cache"),         # a request that sees nothing
    (3, 1, 32, 32, 128, 64, [1024, 1, 63], "causal"),
    (2, 5, 8, 8, 64, 16, [64, 129], "tree"),
    (4, 8, 8, 8, 128, 32, [0, 15, 16, 700], "tree"),
    (2, 7, 12, 4, 64, 32, [3001, 0], "tree"),        # groups of 3: 21 rows
    (2, 16, 2, 2, 128, 128, [250, 1], "tree"),       # 16 rows
    (3, 11, 6, 2, 96, 16, [100, 33, 1], "tree"),     # head_dim 96, 33 rows
    (2, 40, 3, 1, 32, 64, [70, 200], "tree"),        # head_dim 32, 120 rows, two mask words
    (1, 61, 4, 4, 128, 64, [1024], "tree"),
    (2, 65, 8, 2, 128, 64, [1024, 77], "tree"),      # 260 rows: two full tiles and 4 rows
    (2, 65, 8, 2, 64, 16, [130, 600], "tree"),
    (1, 130, 8, 8, 128, 64, [511], "causal"),        # more new keys than a tile
    (2, 200, 16, 2, 128, 256, [0, 1000], "causal"),
    (2, 129, 4, 4, 96, 16, [50, 0], "causal"),
    (1, 33, 8, 1, 64, 32, [64], "cache"),            # MQA, 264 rows, no new keys
    (9, 1, 64, 8, 128, 16, [1, 20000, 3, 0, 511, 4097, 9000, 64, 65], "causal"),  # ragged: split units
    (1, 1, 8, 8, 128, 64, [50000], "causal"),
    (1, 70, 32, 4, 128, 64, [9000], "tree"),         # 560 rows, split units of many rows
    (300, 1, 2, 1, 64, 16, [i % 37 for i in range(300)], "causal"),  # more requests than threads
    (40, 8, 8, 2, 128, 16, [i * 131 % 700 for i in range(40)], "tree"),     # 32 rows of more than 32 requests
    (35, 80, 8, 2, 64, 32, [i * 53 % 300 for i in range(35)], "causal"),    # and 320 rows: units of different lengths
    (900, 17, 1, 1, 64, 16, [i % 21 for i in range(900)], "causal"),        # 17 rows, more requests than threads
    (2, 128, 1, 1, 128, 64, [128, 127], "causal"),   # rows and keys that fill their tiles
    (3, 129, 1, 1, 128, 16, [0, 255, 257], "tree"),  # one row and one key more
    (1, 256, 1, 1, 64, 1024, [1025], "causal"),
    (1, 300, 16, 2, 128, 64, [100], "tree"),         # ten tiles of query rows
    (1, 4097, 1, 1, 64, 16, [5], "causal"),          # the most nodes
    (1, 4097, 1, 1, 32, 16, [5], "causal"),
    (2, 65, 8, 2, 96, 64, [1024, 77], "tree"),
    (3, 150, 4, 2, 32, 32, [900, 0, 131], "causal"),
    (20, 17, 3, 3, 96, 16, [i * 97 % 1500 for i in range(20)], "tree"),
    (2, 40, 8, 1, 96, 128, [3000, 5], "cache"),
    (2, 90, 8, 1, 32, 128, [3000, 5], "cache"),
]


@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: "B%d_n%d_H%d_Hk%d_D%d_page%d_%s" % (*c[:6], c[7]))
def test_attention_matches_the_definition(dev, case):
    made = build(case)
    c, _, _, q, kn, vn, mask = made
    o = c.attention(q, kn, vn, mask=mask)
    c.status()
    check_attention(case, made, o)
    # roundings to bf16 are off by 2^-8 / sqrt(3) in the mean square, everything else by less
    want = torch.cat([ref.attend(q[b], made[1][b, :t], made[2][b, :t], None if kn is None else kn[b],
                                 None if vn is None else vn[b],
                                 ref.sees(q.shape[1], t, None if mask is None else mask[b], "cuda")[:, :t + (0 if kn is None else q.shape[1])])[0]
                      for b, t in enumerate(case[6])])
    assert float((o.double().flatten(0, 1) - want).norm()) <= 2.0 ** -8 * float(want.norm())
    again = c.attention(q, kn, vn, mask=mask)
    assert torch.equal(o, again)  # bit for bit


def many_requests(B, n, kind, D=64, base=50):
    """B requests that repeat `base` ones (their pages shared): more than 32 for every CTA of the device."""
    case = (base, n, 1, 1, D, 16, [i * 37 % 101 for i in range(base)], kind)
    c0, kc, vc, q, kn, vn, mask = made = build(case, 15)
    from eagle_speculative_decoding_draft_gb300 import KV4Cache
    again = torch.arange(B, device="cuda") % base
    c = KV4Cache(B, 1, D, num_pages=c0.num_pages, max_pages=c0.max_pages, page_size=16, pages=c0.pages)
    c.table.copy_(c0.table[again])
    c.lengths.copy_(c0.lengths[again])
    return case, made, again, c, [None if x is None else x[again].contiguous() for x in (q, kn, vn, mask)]


MANY = [(20000, 1, "causal"), (9000, 3, "cache"), (8000, 17, "causal"), (6100, 20, "tree")]


@pytest.mark.parametrize("B,n,kind", MANY, ids=lambda v: str(v))
def test_thousands_of_short_requests(dev, B, n, kind):
    """Runs of a CTA over more than 32 requests, at whose ends the next lengths are read."""
    case, made, again, c, (q, kn, vn, mask) = many_requests(B, n, kind)
    o = c.attention(q, kn, vn, mask=mask)
    c.status()
    base, lens = case[0], case[6]
    for b in range(base):  # every copy of the request (the line cuts them at other places)
        t, (kc, vc, q1, kn, vn, mask1) = lens[b], made[1:]
        see = ref.sees(n, t, None if mask1 is None else mask1[b], "cuda")[:, :t + (0 if kn is None else n)]
        want, tol = ref.attend(q1[b], kc[b, :t], vc[b, :t], None if kn is None else kn[b], None if vn is None else vn[b], see)
        assert torch.all((o[b::base].double() - want).abs() <= tol)


@pytest.mark.parametrize("B,n,kind", MANY + [(5, 1, "causal"), (5, 70, "tree"), (40, 8, "tree"), (40, 130, "causal")], ids=lambda v: str(v))
def test_lengths_that_change_under_a_call(dev, B, n, kind):
    """Outputs are undefined then, but every call ends, no wait runs out, nothing but the outputs is written, and calls
    after it are right."""
    case, made, again, c, (q, kn, vn, mask) = many_requests(B, n, kind)
    lens = c.lengths.clone()
    other = [torch.zeros_like(lens), torch.full_like(lens, c.capacity), lens.flip(0), (lens * 7 + 3) % (c.capacity + 1), lens]
    want = c.attention(q, kn, vn, mask=mask)
    pages = c.pages.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    done = torch.cuda.Event()
    for _ in range(20):
        for _ in range(5):
            c.attention(q, kn, vn, mask=mask)
        done.record()
        while not done.query():
            with torch.cuda.stream(side):
                for x in other:
                    c.lengths.copy_(x)
            side.synchronize()
    torch.cuda.synchronize()
    c.status()
    assert torch.equal(c.pages, pages)
    c.lengths.copy_(lens)
    assert torch.equal(c.attention(q, kn, vn, mask=mask), want)
    c.status()


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("n", [3, 7, 9, 15, 17, 31, 33, 63, 97, 127, 129, 161, 255, 257, 289])
def test_warps_that_a_unit_fills_in_part(dev, n, D):
    """Query rows that end inside a warp's 32 (or 8), in units that one CTA finishes and in split ones,
    with a NaN that some of the warp's queries see and others do not."""
    case = (3, n, 1, 1, D, 64, [0, 100, 9000], "causal")
    made = build(case, 14)
    c, kc, vc, q, kn, vn, mask = made
    o = c.attention(q, kn, vn)
    check_attention(case, made, o)
    vn[:, n // 2, :, 5] = math.nan
    bad = c.attention(q, kn, vn)
    c.status()
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[:, n // 2:, :, 5] = True
    assert torch.equal(torch.isnan(bad), hit)
    assert torch.equal(bad[~hit], o[~hit])


@pytest.mark.parametrize("kscale,vscale,qscale", [(0.8, 60.0, 1.5), (4.0, 1e-3, 4.0), (0.8, 8000.0, 1.5), (1e-3, 1e-5, 1e3),
                                                  (0.8, 0.8, 1e-30), (0.02, 0.8, 1e30)])
@pytest.mark.parametrize("case", [(2, 8, 4, 4, 128, 32, [700, 33], "tree"), (2, 65, 8, 2, 128, 64, [300, 1], "tree"),
                                  (1, 20, 3, 3, 64, 64, [1000], "causal")], ids=["8rows", "260rows", "20rows"])
def test_attention_over_values_of_other_sizes(dev, case, kscale, vscale, qscale):
    made = build(case, 3, kscale, vscale, qscale)
    c, _, _, q, kn, vn, mask = made
    if qscale == 1e30:  # scores near 1e28: one key takes all; the definition is the arg-max's value
        q.zero_()
        q[..., 0] = 1e30
        q[..., 3] = 1e29
    o = c.attention(q, kn, vn, mask=mask)
    check_attention(case, made, o)


ROWS = [(5, 1), (16, 1), (17, 1), (40, 2), (130, 2), (300, 1)]  # nodes, heads of one kv head


def check_sizes(case, made, o):
    B, n, H, Hk, D, page, lens, kind = case
    c, kc, vc, q, kn, vn, mask = made
    for b, t in enumerate(lens):
        see = ref.sees(n, t, None if mask is None else mask[b], "cuda")[:, :t + (0 if kn is None else n)]
        args = q[b], kc[b, :t], vc[b, :t], None if kn is None else kn[b], None if vn is None else vn[b], see
        want = ref.attend(*args)[0]
        tol = ref.relative_tolerance(*args, want)
        err = (o[b].double() - want).abs()
        assert torch.all(err <= tol), (b, float((err / tol.clamp(min=1e-300)).max()))


@pytest.mark.parametrize("D", [96, 128])
@pytest.mark.parametrize("n,H", ROWS, ids=lambda v: str(v))
@pytest.mark.parametrize("kscale,vscale,qscale", [(0.8, 1e-3, 1.0), (0.8, 1e-5, 1.0), (0.8, 1e-7, 1.0), (0.8, 1e-20, 1.0),
                                                  (0.8, 2e5, 1.0), (0.8, 1e20, 1.0), (1e-6, 0.8, 1e6), (1e-12, 1e-3, 1e12),
                                                  (1e15, 0.8, 1e-15)])
def test_new_keys_and_values_of_any_size(dev, n, H, D, kscale, vscale, qscale):
    """Nothing cached: the new keys and values alone, as close for small and large ones as for those near 1."""
    case = (2, n, H, 1, D, 16, [0, 0], "tree")
    made = build(case, 17, kscale, vscale, qscale)
    c, _, _, q, kn, vn, mask = made
    check_sizes(case, made, c.attention(q, kn, vn, mask=mask))
    c.status()


@pytest.mark.parametrize("n,H", ROWS, ids=lambda v: str(v))
def test_new_values_of_many_sizes_at_once(dev, n, H):
    """Dims from 2^0 down to 2^-40 and up to 2^40, each as close as its own size says; a hidden node that holds large
    finite values changes nothing."""
    case = (1, n, H, 1, 128, 16, [0], "tree")
    made = build(case, 18)
    c, _, _, q, kn, vn, mask = made
    vn *= 2.0 ** (torch.arange(128, device="cuda") % 81 - 40)
    kn[0, ::3] *= 2.0 ** -20
    o = c.attention(q, kn, vn, mask=mask)
    check_sizes(case, made, o)
    kn[0, n - 1], vn[0, n - 1] = 1e4, -6e4  # the last node: no one's ancestor
    assert torch.equal(c.attention(q, kn, vn, mask=mask)[0, :n - 1], o[0, :n - 1])


@pytest.mark.parametrize("vscale,other", [(2e-6, 1.0), (3e-5, 1.0), (1e-3, 1.0), (0.8, 1.0), (0.8, 1e-4), (3e-5, 1e4)])
@pytest.mark.parametrize("n", [1, 16, 17])
def test_many_light_keys_beside_a_heavy_one(dev, n, vscale, other):
    """65536 cached keys, of which four (one for each warp that multiplies) weigh e^11 times as much as the others, which
    together still are a fifth of the sum: p and p s of the light ones keep their bits however small the values, also
    beside a group of 32 dims of another size."""
    from eagle_speculative_decoding_draft_gb300 import KV4Cache
    D, t, B = 96, 65536, 600
    case = (1, n, 1, 1, D, 64, [t], "cache")
    made = build(case, 20, 0.05, vscale)
    c0, kc, vc, q, _, _, _ = made
    vc[..., 32:64] *= other
    q.fill_(1.0)
    kc[0, :64:16] = 11.0 / math.sqrt(D)  # q . k / sqrt(D) = 11
    vc[0, :64:16] = -vscale
    vc[0, :64:16, :, 32:64] *= other
    c0.append(kc, vc, start=i32([0]))
    c = KV4Cache(B, 1, D, num_pages=c0.num_pages, max_pages=c0.max_pages, page_size=64, pages=c0.pages)  # all over the same pages
    c.table.copy_(c0.table.expand(B, -1))
    c.lengths.fill_(t)
    o = c.attention(q.expand(B, -1, -1, -1).contiguous())
    c.status()
    see = torch.ones(n, t, dtype=torch.bool, device="cuda")
    args = q[0], kc[0], vc[0], None, None, see
    want = ref.attend(*args)[0]
    over = float(((o.double() - want).abs() / ref.relative_tolerance(*args, want)).max())
    assert over <= 1, over


@pytest.mark.parametrize("D", [64, 96])
@pytest.mark.parametrize("n,B,kind", [(1, 1000, "cache"), (16, 700, "cache"), (17, 350, "cache"), (129, 170, "cache"), (129, 170, "causal")],
                         ids=lambda v: str(v))
def test_millions_of_cached_keys_in_one_run(dev, n, B, kind, D):
    """Requests of 4 M tokens each (the same 65536 over and over, and every request the same pages), so many that
    a CTA sums a whole request: sums of positive values, which accumulators that truncate let shrink.  They may truncate
    2048 products in a row, 2^-23 each: 2^-12; the sum of p over a tile at a time rounds no more than that."""
    from eagle_speculative_decoding_draft_gb300 import KV4Cache
    base, t, page = 1 << 16, 1 << 22, 1024
    c0 = KV4Cache(1, 1, D, num_pages=base // page, max_pages=base // page, page_size=page)
    g = gen(21)
    kc = rows(g, 1, base, 1, D, scale=0.3)
    vc = (1 + torch.rand(1, base, 1, D, generator=g, device="cuda")).to(torch.bfloat16)
    c0.append(kc, vc)
    c = KV4Cache(B, 1, D, num_pages=base // page, max_pages=t // page, page_size=page, pages=c0.pages)
    c.table.copy_((torch.arange(t // page, device="cuda") % (base // page)).expand(B, -1))
    c.lengths.fill_(t)
    q = torch.randn(1, n, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    kn, vn = (rows(g, 1, n, 1, D, scale=0.3), rows(g, 1, n, 1, D)) if kind == "causal" else (None, None)
    many = lambda x: None if x is None else x.expand(B, -1, -1, -1).contiguous()
    o = c.attention(many(q), many(kn), many(vn))
    c.status()
    see = torch.ones(n, base, dtype=torch.bool, device="cuda")
    want, _ = ref.attend(q[0], kc[0], vc[0], None, None, see)
    tol = ref.relative_tolerance(q[0], kc[0], vc[0], None, None, see, want) + 2.0 ** -11 * want.abs()
    if kind == "causal":  # the cached keys' weights count 64 times beside the new keys'
        scores = lambda k: q[0, :, 0].double() @ k[:, 0].T / math.sqrt(D)
        old = scores(ref.stands_for(kc[0])).exp().sum(1, keepdim=True) * (t // base)
        new = scores(kn[0].double()).exp().tril()
        want = ((old * want[:, 0] + new @ vn[0, :, 0].double()) / (old + new.sum(1, keepdim=True)))[:, None]
    over = float(((o.double() - want).abs() / tol).max())
    assert over <= 1, over


@pytest.mark.parametrize("n,H", ROWS, ids=lambda v: str(v))
def test_largest_and_smallest_sizes(dev, n, H):
    """The ends of what the contract names, 2^100 and 2^-100, seen and weighted."""
    case = (1, n, H, 1, 64, 16, [0], "causal")
    made = build(case, 19)
    c, _, _, q, kn, vn, mask = made
    for size in (2.0 ** 100, 2.0 ** -100):
        vn.copy_(torch.where(vn > 0, size, -size / 2))
        check_sizes(case, made, c.attention(q, kn, vn))
        kn.copy_(torch.where(kn > 0, size, -size).to(torch.bfloat16))
        q.copy_((q.float() / q.float().abs().amax(-1, keepdim=True) / size / 64).to(torch.bfloat16))
        check_sizes(case, made, c.attention(q, kn, vn))
        made = build(case, 19)
        c, _, _, q, kn, vn, mask = made
    c.status()


@pytest.mark.parametrize("case", [(2, 9, 4, 4, 128, 32, [70, 0], "tree"), (1, 65, 8, 2, 64, 64, [100], "tree"),
                                  (2, 40, 8, 1, 128, 16, [0, 257], "tree"), (1, 50, 4, 1, 96, 16, [40], "tree"),
                                  (2, 50, 2, 1, 32, 16, [40, 300], "tree")],
                         ids=["9rows", "260rows", "320rows", "200rows96", "100rows32"])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf, 3e38])
def test_what_hidden_keys_hold_has_no_influence(dev, case, what):
    """A leaf that no other node sees: its key and value may hold anything."""
    made = build(case, 4)
    c, kc, vc, q, kn, vn, mask = made
    B, n = q.shape[:2]
    hidden = n - 1  # the last node is no one's ancestor
    clean = c.attention(q, kn, vn, mask=mask)
    kn[:, hidden] = what
    vn[:, hidden, :, 3::5] = what
    dirty = c.attention(q, kn, vn, mask=mask)
    assert torch.equal(clean[:, :hidden], dirty[:, :hidden])
    if not math.isfinite(what):
        assert torch.all(~torch.isfinite(dirty[:, hidden, :, 3]))


@pytest.mark.parametrize("n,H", [(5, 2), (5, 64)], ids=["5rows", "160rows"])
def test_infinite_values_reach_the_rows_that_see_them(dev, n, H):
    case = (1, n, H, 2, 128, 16, [40], "causal")
    made = build(case, 5)
    c, kc, vc, q, kn, vn, mask = made
    clean = c.attention(q, kn, vn)
    vn[0, 2, :, 7] = math.inf
    vn[0, 3, :, 9] = math.nan
    vn[0, 4, :, 7] = -math.inf
    o = c.attention(q, kn, vn)[0]
    assert torch.equal(o[:2], clean[0, :2])
    assert torch.all(o[2:4, :, 7] == math.inf) and torch.all(torch.isnan(o[4, :, 7]))
    assert torch.all(torch.isnan(o[3:, :, 9])) and torch.all(torch.isfinite(o[2, :, 9]))
    rest = [d for d in range(128) if d not in (7, 9)]
    assert torch.equal(o[:, :, rest], clean[0][:, :, rest])


@pytest.mark.parametrize("n,H", [(1, 2), (40, 8)], ids=["1row", "160rows"])
def test_cached_groups_without_numbers_reach_their_dims_only(dev, n, H):
    """A cached value group that is NaN makes its 32 dims NaN for every row, a key group every dim."""
    case = (1, n, H, 2, 128, 16, [200], "causal")
    c, kc, vc, q, kn, vn, mask = made = build(case, 6)
    vc[0, 150, 0, 70] = math.nan  # kv head 0, dims 64 .. 95
    c.append(kc, vc, start=i32([0]))
    o = c.attention(q, kn, vn)[0]
    per = H // 2
    assert torch.all(torch.isnan(o[:, :per, 64:96]))
    assert torch.all(torch.isfinite(o[:, :per, :64])) and torch.all(torch.isfinite(o[:, :per, 96:]))
    assert torch.all(torch.isfinite(o[:, per:]))
    kc[0, 199, 1, 0] = math.inf
    c.append(kc, vc, start=i32([0]))
    o = c.attention(q, kn, vn)[0]
    assert torch.all(torch.isnan(o[:, per:]))


@pytest.mark.parametrize("n,Hq", [(4, 1), (30, 2), (50, 4)])
def test_rows_that_see_nothing_are_zero(dev, n, Hq):
    """Empty mask rows over an empty cache; rows with a key beside them keep their values."""
    case = (2, n, Hq, 1, 128, 16, [0, 9], "tree")
    c, kc, vc, q, kn, vn, mask = made = build(case, 7)
    mask[:, 1::2] = 0
    o = c.attention(q, kn, vn, mask=mask)
    assert torch.all(o[0, 1::2] == 0)
    check_attention(case, made, o)


@pytest.mark.parametrize("n,H,Hk", [(1, 4, 2), (9, 4, 2), (70, 8, 2)])
def test_attention_on_slices_of_wider_rows(dev, n, H, Hk):
    """q, k and v as parts of one projection's rows, as the decoder layer passes them."""
    D = 64
    case = (2, n, H, Hk, D, 32, [100, 41], "causal")
    c, kc, vc, q, kn, vn, mask = build(case, 8)
    want = c.attention(q, kn, vn)
    wide = torch.full((2, n, (H + 2 * Hk) * D + 24), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[..., :H * D] = q.flatten(2)
    wide[..., H * D:(H + Hk) * D] = kn.flatten(2)
    wide[..., (H + Hk) * D:(H + 2 * Hk) * D] = vn.flatten(2)
    view = lambda lo, h: wide[..., lo:lo + h * D].unflatten(2, (h, D))
    got = c.attention(view(0, H), view(H * D, Hk), view((H + Hk) * D, Hk))
    assert torch.equal(got, want)
    c2 = make_cache(2, Hk, D, n, 16)
    c2.append(view(H * D, Hk), view((H + Hk) * D, Hk))
    assert torch.equal(c2.read(rows=n, dtype=torch.float32)[1], ref.stands_for(vn).float())


def test_bad_pages_count_as_absent(dev):
    from eagle_speculative_decoding_draft_gb300._lib import EagleError
    case = (1, 3, 4, 2, 128, 16, [100], "causal")
    c, kc, vc, q, kn, vn, mask = build(case, 9)
    c.table[0, 2] = 1 << 20
    o = c.attention(q, kn, vn)
    with pytest.raises(EagleError, match="BOUNDS"):
        c.status()
    keep = [i for i in range(100) if not 32 <= i < 48]
    see = ref.sees(3, len(keep), None, "cuda")
    want, tol = ref.attend(q[0], kc[0, keep], vc[0, keep], kn[0], vn[0], see)
    assert torch.all((o[0].double() - want).abs() <= tol)


@pytest.mark.parametrize("n,H", [(1, 8), (50, 8)], ids=["8rows", "400rows"])
def test_captured_calls_follow_the_lengths_and_streams(dev, n, H):
    """One graph of a write and the attention after it, replayed over growing lengths; and calls on a
    side stream whose outputs and workspaces belong to it."""
    B, Hk, D = 2, 1, 128
    case = (B, n, H, Hk, D, 16, [600, 600], "causal")
    c, kc, vc, q, kn, vn, _ = build(case, 10)
    lens = [5, 90]
    c.lengths.copy_(i32(lens))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    c.append(kn, vn)  # warm up
    c.attention(q, kn, vn)
    c.lengths.copy_(i32(lens))
    c.append(kc, vc, start=i32([0, 0]))
    c.lengths.copy_(i32(lens))
    with torch.cuda.graph(graph):
        c.append(kn, vn)
        o = c.attention(q)
    have = [kc[b, :lens[b]] for b in range(B)]
    have_v = [vc[b, :lens[b]] for b in range(B)]
    for _ in range(3):
        graph.replay()
        for b in range(B):
            have[b], have_v[b] = torch.cat([have[b], kn[b]]), torch.cat([have_v[b], vn[b]])
            want, tol = ref.attend(q[b], have[b], have_v[b], None, None,
                                   torch.ones(n, len(have[b]), dtype=torch.bool, device="cuda"))
            assert torch.all((o[b].double() - want).abs() <= tol)
    want = c.attention(q)
    side.wait_stream(torch.cuda.current_stream())
    got = [c.attention(q, stream=side) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(g, want) for g in got)


def test_two_graphs_side_by_side(dev):
    """Two captured calls over one cache, replayed on two streams: each graph holds its own
    workspace."""
    case = (4, 6, 16, 4, 128, 32, [3000, 1, 700, 50], "tree")
    c, kc, vc, q, kn, vn, mask = build(case, 11)
    want = c.attention(q, kn, vn, mask=mask), c.attention(kn, vn, kn)
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for args, kw in (((q, kn, vn), dict(mask=mask)), ((kn, vn, kn), {})):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.attention(*args, **kw))
        graphs.append(g)
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@pytest.mark.parametrize("n,H,D", [(3, 8, 128), (7, 6, 96), (30, 8, 128), (130, 4, 64)])
def test_calls_write_their_outputs_and_workspace_only(dev, n, H, D):
    case = (3, n, H, 2, D, 32, [900, 0, 77], "tree")
    c, kc, vc, q, kn, vn, mask = build(case, 13)
    want = c.attention(q, kn, vn, mask=mask)
    size, nbytes = q.numel(), c.attention_workspace_bytes(n, H)
    out = torch.full((size + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((nbytes + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    pages, table, lengths = c.pages.clone(), c.table.clone(), c.lengths.clone()
    got = c.attention(q, kn, vn, mask=mask, out=out[256:256 + size].view(q.shape), workspace=ws[256:256 + nbytes])
    assert torch.equal(got, want)
    assert torch.all(out[:256] == 7.0) and torch.all(out[256 + size:] == 7.0)
    assert torch.all(ws[:256] == 0xA5) and torch.all(ws[256 + nbytes:] == 0xA5)
    assert torch.equal(c.pages, pages) and torch.equal(c.table, table) and torch.equal(c.lengths, lengths)
    row = 2 * D
    back = torch.full((2, 3 * 901 * row + 512), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = (back[i, 256:256 + 3 * 901 * row].view(3, 901, 2, D) for i in range(2))
    c.read(out=(k, v))
    assert torch.all(back[:, :256] == 7.0) and torch.all(back[:, 256 + 3 * 901 * row:] == 7.0)
    for b, t in enumerate(case[6]):
        assert torch.all(k[b, t:] == 7.0) and torch.all(v[b, t:] == 7.0)
    assert torch.equal(c.pages, pages)


def test_refusals(dev):
    from eagle_speculative_decoding_draft_gb300 import KV4Cache
    for kw in (dict(batch=0), dict(head_dim=80), dict(page_size=24), dict(num_pages=0), dict(device="cpu"),
               dict(pages=torch.zeros(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            KV4Cache(**dict(dict(batch=2, kv_heads=2, head_dim=64, num_pages=4, max_pages=2, page_size=16), **kw))
    c = make_cache(2, 2, 64, 32, 16)
    g = gen(1)
    k, v, q = rows(g, 2, 3, 2, 64), rows(g, 2, 3, 2, 64), rows(g, 2, 3, 4, 64)
    mask, one = i32([[[1], [3], [7]]] * 2), i32([3, 3])
    cases = [
        (ValueError, lambda: c.append(k[:1], v[:1])), (ValueError, lambda: c.append(k, v[:, :2])),
        (ValueError, lambda: c.append(k[..., :32], v[..., :32])), (TypeError, lambda: c.append(k.float(), v.float())),
        (ValueError, lambda: c.append(k.cpu(), v.cpu())), (ValueError, lambda: c.append(k.transpose(2, 3), v.transpose(2, 3))),
        (TypeError, lambda: c.append(k, v, count=one.long())), (ValueError, lambda: c.append(k, v, count=one[:1])),
        (ValueError, lambda: c.append(k, v, start=one.cpu())), (ValueError, lambda: c.append(k, v, select=one)),
        (ValueError, lambda: c.append(k, v, select=i32([[0, 1]] * 4)[::2])),
        (ValueError, lambda: c.read(out=(k, v[:, :2]))), (ValueError, lambda: c.read(out=(k.half(), v.half()))),
        (ValueError, lambda: c.read(rows=4, out=(k, v))), (ValueError, lambda: c.read(start=one[:1])),
        (ValueError, lambda: c.attention(q[:1], k, v)), (ValueError, lambda: c.attention(q[:, :, :3], k, v)),
        (ValueError, lambda: c.attention(q[:, :0], k[:, :0], v[:, :0])), (TypeError, lambda: c.attention(q.float(), k, v)),
        (ValueError, lambda: c.attention(q, k)), (ValueError, lambda: c.attention(q, mask=mask)),
        (ValueError, lambda: c.attention(q, k[:, :2], v[:, :2])), (ValueError, lambda: c.attention(q, k, v, mask=mask[:1])),
        (TypeError, lambda: c.attention(q, k.float(), v.float())), (TypeError, lambda: c.attention(q, k, v, mask=mask.long())),
        (ValueError, lambda: c.attention(q, k, v, out=q[:, :2])),
        (ValueError, lambda: c.attention(q, k, v, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))),
    ]
    for i, (error, call) in enumerate(cases):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was not refused")
    c.status()
    assert c.lengths.tolist() == [0, 0]
    c.append(k, v)
    assert torch.equal(c.attention(q, k, v), c.attention(q, k, v, mask=mask))  # the same cache still works


def test_work_beyond_32_bits_is_refused(dev):
    """Before anything is launched: the sizes alone, whatever the pointers hold."""
    import ctypes
    from eagle_speculative_decoding_draft_gb300 import _lib
    lib, P = _lib.load(), ctypes.c_void_p
    c = _lib.KV4CacheStruct(1024, 128, 16, 16, 1 << 20, 256, 256, 256)
    assert lib.eagle_kv4_append(ctypes.byref(c), 1 << 22, 1, 1, P(256), P(256), 1 << 17, None, None, None, None, None) == 2
    assert lib.eagle_kv4_read(ctypes.byref(c), 1 << 22, 1, None, P(256), P(256), 1, None, None) == 2
    need = lib.eagle_kv4_attention_workspace_bytes(ctypes.byref(c), 1, 1024)
    assert lib.eagle_kv4_attention(ctypes.byref(c), 1 << 6, 1, 1024, P(256), 1 << 17, None, None, 0, None, P(256), P(256), need,
                                   None, None) == 2
    w = _lib.DecoderLayerWeights(256, 4, 2, 64, 256, 1e4, 1e-5, *[256] * 5)
    c = _lib.KV4CacheStruct(2, 64, 1024, 16, 1 << 20, 256, 256, 256)
    need = lib.eagle_decoder_layer_kv4_workspace_bytes(ctypes.byref(w), ctypes.byref(c), 128, 1)
    assert need > 0
    assert lib.eagle_decoder_layer_kv4(ctypes.byref(w), ctypes.byref(c), 128, 1, P(256), P(256), None, P(256), None, None, P(256),
                                       need, None, None) == 2


# ------------------------------------------------------------------------------------------------
# the decoder layer and a round of drafting
# ------------------------------------------------------------------------------------------------
LAYERS = [
    # B, n, P, h, H, Hk, D, I
    (2, 9, 37, 256, 4, 2, 64, 512),
    (1, 1, 0, 128, 2, 2, 128, 256),
    (3, 40, 70, 192, 3, 1, 32, 320),
    (2, 33, 150, 256, 8, 2, 128, 512),
]


@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "B%d_n%d_P%d_h%d_H%d_Hk%d_D%d" % c[:7])
def test_decoder_layer_over_the_cache(dev, case):
    """Against the layer's 64-bit restatement over the values that the cache stands for, within the
    bound of the layer over bf16 caches; the new keys and values are that layer's, bit for bit."""
    from eagle_speculative_decoding_draft_gb300.engine import DecoderLayer
    B, n, P, h, H, Hk, D, I = case
    w, d = layer(B=B, n=n, P=P, h=h, H=H, Hk=Hk, D=D, I=I, seed=1)
    rng = np.random.default_rng(1)
    parents, depths = random_tree(n, 5, rng)
    mask = np.broadcast_to(tree_mask(parents), (B, n, (n + 31) // 32)).copy()
    pos = np.broadcast_to(np.asarray(depths) + P, (B, n)).astype(np.int32).copy()
    g = lambda t: t.to(dev).contiguous()
    lay = DecoderLayer(g(w["w_qkv"]), g(w["w_o"]), g(w["w_norm"]), g(w["w_gu"]), g(w["w_d"]), H, Hk)
    c = make_cache(B, Hk, D, max(P, 1), 16)
    if P:
        c.append(g(w["k_cache"]), g(w["v_cache"]))
    mask_d, pos_d = torch.from_numpy(mask.view(np.int32)).to(dev), torch.from_numpy(pos).to(dev)
    out, kn, vn = lay.kv4(g(w["x"]), c, pos_d, mask_d, new_kv=True)
    c.status()
    held = dict(w, k_cache=ref.stands_for(w["k_cache"]), v_cache=ref.stands_for(w["v_cache"])) if P else w
    want, h1, absterms = reference_layer(held, d, parents, pos)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tolerance(h1, want, absterms))
    _, kb, vb = lay(g(w["x"]), g(w["k_cache"]) if P else None, g(w["v_cache"]) if P else None, pos_d, mask_d, new_kv=True)
    assert torch.equal(kn, kb) and torch.equal(vn, vb)
    assert torch.equal(lay.kv4(g(w["x"]), c, pos_d, mask_d), out)


def test_decoder_layer_without_a_mask_is_the_next_piece_of_a_prompt(dev):
    from eagle_speculative_decoding_draft_gb300.engine import DecoderLayer
    B, n, P, h, H, Hk, D, I = 2, 37, 50, 256, 8, 2, 64, 512
    w, d = layer(B=B, n=n, P=P, h=h, H=H, Hk=Hk, D=D, I=I, seed=4)
    g = lambda t: t.to(dev).contiguous()
    lay = DecoderLayer(g(w["w_qkv"]), g(w["w_o"]), g(w["w_norm"]), g(w["w_gu"]), g(w["w_d"]), H, Hk)
    c = make_cache(B, Hk, D, P, 16)
    c.append(g(w["k_cache"]), g(w["v_cache"]))
    pos = i32([[P + i for i in range(n)]] * B)
    chain = tree_mask(np.arange(n) - 1)  # every node's parent is the one before it
    chain = torch.from_numpy(np.broadcast_to(chain, (B, n, 2)).copy().view(np.int32)).to(dev)
    assert torch.equal(lay.kv4(g(w["x"]), c, pos), lay.kv4(g(w["x"]), c, pos, chain))
    c.status()


def test_decoder_layer_captured_with_changing_sizes(dev):
    """Workspaces hold anything: eager calls of other sizes between a graph's replays, one workspace of
    0xFF for several sizes, and two graphs replayed side by side."""
    from eagle_speculative_decoding_draft_gb300.engine import DecoderLayer
    B, h, H, Hk, D, I = 2, 256, 4, 2, 64, 512
    w, d = layer(B=B, n=70, P=30, h=h, H=H, Hk=Hk, D=D, I=I, seed=6)
    g = lambda t: t.to(dev).contiguous()
    lay = DecoderLayer(g(w["w_qkv"]), g(w["w_o"]), g(w["w_norm"]), g(w["w_gu"]), g(w["w_d"]), H, Hk)
    c = make_cache(B, Hk, D, 30, 16)
    c.append(g(w["k_cache"]), g(w["v_cache"]))
    x, pos = g(w["x"]), i32([[30 + i for i in range(70)]] * B)
    sizes = [70, 1, 9]
    args = [(x[:, :n].contiguous(), c, pos[:, :n].contiguous()) for n in sizes]
    graphs, outs = [], []
    for a in args[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):  # the first call of these sizes
            outs.append(lay.kv4(*a))
        graphs.append(graph)
    want = [lay.kv4(*a) for a in args]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        lay.kv4(*args[2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, v) for o, v in zip(outs, want))
    ws = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 1, 0):
        assert torch.equal(lay.kv4(*args[i], workspace=ws), want[i])
    c.status()


def test_rounds_of_drafting_over_the_cache(dev):
    """Three rounds as an engine makes them: the layer over the cache and a tree, a verify of that
    tree, and the accepted nodes' rows into the cache.  After each round the cache holds the accepted
    rows behind the earlier ones, and the layer's output follows the definition over them."""
    from eagle_speculative_decoding_draft_gb300.engine import DecoderLayer, verify_walk
    B, n, h, H, Hk, D, I, depth = 3, 12, 256, 8, 2, 64, 512, 4
    w, d = layer(B=B, n=n, P=20, h=h, H=H, Hk=Hk, D=D, I=I, seed=2)
    g = lambda t: t.to(dev).contiguous()
    lay = DecoderLayer(g(w["w_qkv"]), g(w["w_o"]), g(w["w_norm"]), g(w["w_gu"]), g(w["w_d"]), H, Hk)
    c = make_cache(B, Hk, D, 64, 16)
    prompt = [20, 3, 11]
    c.append(g(w["k_cache"]), g(w["v_cache"]), count=i32(prompt))
    held_k = [w["k_cache"][b, :t] for b, t in enumerate(prompt)]
    held_v = [w["v_cache"][b, :t] for b, t in enumerate(prompt)]
    rng = np.random.default_rng(3)
    for rnd in range(3):
        parents, depths = random_tree(n, depth, rng)
        tokens = np.tile(np.arange(n, dtype=np.int32), (B, 1))
        par = np.tile(np.asarray(parents, np.int32), (B, 1))
        want_child = rng.integers(0, n, size=(B, n)).astype(np.int32)  # the target's token at each node
        mask = np.broadcast_to(tree_mask(parents), (B, n, 1)).copy()
        lens = c.lengths.tolist()
        pos = np.stack([np.asarray(depths) + t for t in lens]).astype(np.int32)
        x = torch.randn(B, n, h, generator=torch.Generator().manual_seed(rnd)).to(torch.bfloat16)
        out, kn, vn = lay.kv4(g(x), c, torch.from_numpy(pos).to(dev), torch.from_numpy(mask.view(np.int32)).to(dev), new_kv=True)
        for b in range(B):
            one = dict(w, x=x[b:b + 1], k_cache=ref.stands_for(held_k[b])[None], v_cache=ref.stands_for(held_v[b])[None])
            want, h1, absterms = reference_layer(one, dict(d, B=1, P=lens[b]), parents, pos[b:b + 1])
            assert np.all(np.abs(out[b].double().cpu().numpy() - want[0]) <= tolerance(h1, want, absterms)[0])
        ver = verify_walk(i32(tokens), i32(par), i32(want_child), depth)
        c.append(kn, vn, select=ver["accept_nodes"])
        c.status()
        acc = (ver["accept_len"] + 1).tolist()
        assert c.lengths.tolist() == [t + a for t, a in zip(lens, acc)]
        got_k, got_v = c.read(rows=64, dtype=torch.float32)
        for b in range(B):
            path = ver["accept_nodes"][b, :acc[b]].long().cpu()
            held_k[b] = torch.cat([held_k[b], kn[b].cpu()[path]])
            held_v[b] = torch.cat([held_v[b], vn[b].cpu()[path]])
            m = len(held_k[b])
            assert torch.equal(got_k[b, :m].cpu(), ref.stands_for(held_k[b]).float())
            assert torch.equal(got_v[b, :m].cpu(), ref.stands_for(held_v[b]).float())
