"""The 4-bit cache's definition in 64 bits, written apart from the library: the values a bf16 row
stands for once cached, attention over them, and how far the library's arithmetic may be off."""
import math

import torch


def half_grid(x, up):
    """x (fp64) to a multiple of its fp16 step, down or up (normal and subnormal)."""
    e = torch.frexp(x).exponent.clamp(min=-13).long()  # |x| in [2^(e-1), 2^e)
    step = ((e - 11 + 1023) << 52).view(torch.float64)
    return (torch.ceil(x / step) if up else torch.floor(x / step)) * step


def parts(x):
    """(m, s, c) of bf16 rows [..., D]: m and s [..., D/32, 1], c [..., D/32, 32], all fp64."""
    g = x.double().unflatten(-1, (-1, 32))
    bad = ~((g.abs() <= 32768).all(-1, keepdim=True))
    z = torch.where(bad, 0.0, g)
    m = half_grid(z.amin(-1, keepdim=True), up=False)
    s = half_grid((z.amax(-1, keepdim=True) - m) / 15, up=True)
    c = torch.where(s > 0, torch.round((z - m) / torch.where(s > 0, s, 1.0)), 0.0).clamp(0, 15)
    nan = torch.full_like(m, math.nan)
    return torch.where(bad, nan, m), torch.where(bad, nan, s), c


def stands_for(x):
    m, s, c = parts(x)
    return (m + s * c).flatten(-2)


def size_of(x):
    """|m| + s c: the terms whose roundings the value sums carry."""
    m, s, c = parts(x)
    return (m.abs() + s * c).flatten(-2)


def sees(n, t, mask_row_bits, device):
    """[n][t + n]: cached positions, then the new keys that mask bits mark (None: causal)."""
    new = torch.ones(n, n, dtype=torch.bool, device=device).tril()
    if mask_row_bits is not None:
        j = torch.arange(n, device=device)
        new = ((mask_row_bits[:, j // 32].long() >> (j % 32)) & 1).bool()
    return torch.cat([torch.ones(n, t, dtype=torch.bool, device=device), new], 1)


def attend(q, kc, vc, kn, vn, see):
    """One request.  q [n][H][D]; kc, vc the bf16 rows that were cached [t][Hk][D]; kn, vn the new
    rows [n][Hk][D] or None; see [n][t (+ n)].  Returns (o, tol) in fp64.

    tol, from the library's arithmetic:
      output rounding            2^-8 |o|                       (half a bf16 step)
      p and p s to fp16          2 x 2^-11 of the sum of p (|m| + s c)   (half fp16 steps)
      scores in fp32             a sum of D products and D / 32 + 2 more terms, each step at most
                                 2^-22 (accumulation that truncates) of the sum of magnitudes A: the
                                 exponent is off by delta = (D + 16) 2^-22 A at most, p relatively by
                                 as much, numerator and denominator: 2 delta
      exponentials               2^-21 relative each
      fp16 range                 products below 2^-14 lose at most 2^-25 of a scale where the largest
                                 p is 2^9 or more (2^0 where some s is 16 or more): 15 N 2^-34 or 2^-25
    More than 16 query rows a kv head go through tiles of fp16 values instead:
      cached k, v to fp16        2^-11 of their size and 2^-25: the exponent is off by 2^-11 A +
                                 2^-25 sum |q| / sqrt(D) more, v by 2^-11 |v| + 2^-25
      new k, v to fp16           exact but for 2^-25 below 2^-14: the same 2^-25 terms
      p to fp16                  2^-11 |v|; below 2^-14 at most 2^-25 where the largest is 2^4 or
                                 more (a reference puts a row's largest p at 2^4, later ones pass
                                 it): N 2^-29 of the largest |v|
    """
    n, H, D = q.shape
    Hk = kc.shape[1]
    tiles = n * H // Hk > 16
    k, v, size, ksize = stands_for(kc), stands_for(vc), size_of(vc), size_of(kc)
    steep = bool((parts(vc)[1] >= 16).any()) if vc.numel() else False
    if kn is not None:
        k, v = torch.cat([k, kn.double()]), torch.cat([v, vn.double()])
        size, ksize = torch.cat([size, vn.double().abs()]), torch.cat([ksize, kn.double().abs()])
    if k.shape[0] == 0:
        return torch.zeros_like(q, dtype=torch.float64), torch.zeros_like(q, dtype=torch.float64)
    rep = H // Hk
    kh, vh = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    z = torch.einsum("nhd,thd->hnt", q.double(), kh) / math.sqrt(D)
    z = torch.nan_to_num(z, nan=0.0).masked_fill(~see, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    p = torch.where(see, p, 0.0)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total == 0, 0.0, p / total)
    seen_v = torch.where(see.any(0)[:, None, None], vh, 0.0)
    o = torch.einsum("hnt,thd->nhd", p, torch.nan_to_num(seen_v, nan=0.0, posinf=0.0, neginf=0.0))
    # a cached group that is NaN: its dims of every row that sees it (a key's: the whole row)
    see_f = see.double()
    o[torch.einsum("nt,thd->nhd", see_f, torch.isnan(vh).double()) > 0] = math.nan
    o[torch.einsum("nt,th->nh", see_f, torch.isnan(kh).any(-1).double()) > 0] = math.nan
    A = torch.einsum("nhd,thd->hnt", q.double().abs(), torch.nan_to_num(ksize.repeat_interleave(rep, 1))) / math.sqrt(D)
    delta = (D + 16) * 2.0 ** -22 * torch.where(see, A, 0.0).amax(-1, keepdim=True)
    if tiles:
        kabs = torch.nan_to_num(k[:kc.shape[0]].abs().repeat_interleave(rep, 1))
        Ac = torch.einsum("nhd,thd->hnt", q.double().abs(), kabs) / math.sqrt(D)
        worst = torch.where(see[:, :kc.shape[0]], Ac, 0.0).amax(-1, keepdim=True) if kc.shape[0] else 0.0
        delta = delta + 2.0 ** -11 * worst + 2.0 ** -25 * q.double().abs().sum(-1).T[..., None] / math.sqrt(D)
        vfin = torch.nan_to_num(seen_v, posinf=0.0, neginf=0.0).abs()
        mag = torch.einsum("hnt,thd->nhd", p * (2.0 ** -10 + 2.0 ** -19 + 2 * delta), vfin)
        big = vfin.amax(0)[None]
        return o, 2.0 ** -8 * torch.nan_to_num(o).abs() * 1.001 + mag + 2.0 ** -25 + k.shape[0] * 2.0 ** -29 * big
    mag = torch.einsum("hnt,thd->nhd", p * (2.0 ** -10 + 2.0 ** -19 + 2 * delta),
                       torch.nan_to_num(size.repeat_interleave(rep, 1), posinf=0.0))
    tol = 2.0 ** -8 * torch.nan_to_num(o).abs() * 1.001 + mag + 15 * k.shape[0] * (2.0 ** -25 if steep else 2.0 ** -34)
    return o, tol


def rounded_off(x):
    """What over 16 query rows a new key's or value's elements may lose: 2^-25, half of fp16's last step, where an
    element below 2^-17 (those above are whole steps: 8 bits of bf16) has one of 2^-12 .. 65504 as the largest of its
    aligned 8 neighbours."""
    a = x.double().abs().unflatten(-1, (-1, 8))
    most = a.amax(-1, keepdim=True)
    return torch.where((a > 0) & (a < 2.0 ** -17) & (most >= 2.0 ** -12) & (most <= 65504), 2.0 ** -25, 0.0).flatten(-2)


def relative_tolerance(q, kc, vc, kn, vn, see, o):
    """How far the attention of one request may be off where sizes are far from 1: terms that follow the
    sizes of what a row sees, with none of an absolute size.  Arguments as attend's; o its result.
      output rounding            2^-8 |o|
      scores in fp32             delta = (D + 16) 2^-22 of the sum of magnitudes, numerator and denominator;
                                 over 16 rows cached keys are fp16 values: 2^-11 of their magnitudes more
      p (and p s) to fp16        2 x 2^-11 of the sum of p (|m| + s c); new keys' p is bf16 hi + lo: less
      new keys and values        over 16 rows what rounded_off says
      fp16 range, cached keys    up to 16 rows: a row's largest p is 2^9 or more, the largest s is scaled to 8 or more
                                 (or by 2^15): 15 codes off by 2^-25 are 15 2^-37 of it (or 15 2^-49); over 16 rows the
                                 largest p is 2^4 or more: 2^-29 of the largest value
    """
    n, H, D = q.shape
    Hk = kc.shape[1]
    rep, tiles, t = H // Hk, n * H // Hk > 16, kc.shape[0]
    k, size, ksize = stands_for(kc), size_of(vc), size_of(kc)
    if kn is not None:
        k, size, ksize = torch.cat([k, kn.double()]), torch.cat([size, vn.double().abs()]), torch.cat([ksize, kn.double().abs()])
    kh, size, ksize = (x.repeat_interleave(rep, 1) for x in (k, size, ksize))
    z = torch.einsum("nhd,thd->hnt", q.double(), kh) / math.sqrt(D)
    p = torch.softmax(z.masked_fill(~see, -math.inf), -1).nan_to_num(0.0)
    A = torch.where(see, torch.einsum("nhd,thd->hnt", q.double().abs(), ksize), 0.0) / math.sqrt(D)
    delta = (D + 16) * 2.0 ** -22 * A.amax(-1, keepdim=True)
    if tiles and t:
        delta = delta + 2.0 ** -11 * A[..., :t].amax(-1, keepdim=True)
    held = torch.zeros_like(size)  # what the tiles may round off each new value
    if tiles and kn is not None:
        lost_k = torch.cat([torch.zeros_like(kc.double()), rounded_off(kn)]).repeat_interleave(rep, 1)
        held = torch.cat([torch.zeros_like(kc.double()), rounded_off(vn)]).repeat_interleave(rep, 1)
        B = torch.where(see, torch.einsum("nhd,thd->hnt", q.double().abs(), lost_k), 0.0) / math.sqrt(D)
        delta = delta + B.amax(-1, keepdim=True)
    tol = 2.0 ** -8 * 1.001 * o.abs() + torch.einsum("hnt,thd->nhd", p * (2.0 ** -10 + 2.0 ** -19 + 2 * delta), size)
    tol = tol + torch.einsum("hnt,thd->nhd", p, held)
    if t and tiles:
        tol = tol + t * 2.0 ** -29 * size[:t].amax(0)[None]
    elif t:
        step = parts(vc)[1].amax((0, 2, 3)).repeat_interleave(rep)[None, :, None]  # of a kv head
        tol = tol + 15 * t * torch.clamp(2.0 ** -37 * step, min=2.0 ** -49)
    return tol
