"""Plain fp64 references of the paged-cache attention operators, and input makers (CPU torch)."""
from __future__ import annotations

import math

import torch

HALF_STEP = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
P_HALF_STEP = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -11}  # the weights' rounding: bf16 or fp16


def make(Hkv, D, page, kv, lens, seed=0, extra_pages=3, fill=math.nan):
    """A cache on the CPU: K, V pools (rows no sequence owns hold `fill`), page_table, lens,
    scales, and the keys and values of each sequence as fp64 [len, Hkv, D]."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages = [-(-n // page) for n in lens]
    width, total = max([1] + pages), sum(pages) + extra_pages
    ids = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)  # unused entries are never read
    K = torch.full((total, Hkv, page, D), fill)
    V = torch.full((total, Hkv, page, D), fill)
    dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    at = 0
    for b, n in enumerate(lens):
        for i in range(pages[b]):
            table[b, i] = ids[at]
            rows = min(page, n - i * page)
            for pool in (K, V):
                x = torch.randn((Hkv, rows, D), generator=g)
                pool[ids[at], :, :rows] = x if kv == "bf16" else x * 60.0
            at += 1
    K, V = K.to(dtype), V.to(dtype)
    if kv == "bf16":
        ks = vs = torch.ones(Hkv)
    else:
        ks = (1 + torch.rand(Hkv, generator=g)) / 64
        vs = (1 + torch.rand(Hkv, generator=g)) / 64
    return dict(K=K, V=V, table=table, lens=torch.tensor(lens, dtype=torch.int32), ks=ks, vs=vs,
                page=page, kv=kv)


def rows_of(c, which, b, n):
    """fp64 [n, Hkv, D]: the first n keys or values of sequence b."""
    page = c["page"]
    ids = c["table"][b, :-(-n // page)].long()
    x = c[which].float().double()[ids].transpose(1, 2).reshape(-1, *c[which].shape[1::2])[:n]
    return x * (c["ks"] if which == "K" else c["vs"]).double()[:, None]


def attend(c, b, q, hi, lo, scale):
    """q fp64 [Hq, D] over keys [lo, hi) of sequence b: (out, lse, sum of p |v|, largest
    scale * sum |q k|)."""
    Hq, D = q.shape
    Hkv = c["K"].shape[1]
    if hi <= lo:
        return (torch.zeros(Hq, D, dtype=torch.float64), torch.full((Hq,), -math.inf).double(),
                torch.zeros(Hq, D, dtype=torch.float64), torch.zeros(Hq, dtype=torch.float64))
    k = rows_of(c, "K", b, hi)[lo:].repeat_interleave(Hq // Hkv, 1)
    v = rows_of(c, "V", b, hi)[lo:].repeat_interleave(Hq // Hkv, 1)
    s = torch.einsum("hd,jhd->hj", q, k) * scale
    big = torch.einsum("hd,jhd->hj", q.abs(), k.abs()).amax(1) * scale
    p = torch.softmax(s, 1)
    return (torch.einsum("hj,jhd->hd", p, v), torch.logsumexp(s, 1),
            torch.einsum("hj,jhd->hd", p, v.abs()), big)


def out_tolerance(out, spread, kv):
    """The output's rounding, the weights' rounding, and the fp32 of scores, exponentials and
    sums (relative 2^-13 of the weights: 128 products of magnitude up to 2^3 at 2^-24 each, as
    the exponent of e, with a margin of 4)."""
    return out.abs() * HALF_STEP["bf16"] + spread * (P_HALF_STEP[kv] + 2.0 ** -12) + 1e-30


def lse_tolerance(lse, big, D):
    return big * D * 2.0 ** -23 + (1 + lse.abs()) * 2.0 ** -18


def rotate(x, pos, rot, interleaved, freq):
    """x fp64 [T, heads, D]; pos [T]; freq [rot / 2]: rotated, fp64."""
    y = x.clone()
    ang = pos.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64)
    c, s = ang.cos(), ang.sin()
    i = torch.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y
