"""Plain 64-bit forms of the serving operators, and caches to run them on.

A test draws keys and latents in token order; ``store`` puts them into pages as
include/basiskv.h lays them out, with NaN in every slot and page that holds no
token, so that a kernel which lets such a slot into a sum shows it.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from long_context_decode_basiskv_b200 import binding as bk


def swizzle(rows: torch.Tensor, on: bool) -> torch.Tensor:
    """[..., P, x]: the 16-byte chunk c of row j goes to chunk c ^ (j & mask)."""
    P, x = rows.shape[-2:]
    chunks = x // 8
    if not on:
        return rows
    mask = 7 if chunks % 8 == 0 else 3 if chunks % 4 == 0 else 1 if chunks % 2 == 0 else 0
    out = torch.empty_like(rows)
    for j in range(P):
        for c in range(chunks):
            to = c ^ (j & mask)
            out[..., j, 8 * to:8 * to + 8] = rows[..., j, 8 * c:8 * c + 8]
    return out


class Cache:
    """Keys and latents of `lengths` tokens in token order, and the paged cache that holds them."""

    def __init__(self, cfg, lengths, seed, max_pages=None, spare=3, kscale=0.8):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        P, H, d, r = cfg.page_size, cfg.num_kv_heads, cfg.head_dim, cfg.rank_v
        self.cfg, self.lengths = cfg, list(lengths)
        have = [-(-L // P) for L in lengths]
        self.max_pages = max_pages or max(1, max(have))
        phys = sum(have) + spare
        perm = rng.permutation(phys).astype(np.int32)
        table = np.full((len(lengths), self.max_pages), -1, np.int32)
        on = cfg.dtype == torch.bfloat16 and d % 16 == 0 and r % 16 == 0
        k_raw = torch.full((phys, H, P, d), float("nan"), dtype=cfg.dtype, device="cuda")
        c_lat = torch.full((phys, H, P, r), float("nan"), dtype=cfg.dtype, device="cuda")
        self.K, self.C, at = [], [], 0
        for b, L in enumerate(lengths):
            n = have[b]
            table[b, :n] = perm[at:at + n]
            at += n
            K = (torch.randn((L, H, d), generator=g, device="cuda") * kscale).to(cfg.dtype)
            C = torch.randn((L, H, r), generator=g, device="cuda").to(cfg.dtype)
            self.K.append(K)
            self.C.append(C)
            if n:
                ids = torch.from_numpy(table[b, :n].astype(np.int64)).cuda()
                for rows, pages in ((K, k_raw), (C, c_lat)):
                    full = torch.full((n * P, H, rows.shape[2]), float("nan"), dtype=cfg.dtype, device="cuda")
                    full[:L] = rows
                    pages[ids] = swizzle(full.reshape(n, P, H, -1).transpose(1, 2).contiguous(), on)
        self.paged = bk.PagedCache(cfg, phys, torch.from_numpy(table), torch.tensor(lengths, dtype=torch.int32))
        self.paged.k_raw, self.paged.c_lat = k_raw, c_lat


def attention(K, C, q, scale, softcap=0.0, window=0, slopes=None, prefix=0, hidden_keys=()):
    """One sequence in 64 bits: q [n, Hq, d] -> o [n, Hq, r], lse [n, Hq], and the sums of w |C|
    that rounding errors are measured by."""
    n, Hq, _ = q.shape
    L, H, r = C.shape
    G = Hq // H
    o = torch.zeros((n, Hq, r), dtype=torch.float64, device=q.device)
    size = torch.zeros_like(o)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    if L == 0:
        return o, lse, size
    i = torch.arange(L - n, L, device=q.device)[:, None]
    j = torch.arange(L, device=q.device)[None, :]
    see = j <= i
    if window:
        see &= i - j < window
    see = see | (j < prefix)
    for x in hidden_keys:
        see[:, x] = False
    for h in range(Hq):
        s = q[:, h].double() @ K[:, h // G].double().T * scale
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        if slopes is not None:
            s = s - slopes[h].double() * (i - j).abs()
        s = torch.where(see, s, -math.inf)
        m = s.amax(1, keepdim=True)
        w = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
        l = w.sum(1, keepdim=True)
        some = (l > 0)
        w = torch.where(some, w / torch.where(some, l, 1.0), 0.0)
        o[:, h] = w @ C[:, h // G].double()
        size[:, h] = w @ C[:, h // G].double().abs()
        lse[:, h] = torch.where(some, torch.where(m == -math.inf, 0.0, m) + torch.log(l), -math.inf)[:, 0]
    return o, lse, size


# Bounds of o_lat and lse against 64 bits, with |s| the size of a score and w its weight:
#   a score: products exact (bf16) or rounded (fp32), d sums of fp32: about sqrt(d) 2^-24 sum|q k| scale,
#     below 2^-19 at these sizes (sum|q k| scale < 40); scale, maximum and exponent: |s| 2^-23 < 2^-17 at |s| < 60;
#     tanh: 2e-7 cap < 2^-16 (cap <= 50); exp2: 2^-22
#   a weight as hi + lo bf16: 2^-16;  sums of weights and products: below 2^-18
# Together below 2^-14 of sum w |C| for every element, and (independent, most far below their bounds) a
# quarter of that in the 2-norm.  lse: the score's part alone.
ELEMENT = 2.0 ** -14
NORM = 2.0 ** -16


def assert_attention(got_o, got_lse, want_o, want_lse, size, what):
    err = (got_o.double() - want_o).abs()
    assert torch.isfinite(got_o).all(), f"{what}: not finite"
    assert (err <= ELEMENT * size.amax(-1, keepdim=True) + 1e-30).all(), f"{what}: {(err / size.clamp(min=1e-30)).max()}"
    assert err.norm() <= NORM * size.norm() + 1e-30, f"{what}: norm {float(err.norm() / size.norm())}"
    if got_lse is not None:
        none = want_lse == -math.inf
        assert torch.equal(got_lse == -math.inf, none), f"{what}: empty rows"
        e = torch.where(none, 0.0, (got_lse.double() - torch.where(none, 0.0, want_lse)).abs())
        assert (e <= 2.0 ** -15 + 2.0 ** -22 * want_lse.abs().clamp(max=1e6)).all(), f"{what}: lse {float(e.max())}"


def rotate(x, pos, inv_freq, mscale, layout):
    """x [n, H, d] at positions pos [n], in 64 bits; also the sizes |u| + |v| of every element's pair."""
    y = x.double().clone()
    size = torch.zeros_like(y)
    f = torch.tensor(inv_freq, dtype=torch.float64, device=x.device)
    a = pos.double()[:, None, None] * f
    rot = 2 * len(inv_freq)
    if layout == "half":
        i0, i1 = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        i0, i1 = slice(0, rot, 2), slice(1, rot, 2)
    u, v = y[..., i0].clone(), y[..., i1].clone()
    y[..., i0], y[..., i1] = (u * a.cos() - v * a.sin()) * mscale, (v * a.cos() + u * a.sin()) * mscale
    size[..., i0] = size[..., i1] = (u.abs() + v.abs()) * mscale
    return y, size
