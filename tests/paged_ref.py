"""Caches, tables and 64-bit references for the paged-cache tests."""

from __future__ import annotations

import math

import numpy as np
import torch

import attn_check as ac
import oracle

# |lse error|: a score is a sum of at most 128 products in 32 bits, |sum of
# terms| * scale about 7 for normal inputs, so 128 * 2^-24 * 7 = 5.5e-5; the
# row sum takes up to 2500 additions per chain, 2500 * 2^-24 = 1.5e-4.
TOL_LSE = 3e-4


def make_cache(seed, Hkv, d, P, lens, dtype, prefix=0, spare=4, table_slack=1, garbage=float("nan")):
    """A pool of pages in shuffled order holding sequences of the given lengths
    (the first `prefix` tokens, a multiple of P, in the same pages for all);
    slots that hold no token, and spare pages, hold `garbage`.  Returns
    k_cache, v_cache, table, lens."""
    g = torch.Generator("cpu").manual_seed(seed)
    shared = prefix // P
    own = [max(0, -(-L // P) - shared) for L in lens]
    width = shared + max(own) + table_slack
    count = shared + sum(own) + spare
    perm = torch.randperm(count, generator=g).to(torch.int32)
    kc = torch.full((count, Hkv, P, d), garbage).to(dtype)
    vc = torch.full((count, Hkv, P, d), garbage).to(dtype)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    used = shared
    first_live = next((b for b, L in enumerate(lens) if L > 0), 0)
    for b, (L, n) in enumerate(zip(lens, own)):
        if L == 0:
            continue
        table[b, :shared] = perm[:shared]
        table[b, shared:shared + n] = perm[used:used + n]
        used += n
        for i in range(-(-max(L, prefix) // P)):
            page, m = int(table[b, i]), min(P, max(L, prefix) - i * P)
            if i < shared and b > first_live:
                continue
            kc[page, :, :m] = torch.randn((Hkv, m, d), generator=g).to(dtype)
            vc[page, :, :m] = torch.randn((Hkv, m, d), generator=g).to(dtype)
    return kc, vc, table, torch.tensor(lens, dtype=torch.int32)


def attention(q, kc, vc, table, lens, new_lens, scale):
    """The fp64 oracle, sequence by sequence: (O, lse, sum p |v|) with O = 0,
    lse = -inf in rows of idle sequences and behind the new tokens."""
    B, Hq, N, d = q.shape
    o, lse, o_abs = np.zeros((B, Hq, N, d)), np.full((B, Hq, N), -np.inf), np.zeros((B, Hq, N, d))
    for b in range(B):
        L, n = int(lens[b]), int(new_lens[b])
        if L == 0 or n == 0:
            continue
        args = (table[b:b + 1].numpy(), np.array([L]), scale)
        pages = -(-L // kc.shape[2])
        kb, vb = kc[table[b, :pages].long()], vc[table[b, :pages].long()]      # only its own pages
        idx = np.arange(pages)[None]
        clean = lambda x: torch.nan_to_num(x.double(), nan=0.0, posinf=0.0, neginf=0.0)
        o[b, :, :n], lse[b, :, :n] = (x[0] for x in oracle.decode_paged(q[b:b + 1, :, :n].contiguous(), clean(kb), clean(vb),
                                                                         idx, *args[1:]))
        o_abs[b, :, :n] = oracle.decode_paged(q[b:b + 1, :, :n].contiguous(), clean(kb), clean(vb).abs(), idx,
                                              *args[1:])[0][0]
    return o, lse, o_abs


def check_attention(o, lse, ref, dtype, new_lens):
    """O within the rounding bound of the 16-bit path, lse within TOL_LSE, in
    the rows of new tokens; every one of them finite (or -inf where the
    reference is)."""
    o_r, lse_r, o_abs = ref
    o, lse = o.cpu(), lse.cpu()
    for b, n in enumerate(new_lens):
        rows = (b, slice(None), slice(0, int(n)))
        assert bool(torch.isfinite(o[rows].float()).all()), f"sequence {b}: O is not finite"
        ac.check_o_rounding_bound(o[rows], o_r[rows], dtype, o_abs[rows], what=f"O of sequence {b}")
        got, want = lse[rows].double().numpy(), lse_r[rows]
        empty = np.isneginf(want)
        assert np.array_equal(np.isneginf(got), empty), f"sequence {b}: empty rows"
        err = np.abs(got[~empty] - want[~empty]).max(initial=0.0)
        assert err <= TOL_LSE, f"lse of sequence {b}: {err:.2e}"


def rotated(x, pos, inv_freq, interleaved):
    """x [heads, tokens, d] turned by position in 64 bits; also the bound
    |x| + |y| of each feature's pair."""
    x = x.double()
    rot = 2 * len(inv_freq)
    a = pos.double()[:, None] * inv_freq.double()[None]
    c, s = a.cos(), a.sin()
    y, mag = x.clone(), x.abs()
    i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    u, w = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = u * c - w * s, u * s + w * c
    mag[..., i0] = mag[..., i1] = u.abs() + w.abs()
    return y, mag


def check_rotated(got, want, mag, what):
    """Half a step of the I/O type, and 2^-19 of the pair's magnitude for the
    32-bit sine, cosine (angle rounded to 2^-24 of a half turn, 2 ulp each)
    and products."""
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * half    # half a subnormal step
    err = (got.double() - want).abs()
    bound = half * want.abs() * (1 + half) + 2.0 ** -19 * mag + tiny
    assert bool((err <= bound).all()), f"{what}: off by {float((err - bound).max()):.2e} above the bound"


def inv_freq(rot, base=10000.0):
    h = rot // 2
    return (base ** (-torch.arange(h, dtype=torch.float64) / max(h, 1))).float()


def default_scale(d):
    return 1.0 / math.sqrt(d)
