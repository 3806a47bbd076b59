"""The paged-cache operators on the GPU against 64-bit references: append with
position rotation, the forward pass over the cache and decode behind a shared
prefix; their run together as a server uses them; captured, replayed and on
other streams; bad lengths and table entries."""

import numpy as np
import pytest
import torch

import oracle
import paged_ref as pr
from exact_io_aware_bwd_b200 import binding
from exact_io_aware_bwd_b200.build import build

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    binding.load()


def ok():
    status = binding.fa_get_device_status()
    assert status == binding.FA_OK, binding.fa_status_string(status)


# ------------------------------------------------------------------- append

APPEND = [
    # B, Hq, Hkv, N, d, P, rot, interleaved, layout, lens, new_lens, dtype
    (1, 8, 2, 1, 128, 16, 128, False, "dense", (1,), None, BF),
    (1, 32, 8, 1, 128, 64, 128, True, "token", (1_000_000,), None, BF),
    (3, 4, 4, 1, 64, 32, 32, False, "token", (33, 1, 64), None, FP),
    (2, 6, 2, 37, 64, 16, 64, True, "dense", (37, 60), None, BF),
    (4, 5, 5, 50, 128, 128, 64, False, "token", (50, 20, 0, 300), (50, 3, 0, 17), FP),
    (2, 28, 4, 333, 128, 32, 16, True, "token", (333, 500), (332, 1), BF),
    (5, 8, 1, 9, 64, 16, 0, False, "dense", (9, 10, 11, 24, 25), None, FP),
    (1, 16, 16, 700, 64, 64, 48, False, "dense", (700,), None, BF),
]


def append_case(case, seed=3):
    B, Hq, Hkv, N, d, P, rot, inter, layout, lens, new, dtype = case
    g = torch.Generator("cpu").manual_seed(seed + d + N)
    width = max(1, max(-(-L // P) for L in lens))
    # far positions: only the pages that the new tokens touch exist
    n_of = [N if new is None else n for n in (new or [None] * B)]
    touched = [sorted({p // P for p in range(L - n, L)}) for L, n in zip(lens, n_of)]
    count = sum(len(t) for t in touched) + 3
    perm = torch.randperm(count, generator=g).to(torch.int32).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    for b, pages in enumerate(touched):
        for i in pages:
            table[b, i] = perm.pop()
    if layout == "token":
        x = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g).to(dtype).transpose(1, 2)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        q, k, v = (torch.randn((B, h, N, d), generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
    kc, vc = (torch.randn((count, Hkv, P, d), generator=g).to(dtype) for _ in range(2))
    return q, k, v, kc, vc, table, torch.tensor(lens, dtype=torch.int32), \
        None if new is None else torch.tensor(new, dtype=torch.int32), n_of


def append_reference(q, k, v, kc, vc, table, lens, n_of, freq, inter, P):
    """[(got-index, want, magnitude)] of every written row, and the masks of untouched slots."""
    touched = torch.zeros(kc.shape[0], P, dtype=torch.bool)
    rows = []
    for b, n in enumerate(n_of):
        L = int(lens[b])
        if L == 0 or n == 0:
            continue
        pos = torch.arange(L - n, L)
        page, slot = table[b].long()[pos // P], pos % P
        touched[page, slot] = True
        rows.append((b, n, page, slot, pr.rotated(q[b, :, :n], pos, freq, inter), pr.rotated(k[b, :, :n], pos, freq, inter)))
    return rows, touched


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"B{c[0]}-H{c[1]}/{c[2]}-N{c[3]}-d{c[4]}-P{c[5]}-rot{c[6]}"
                         f"-{'il' if c[7] else 'hs'}-{c[8]}")
def test_append(case):
    B, Hq, Hkv, N, d, P, rot, inter, layout, _, _, dtype = case
    q, k, v, kc, vc, table, lens, new, n_of = append_case(case)
    freq = pr.inv_freq(rot)
    dev = lambda t: None if t is None else t.to(DEV)
    if layout == "token":  # keep the packed rows packed on the device
        x = torch.cat([q, k, v], 1).transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
        qd, kd, vd = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        assert N == 1 or not qd.is_contiguous()
    else:
        qd, kd, vd = dev(q), dev(k), dev(v)
    kcd, vcd = dev(kc), dev(vc)
    q_out = torch.full((B, Hq, N, d), 7.0, dtype=dtype, device=DEV)
    k_out = torch.full((B, Hkv, N, d), 7.0, dtype=dtype, device=DEV)
    binding.fa_append_paged(qd, kd, vd, q_out, k_out, kcd, vcd, dev(table), dev(lens), dev(new),
                            dev(freq) if rot else None, inter)
    ok()
    rows, touched = append_reference(q, k, v, kc, vc, table, lens, n_of, freq, inter, P)
    q_out, k_out, kcd, vcd = q_out.cpu(), k_out.cpu(), kcd.cpu(), vcd.cpu()
    for b, n, page, slot, (qr, qm), (kr, km) in rows:
        pr.check_rotated(q_out[b, :, :n], qr, qm, "q")
        pr.check_rotated(k_out[b, :, :n], kr, km, "k")
        got = kcd[page, :, slot].transpose(0, 1)
        assert torch.equal(got, k_out[b, :, :n])
        assert torch.equal(vcd[page, :, slot].transpose(0, 1), v[b, :, :n])
    # rows behind the new tokens and slots of no new token keep what they held
    for b, n in enumerate(n_of):
        n = 0 if int(lens[b]) == 0 else n
        assert bool((q_out[b, :, n:] == 7).all()) and bool((k_out[b, :, n:] == 7).all())
    for got, had in ((kcd, kc), (vcd, vc)):
        keep = ~touched[:, None, :, None].expand_as(had)
        assert torch.equal(got[keep], had[keep])


def test_append_in_place_and_without_queries():
    case = APPEND[3]
    B, Hq, Hkv, N, d, P, rot, inter, layout, _, _, dtype = case
    q, k, v, kc, vc, table, lens, new, n_of = append_case(case)
    freq = pr.inv_freq(rot)
    t = [x.to(DEV) for x in (q, k, v, kc, vc, table, lens, freq)]
    ref = [x.clone() for x in t]
    q_out, k_out = torch.empty_like(t[0]), torch.empty_like(t[1])
    binding.fa_append_paged(ref[0], ref[1], ref[2], q_out, k_out, ref[3], ref[4], ref[5], ref[6], None, ref[7], inter)
    binding.fa_append_paged(t[0], t[1], t[2], t[0], t[1], t[3], t[4], t[5], t[6], None, t[7], inter)
    kc2, vc2 = kc.to(DEV), vc.to(DEV)
    assert binding.cache_append(None, k.to(DEV), v.to(DEV), kc2, vc2, t[5], t[6], t[7], interleaved=inter) is None
    ok()
    assert torch.equal(t[0], q_out) and torch.equal(t[1], k_out)
    for got in (t[3], kc2):
        assert torch.equal(got, ref[3])
    for got in (t[4], vc2):
        assert torch.equal(got, ref[4])


def test_append_from_rows_with_odd_or_zero_strides():
    """One token a sequence: its token stride is never stepped over, whatever
    it says; and keys expanded from one head have a head stride of 0."""
    B, Hq, Hkv, d, P = 3, 4, 2, 64, 16
    g = torch.Generator().manual_seed(8)
    flat = torch.randn((B, Hq, d), generator=g).to(BF).to(DEV)
    q = flat.as_strided((B, Hq, 1, d), (Hq * d, d, 3, 1))
    k1 = torch.randn((B, 1, 1, d), generator=g).to(BF).to(DEV)
    k = k1.expand(B, Hkv, 1, d)
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None]
    lens = torch.tensor([1, 5, 16], dtype=torch.int32, device=DEV)
    freq = pr.inv_freq(d).to(DEV)
    caches = [torch.zeros((B, Hkv, P, d), dtype=BF, device=DEV) for _ in range(4)]
    a = binding.cache_append(q, k, k, caches[0], caches[1], table, lens, freq)
    b = binding.cache_append(q.contiguous(), k.contiguous(), k.contiguous(), caches[2], caches[3], table, lens, freq)
    ok()
    assert torch.equal(a, b) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    assert bool((caches[0].abs().sum((1, 2, 3)) > 0).all())


def test_append_far_positions_keep_their_angle():
    """Positions up to the largest a table can hold: the angle is taken in 64
    bits, so a far position is turned as exactly as a near one."""
    for L in (1 << 20, (1 << 31) - 129):
        P, d, Hkv = 128, 64, 1
        table = torch.full((1, -(-L // P)), -1, dtype=torch.int32)
        table[0, (L - 1) // P] = 0
        k = torch.randn((1, Hkv, 1, d), generator=torch.Generator().manual_seed(4)).to(FP)
        kc = torch.zeros((1, Hkv, P, d), dtype=FP, device=DEV)
        vc = torch.zeros_like(kc)
        freq = pr.inv_freq(d)
        binding.fa_append_paged(None, k.to(DEV), k.to(DEV), None, None, kc, vc, table.to(DEV),
                                torch.tensor([L], dtype=torch.int32, device=DEV), None, freq.to(DEV))
        ok()
        want, mag = pr.rotated(k[0], torch.tensor([L - 1]), freq, False)
        pr.check_rotated(kc[0, :, (L - 1) % P].cpu()[:, None], want, mag, f"k at {L - 1}")


# ------------------------------------------------------- forward over the cache

PAGED = [
    # Hq, Hkv, N, d, P, lens, new_lens, dtype
    (2, 2, 1, 64, 16, (1,), None, BF),
    (8, 2, 40, 128, 16, (340,), None, BF),
    (8, 2, 128, 128, 128, (128, 129), None, FP),
    (4, 4, 129, 64, 32, (129, 700), None, FP),
    (6, 2, 300, 128, 64, (300, 1000, 555), None, BF),
    (5, 5, 257, 64, 16, (257, 256, 300), (257, 100, 3), FP),
    (8, 1, 33, 128, 32, (4000, 33), None, BF),
    (28, 4, 64, 64, 64, (64, 2000, 0, 63), (64, 64, 0, 1), BF),
    (12, 12, 200, 64, 128, (0, 210, 199), (200, 200, 199), FP),
    (32, 8, 16, 128, 64, (9000, 16, 300), None, FP),
]


@pytest.mark.parametrize("case", PAGED, ids=lambda c: f"H{c[0]}/{c[1]}-N{c[2]}-d{c[3]}-P{c[4]}-L{max(c[5])}")
def test_fwd_paged(case):
    Hq, Hkv, N, d, P, lens, new, dtype = case
    B = len(lens)
    kc, vc, table, tl = pr.make_cache(N + d + P, Hkv, d, P, lens, dtype)
    g = torch.Generator("cpu").manual_seed(N)
    q = torch.randn((B, Hq, N, d), generator=g).to(dtype)
    n_of = [N] * B if new is None else list(new)
    for b, n in enumerate(n_of):
        q[b, :, n:] = float("nan")          # padding rows are not looked at
    scale = pr.default_scale(d)
    nl = None if new is None else torch.tensor(new, dtype=torch.int32, device=DEV)
    o = torch.full((B, Hq, N, d), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((B, Hq, N), 7.0, device=DEV)
    ws = torch.full((max(16, binding.fa_fwd_paged_workspace_bytes(B, Hq, Hkv, N, d, P, table.shape[1])),), 255,
                    dtype=torch.uint8, device=DEV)
    binding.fa_fwd_paged(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), tl.to(DEV), nl, o, lse, scale, ws)
    ok()
    pr.check_attention(o, lse, pr.attention(q, kc, vc, table, lens, n_of, scale), dtype, n_of)
    for b, n in enumerate(n_of):
        assert bool((o[b, :, n:] == 7).all()) and bool((lse[b, :, n:] == 7).all())


def test_fwd_paged_is_fa_fwd_of_the_same_keys():
    """Without cached tokens the pass is the causal forward pass."""
    Hq, Hkv, N, d, P, dtype = 8, 2, 513, 128, 64, BF
    kc, vc, table, tl = pr.make_cache(1, Hkv, d, P, (N, N), dtype)
    q = torch.randn((2, Hq, N, d), generator=torch.Generator().manual_seed(2)).to(dtype)
    dense = lambda c: torch.stack([c[table[b, :-(-N // P)].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, :N]
                                   for b in range(2)]).contiguous().to(DEV)
    o, lse = binding.attention_fwd_paged(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), tl.to(DEV))
    o2, lse2 = binding.attention_fwd(q.to(DEV), dense(kc), dense(vc), causal=True)
    ok()
    assert float((lse - lse2).abs().max()) <= pr.TOL_LSE
    # two roundings of O to 8 bits of values up to 4 and P rounded in both
    assert float((o.float() - o2.float()).abs().max()) <= 4 * 2.0 ** -7 + 2 * 2.0 ** -8


@pytest.mark.parametrize("d,P", [(128, 32), (64, 16)])
def test_fwd_paged_peaked_scores(d, P):
    """Scale 0.5: the running reference of a row moves again and again."""
    lens, N, Hq, Hkv = (900, 300), 200, 4, 2
    kc, vc, table, tl = pr.make_cache(5, Hkv, d, P, lens, BF)
    q = torch.randn((2, Hq, N, d), generator=torch.Generator().manual_seed(6)).to(BF)
    o, lse = binding.attention_fwd_paged(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), tl.to(DEV), scale=0.5)
    ok()
    pr.check_attention(o, lse, pr.attention(q, kc, vc, table, lens, [N, N], 0.5), BF, [N, N])


# --------------------------------------------------------------- shared prefix

PREFIX = [
    # Hq, Hkv, Nq, d, P, prefix, lens, dtype
    (2, 2, 1, 64, 16, 0, (1, 5), BF),
    (8, 2, 1, 128, 16, 16, (17, 18, 40), BF),
    (8, 2, 1, 128, 16, 1024, (1025, 1100, 1030, 1111), BF),
    (32, 8, 1, 128, 64, 512, tuple(513 + 37 * i for i in range(9)), FP),
    (4, 4, 3, 64, 32, 320, tuple(323 + i for i in range(50)), FP),
    (8, 1, 4, 128, 128, 2048, (2052, 2100, 2052, 3000, 2200), BF),
    (16, 16, 2, 64, 16, 144, tuple(146 + 5 * i for i in range(70)), BF),
    (28, 4, 1, 64, 64, 4096, (4097,) * 40, FP),
    (12, 12, 1, 64, 128, 256, (300,) * 129, BF),
    (8, 2, 1, 128, 32, 640, (641, 0, 700, 0), BF),          # idle sequences
    (8, 2, 2, 128, 32, 640, (700, 100, 3, 640, 641, 642), FP),  # shorter than the prefix
    (32, 4, 4, 128, 64, 1280, tuple(1300 + i for i in range(33)), BF),
]


@pytest.mark.parametrize("case", PREFIX, ids=lambda c: f"B{len(c[6])}-H{c[0]}/{c[1]}-Nq{c[2]}-d{c[3]}-P{c[4]}-pre{c[5]}")
def test_decode_prefix(case):
    Hq, Hkv, Nq, d, P, prefix, lens, dtype = case
    B = len(lens)
    kc, vc, table, tl = pr.make_cache(Nq + d + P, Hkv, d, P, lens, dtype, prefix=prefix)
    q = torch.randn((B, Hq, Nq, d), generator=torch.Generator().manual_seed(B)).to(dtype)
    scale = pr.default_scale(d)
    ref = pr.attention(q, kc, vc, table, lens, [Nq] * B, scale)
    seen = table.clone()
    seen[1:, :prefix // P] = -1               # only sequence 0's entries are read
    o = torch.full((B, Hq, Nq, d), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((B, Hq, Nq), 7.0, device=DEV)
    ws = torch.full((max(16, binding.fa_decode_prefix_workspace_bytes(B, Hq, Hkv, Nq, d, P, table.shape[1], prefix)),), 255,
                    dtype=torch.uint8, device=DEV)
    binding.fa_decode_prefix(q.to(DEV), kc.to(DEV), vc.to(DEV), seen.to(DEV), tl.to(DEV), o, lse, scale, prefix, ws)
    ok()
    pr.check_attention(o, lse, ref, dtype, [Nq] * B)


def test_decode_prefix_agrees_with_decode_paged():
    Hq, Hkv, Nq, d, P, prefix, lens, dtype = 16, 4, 2, 128, 64, 1024, (1100, 1026, 2000), BF
    kc, vc, table, tl = pr.make_cache(8, Hkv, d, P, lens, dtype, prefix=prefix, garbage=0.0)
    q = torch.randn((3, Hq, Nq, d), generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    args = [t.to(DEV) for t in (kc, vc, table, tl)]
    o, lse = binding.attention_decode_prefix(q, *args, prefix)
    o2, lse2 = binding.attention_decode_paged(q, *args)
    ok()
    assert float((lse - lse2).abs().max()) <= pr.TOL_LSE
    assert float((o.float() - o2.float()).abs().max()) <= 2.0 ** -7 + 2 * 2.0 ** -8


@pytest.mark.parametrize("d,P", [(128, 32), (64, 16)])
def test_decode_prefix_peaked_scores(d, P):
    lens, Hq, Hkv, Nq = tuple(1000 + 13 * i for i in range(20)), 16, 2, 2
    kc, vc, table, tl = pr.make_cache(5, Hkv, d, P, lens, BF, prefix=960)
    q = torch.randn((20, Hq, Nq, d), generator=torch.Generator().manual_seed(6)).to(BF)
    o, lse = binding.attention_decode_prefix(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), tl.to(DEV), 960, 0.5)
    ok()
    pr.check_attention(o, lse, pr.attention(q, kc, vc, table, lens, [Nq] * 20, 0.5), BF, [Nq] * 20)


SPLIT = [
    # Hq, Hkv, Nq, d, P, prefix, lens, table slack: few sequences with many own
    # keys (split over several blocks), tables far wider than the sequences
    (8, 2, 1, 128, 64, 128, (9000, 129, 4000), 1),
    (4, 1, 2, 64, 16, 0, (7000,), 1),
    (32, 4, 4, 128, 32, 64, (5000, 70), 3),
    (8, 2, 1, 128, 16, 16, (17, 20), 3000),
    (6, 2, 3, 64, 128, 1024, (1027, 1030), 500),
]


@pytest.mark.parametrize("case", SPLIT, ids=lambda c: f"B{len(c[6])}-H{c[0]}/{c[1]}-Nq{c[2]}-d{c[3]}-P{c[4]}-pre{c[5]}")
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_own_keys_split_over_blocks(case, dtype):
    Hq, Hkv, Nq, d, P, prefix, lens, slack = case
    B = len(lens)
    kc, vc, table, tl = pr.make_cache(d + P, Hkv, d, P, lens, dtype, prefix=prefix, table_slack=slack)
    q = torch.randn((B, Hq, Nq, d), generator=torch.Generator().manual_seed(B)).to(dtype)
    dev = [t.to(DEV) for t in (q, kc, vc, table, tl)]
    ref = pr.attention(q, kc, vc, table, lens, [Nq] * B, pr.default_scale(d))
    pr.check_attention(*binding.attention_decode_prefix(*dev, prefix), ref, dtype, [Nq] * B)
    pr.check_attention(*binding.attention_fwd_paged(*dev), ref, dtype, [Nq] * B)
    ok()


def test_many_heads_to_a_kv_head():
    """128 query heads share one kv head: a token fills a row tile."""
    Hq, N, d, P, lens = 128, 3, 64, 16, (200, 3)
    kc, vc, table, tl = pr.make_cache(2, 1, d, P, lens, BF)
    q = torch.randn((2, Hq, N, d), generator=torch.Generator().manual_seed(1)).to(BF)
    o, lse = binding.attention_fwd_paged(*[t.to(DEV) for t in (q, kc, vc, table, tl)])
    ok()
    pr.check_attention(o, lse, pr.attention(q, kc, vc, table, lens, [N, N], pr.default_scale(d)), BF, [N, N])


def test_no_new_tokens_write_nothing():
    kc, vc, table, tl = pr.make_cache(2, 2, 64, 16, (40, 20), BF)
    dev = [t.to(DEV) for t in (kc, vc, table, tl)]
    x = torch.randn((2, 2, 5, 64)).to(BF).to(DEV)
    none = torch.zeros(2, dtype=torch.int32, device=DEV)
    o, lse = torch.full_like(x, 7.0), torch.full((2, 2, 5), 7.0, device=DEV)
    ws = torch.empty(max(16, binding.fa_fwd_paged_workspace_bytes(2, 2, 2, 5, 64, 16, table.shape[1])), dtype=torch.uint8,
                     device=DEV)
    binding.fa_fwd_paged(x, *dev, none, o, lse, 0.125, ws)
    kd, vd = dev[0].clone(), dev[1].clone()
    binding.fa_append_paged(x, x, x, o, None, kd, vd, dev[2], dev[3], none, None)
    ok()
    assert bool((o == 7).all()) and bool((lse == 7).all())
    assert torch.equal(kd.view(torch.int16), dev[0].view(torch.int16))
    assert torch.equal(vd.view(torch.int16), dev[1].view(torch.int16))


def test_a_pool_of_more_than_2_32_values():
    """Pages whose element offset passes 32 bits, written and read back."""
    Hkv, d, P, dtype, N = 8, 128, 128, BF, 40
    pages = (1 << 32) // (Hkv * d * P) + 40
    kc = torch.empty((pages, Hkv, P, d), dtype=dtype, device=DEV)
    vc = torch.empty_like(kc)
    lens, prefix = (170, 300), 128
    table = torch.tensor([[pages - 1, pages - 3, -1], [pages - 1, pages - 2, pages - 5]], dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    small_k, small_v = (torch.randn((6, Hkv, P, d), generator=g).to(dtype) for _ in range(2))
    local = torch.where(table < 0, table, pages - table)     # the same pages in a small pool
    for i in (1, 2, 3, 5):
        kc[pages - i], vc[pages - i] = small_k[i].to(DEV), small_v[i].to(DEV)
    q, k, v = (torch.randn((2, h, N, d), generator=g).to(dtype) for h in (16, Hkv, Hkv))
    tl = torch.tensor(lens, dtype=torch.int32)
    freq = pr.inv_freq(d)
    args = [t.to(DEV) for t in (table, tl)]
    q_rot = binding.cache_append(q.to(DEV), k.to(DEV), v.to(DEV), kc, vc, *args, freq.to(DEV))
    o, lse = binding.attention_fwd_paged(q_rot, kc, vc, *args)
    one = q_rot[:, :, -1:].contiguous()
    o1, lse1 = binding.attention_decode_prefix(one, kc, vc, *args, prefix)
    ok()
    for i in (1, 2, 3, 5):
        small_k[i], small_v[i] = kc[pages - i].cpu(), vc[pages - i].cpu()
    for b, L in enumerate(lens):
        pos = torch.arange(L - N, L)
        want, mag = pr.rotated(k[b], pos, freq, False)
        pr.check_rotated(small_k[local[b].long()[pos // P], :, pos % P].transpose(0, 1).contiguous(), want, mag, "k")
        assert torch.equal(small_v[local[b].long()[pos // P], :, pos % P].transpose(0, 1), v[b])
    qc = q_rot.cpu()
    pr.check_attention(o, lse, pr.attention(qc, small_k, small_v, local, lens, [N, N], pr.default_scale(d)), dtype, [N, N])
    ref = pr.attention(qc[:, :, -1:].contiguous(), small_k, small_v, local, lens, [1, 1], pr.default_scale(d))
    pr.check_attention(o1, lse1, ref, dtype, [1, 1])


# ------------------------------------------------------------------ bad inputs

@pytest.mark.parametrize("bad", ["page", "page_negative", "too_long", "new_too_many", "new_negative", "short"])
def test_bad_lengths_and_pages_are_reported(bad):
    Hq, Hkv, N, d, P, lens, dtype = 4, 2, 20, 64, 16, [40, 30], BF
    kc, vc, table, tl = pr.make_cache(3, Hkv, d, P, lens, dtype)
    new = torch.tensor([20, 20], dtype=torch.int32)
    if bad == "page":
        table[1, 1] = kc.shape[0]
    elif bad == "page_negative":
        table[1, 1] = -7
    elif bad == "too_long":
        tl[1] = table.shape[1] * P + 1
    elif bad == "new_too_many":
        new[1] = N + 1
    elif bad == "new_negative":
        new[1] = -1
    else:
        tl[1] = 19
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn((2, h, N, d), generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
    dev = [t.to(DEV) for t in (kc, vc, table, tl)]
    nd = new.to(DEV)
    # the forward pass: the good sequence is right, the bad one is reported
    o, lse = binding.attention_fwd_paged(q.to(DEV), *dev, nd)
    assert binding.fa_get_device_status() == binding.FA_ERR_INVALID_ARG
    ref = pr.attention(q, kc, vc, table, [40, 0], [20, 0], pr.default_scale(d))
    pr.check_attention(o[:1], lse[:1], [x[:1] for x in ref], dtype, [20])
    if not bad.startswith("page"):
        assert bool((o[1] == 0).all()) and bool((lse[1] == float("-inf")).all())
    # append: the good sequence's slots, and nothing outside the cache
    kd, vd = dev[0].clone(), dev[1].clone()
    binding.cache_append(q.to(DEV), k.to(DEV), v.to(DEV), kd, vd, dev[2], dev[3], new_lens=nd)
    assert binding.fa_get_device_status() == binding.FA_ERR_INVALID_ARG
    pos = torch.arange(20, 40)
    page = table[0].long()[pos // P]
    assert torch.equal(vd.cpu()[page, :, pos % P].transpose(0, 1), v[0])
    if bad in ("page", "page_negative", "too_long", "short"):
        qd = q[:, :, -3:].contiguous().to(DEV)
        if bad == "short":
            dev[3][1] = 2
        o, lse = binding.attention_decode_prefix(qd, *dev, 0)
        assert binding.fa_get_device_status() == binding.FA_ERR_INVALID_ARG
        ref = pr.attention(q[:1, :, -3:].contiguous(), kc, vc, table, [40], [3], pr.default_scale(d))
        pr.check_attention(o[:1], lse[:1], ref, dtype, [3])
    ok()


def test_bad_prefix_page_is_reported():
    Hq, Hkv, d, P, prefix, lens = 8, 2, 128, 16, 256, (300, 280)
    kc, vc, table, tl = pr.make_cache(3, Hkv, d, P, lens, BF, prefix=prefix)
    table[0, 3] = kc.shape[0] + 100
    q = torch.randn((2, Hq, 1, d)).to(BF).to(DEV)
    binding.attention_decode_prefix(q, kc.to(DEV), vc.to(DEV), table.to(DEV), tl.to(DEV), prefix)
    assert binding.fa_get_device_status() == binding.FA_ERR_INVALID_ARG
    ok()


def test_bad_page_of_a_long_prefix_is_reported():
    Hq, Hkv, d, P, prefix, lens = 8, 2, 128, 16, 2048, (2100, 2060)
    kc, vc, table, tl = pr.make_cache(3, Hkv, d, P, lens, BF, prefix=prefix)
    table[0, 77] = -4
    q = torch.randn((2, Hq, 1, d)).to(BF).to(DEV)
    binding.attention_decode_prefix(q, kc.to(DEV), vc.to(DEV), table.to(DEV), tl.to(DEV), prefix)
    assert binding.fa_get_device_status() == binding.FA_ERR_INVALID_ARG
    ok()


@pytest.mark.parametrize("prefix", [64, 512, 528])
@pytest.mark.parametrize("B", [2, 17, 70])
def test_prefix_lengths_around_the_pass_of_their_own(prefix, B):
    """Short prefixes are taken with the own keys, longer ones and those of
    many sequences in a pass of their own; sequence 0 idle or not."""
    Hq, Hkv, Nq, d, P = 8, 4, 2, 128, 16
    for first in (prefix + 5, 0):
        lens = (first,) + tuple(prefix + 2 + 7 * i for i in range(B - 1))
        kc, vc, table, tl = pr.make_cache(B, Hkv, d, P, lens, BF, prefix=prefix)
        if first == 0:   # the prefix is still found through sequence 0's table
            table[0, :prefix // P] = table[1, :prefix // P]
        q = torch.randn((B, Hq, Nq, d), generator=torch.Generator().manual_seed(B)).to(BF)
        ref = pr.attention(q, kc, vc, table, lens, [Nq] * B, pr.default_scale(d))
        seen = table.clone()
        seen[1:, :prefix // P] = -1
        o, lse = binding.attention_decode_prefix(q.to(DEV), kc.to(DEV), vc.to(DEV), seen.to(DEV), tl.to(DEV), prefix)
        ok()
        pr.check_attention(o, lse, ref, BF, [Nq] * B)


# ---------------------------------------------------------------- as one server

class Server:
    """A batch behind one prefix: the prefix and each sequence's own prompt
    appended and run over the cache, then decode steps; the same tokens kept
    on the host for the 64-bit reference."""

    def __init__(self, dtype, Hq=8, Hkv=2, d=128, P=32, prefix=96, prompts=(5, 33, 1, 20), steps=3, seed=11):
        self.dtype, self.Hq, self.Hkv, self.d, self.P, self.prefix = dtype, Hq, Hkv, d, P, prefix
        self.prompts, self.steps = prompts, steps
        self.g = torch.Generator("cpu").manual_seed(seed)
        self.freq = pr.inv_freq(d)
        B, own = len(prompts), -(-(max(prompts) + steps) // P)
        pages = prefix // P + B * own + 2
        perm = torch.randperm(pages, generator=self.g).to(torch.int32)
        shared = perm[:prefix // P]
        self.table = torch.stack([torch.cat([shared, perm[prefix // P + b * own:prefix // P + (b + 1) * own]])
                                  for b in range(B)])
        self.kc = torch.full((pages, Hkv, P, d), float("nan"), dtype=dtype, device=DEV)
        self.vc = torch.full_like(self.kc, float("nan"))
        self.k_ref, self.v_ref = [None] * B, [None] * B      # rotated keys and values of every sequence, 64-bit

    def tokens(self, B, N):
        return [torch.randn((B, h, N, self.d), generator=self.g).to(self.dtype) for h in (self.Hq, self.Hkv, self.Hkv)]

    def keep(self, b, k, v, start):
        n = k.shape[1]
        kr = pr.rotated(k, torch.arange(start, start + n), self.freq, False)[0].to(self.dtype).double()
        cat = lambda a, x: x if a is None else torch.cat([a, x], 1)
        self.k_ref[b], self.v_ref[b] = cat(self.k_ref[b], kr), cat(self.v_ref[b], v.double())

    def check(self, o, lse, q, new):
        """The reference reads the keys rounded to the I/O type.  Keys and
        queries turned in 32 bits may land on the neighbouring value where the
        exact one is a tie within 2^-19: a step of 2^-8 (bf16) of the feature
        moves a score by at most 2^-8 |q_c k_c| scale, 1e-2 for normal inputs
        at one feature; O and lse are held to 4e-2."""
        for b, n in enumerate(new):
            L = self.k_ref[b].shape[1]
            qr = pr.rotated(q[b, :, :n], torch.arange(L - n, L), self.freq, False)[0].to(self.dtype).double()
            G = self.Hq // self.Hkv
            s = torch.einsum("hnd,hld->hnl", qr, self.k_ref[b].repeat_interleave(G, 0)) * pr.default_scale(self.d)
            s.masked_fill_(torch.arange(L)[None] > torch.arange(L - n, L)[:, None], float("-inf"))
            want = s.softmax(-1) @ self.v_ref[b].repeat_interleave(G, 0)
            assert float((o[b, :, :n].cpu().double() - want).abs().max()) <= 4e-2
            assert float((lse[b, :, :n].cpu().double() - s.logsumexp(-1)).abs().max()) <= 4e-2

    def run(self, decode_step=None):
        B, freq = len(self.prompts), self.freq.to(DEV)
        table = self.table.to(DEV)
        dev = lambda *ts: [t.to(DEV) for t in ts]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        # the prefix: once, through sequence 0's table, its attention by fa_fwd on the rotated keys
        q, k, v = self.tokens(1, self.prefix)
        qd, kd, vd = dev(q, k, v)
        q_rot, k_rot = torch.empty_like(qd), torch.empty_like(kd)
        binding.fa_append_paged(qd, kd, vd, q_rot, k_rot, self.kc, self.vc, table[:1], i32([self.prefix]), None, freq)
        for b in range(B):
            self.keep(b, k[0], v[0], 0)
        self.check(*binding.attention_fwd(q_rot, k_rot, vd, causal=True), q, [self.prefix])
        # each sequence's own prompt, padded to the longest
        N, lens = max(self.prompts), [self.prefix + n for n in self.prompts]
        q, k, v = self.tokens(B, N)
        new = i32(self.prompts)
        q_rot = binding.cache_append(*dev(q, k, v), self.kc, self.vc, table, i32(lens), freq, new)
        o, lse = binding.attention_fwd_paged(q_rot, self.kc, self.vc, table, i32(lens), new)
        for b, n in enumerate(self.prompts):
            self.keep(b, k[b, :, :n], v[b, :, :n], self.prefix)
        self.check(o, lse, q, self.prompts)
        # decode
        for step in range(self.steps):
            lens = [L + 1 for L in lens]
            q, k, v = self.tokens(B, 1)
            if decode_step is None:
                q_rot = binding.cache_append(*dev(q, k, v), self.kc, self.vc, table, i32(lens), freq)
                o, lse = binding.attention_decode_prefix(q_rot, self.kc, self.vc, table, i32(lens), self.prefix)
            else:
                o, lse = decode_step(self, table, freq, *dev(q, k, v), i32(lens))
            for b in range(B):
                self.keep(b, k[b], v[b], lens[b] - 1)
            self.check(o, lse, q, [1] * B)
        ok()


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_prefix_prompts_and_decode_together(dtype):
    Server(dtype).run()


def test_decode_step_captured_once_and_replayed():
    """Append and decode captured as one graph over fixed buffers; every step
    copies its inputs in and replays it."""
    state = {}

    def step(server, table, freq, q, k, v, lens):
        if not state:
            for n, t in dict(q=q, k=k, v=v, lens=lens).items():
                state[n] = t.clone()
            B, Hq, _, d = q.shape
            state["o"], state["lse"] = torch.empty_like(q), torch.empty((B, Hq, 1), device=DEV)
            state["q_rot"] = torch.empty_like(q)
            state["ws"] = torch.empty(max(16, binding.fa_decode_prefix_workspace_bytes(
                B, Hq, server.Hkv, 1, d, server.P, table.shape[1], server.prefix)), dtype=torch.uint8, device=DEV)

            def work():
                binding.fa_append_paged(state["q"], state["k"], state["v"], state["q_rot"], None, server.kc, server.vc,
                                        table, state["lens"], None, freq)
                binding.fa_decode_prefix(state["q_rot"], server.kc, server.vc, table, state["lens"], state["o"],
                                         state["lse"], pr.default_scale(d), server.prefix, state["ws"])

            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                work()  # first call outside the capture: loads the kernels
            torch.cuda.current_stream().wait_stream(side)
            state["graph"] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(state["graph"]):
                work()
        for n, t in dict(q=q, k=k, v=v, lens=lens).items():
            state[n].copy_(t)
        state["graph"].replay()
        return state["o"], state["lse"]

    Server(BF, steps=4).run(step)


def test_two_graphs_share_a_workspace():
    """Two captured passes of different sizes over one workspace, replayed in
    turn: neither leaves anything the other depends on."""
    Hq, Hkv, d, P = 8, 2, 128, 16
    calls = []
    nbytes = 16
    for prefix, lens, N in ((512, (600, 520, 530), 1), (64, (70, 80), 4)):
        kc, vc, table, tl = pr.make_cache(prefix, Hkv, d, P, lens, BF, prefix=prefix)
        q = torch.randn((len(lens), Hq, N, d), generator=torch.Generator().manual_seed(N)).to(BF)
        ref = pr.attention(q, kc, vc, table, lens, [N] * len(lens), pr.default_scale(d))
        calls.append((q, kc, vc, table, tl, prefix, ref, N))
        nbytes = max(nbytes, binding.fa_decode_prefix_workspace_bytes(len(lens), Hq, Hkv, N, d, P, table.shape[1], prefix),
                     binding.fa_fwd_paged_workspace_bytes(len(lens), Hq, Hkv, N, d, P, table.shape[1]))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    graphs = []
    for q, kc, vc, table, tl, prefix, ref, N in calls:
        dev = [t.to(DEV) for t in (q, kc, vc, table, tl)]
        for which in ("prefix", "paged"):
            o, lse = torch.zeros_like(dev[0]), torch.zeros(q.shape[:3], device=DEV)

            def work():
                if which == "prefix":
                    binding.fa_decode_prefix(*dev, o, lse, pr.default_scale(d), prefix, ws)
                else:
                    binding.fa_fwd_paged(*dev, None, o, lse, pr.default_scale(d), ws)

            work()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                work()
            graphs.append((graph, o, lse, ref, N, q.shape[0], dev))
    for order in ((0, 1, 2, 3), (3, 1, 0, 2), (2, 2, 0, 0)):
        for i in order:
            graphs[i][1].zero_(), graphs[i][2].zero_()
            graphs[i][0].replay()
        for i in order:
            _, o, lse, ref, N, B, _ = graphs[i]
            pr.check_attention(o, lse, ref, BF, [N] * B)
    ok()


def test_calls_on_two_streams_do_not_meet():
    """Two streams, each with its own buffers, a row of calls in flight on both."""
    Hq, Hkv, d, P, prefix, N = 8, 2, 128, 16, 256, 2
    runs = []
    for seed, lens in ((1, (300, 258, 400)), (2, (270, 900))):
        kc, vc, table, tl = pr.make_cache(seed, Hkv, d, P, lens, FP, prefix=prefix)
        q = torch.randn((len(lens), Hq, N, d), generator=torch.Generator().manual_seed(seed)).to(FP)
        ref = pr.attention(q, kc, vc, table, lens, [N] * len(lens), pr.default_scale(d))
        runs.append((torch.cuda.Stream(), [t.to(DEV) for t in (q, kc, vc, table, tl)], ref, len(lens), []))
    torch.cuda.synchronize()
    for _ in range(5):
        for stream, dev, _, _, outs in runs:
            outs.append(binding.attention_decode_prefix(*dev, prefix, stream=stream))
            outs.append(binding.attention_fwd_paged(*dev, stream=stream.cuda_stream))
    torch.cuda.synchronize()
    for _, _, ref, B, outs in runs:
        for o, lse in outs:
            pr.check_attention(o, lse, ref, FP, [N] * B)
    ok()


def test_the_default_stream_by_its_number():
    kc, vc, table, tl = pr.make_cache(2, 2, 64, 16, (40, 20), BF)
    q = torch.randn((2, 2, 5, 64), generator=torch.Generator().manual_seed(1)).to(BF)
    dev = [t.to(DEV) for t in (q, kc, vc, table, tl)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o, lse = binding.attention_fwd_paged(*dev, stream=0)
    torch.cuda.synchronize()
    ok()
    pr.check_attention(o, lse, pr.attention(q, kc, vc, table, (40, 20), (5, 5), pr.default_scale(64)), BF, (5, 5))


def test_results_repeat_bit_for_bit():
    Hq, Hkv, d, P, prefix, lens = 32, 8, 128, 64, 4096, tuple(4100 + 31 * i for i in range(12))
    kc, vc, table, tl = pr.make_cache(9, Hkv, d, P, lens, BF, prefix=prefix)
    q = torch.randn((12, Hq, 1, d), generator=torch.Generator().manual_seed(1)).to(BF)
    dev = [t.to(DEV) for t in (q, kc, vc, table, tl)]
    first = binding.attention_decode_prefix(*dev, prefix), binding.attention_fwd_paged(*dev)
    for _ in range(3):
        again = binding.attention_decode_prefix(*dev, prefix), binding.attention_fwd_paged(*dev)
        for a, b in zip(first, again):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ok()


def test_empty_batches_are_no_ops():
    kc = torch.zeros((2, 2, 16, 64), dtype=BF, device=DEV)
    table = torch.zeros((0, 2), dtype=torch.int32, device=DEV)
    lens = torch.zeros((0,), dtype=torch.int32, device=DEV)
    q = torch.zeros((0, 4, 1, 64), dtype=BF, device=DEV)
    assert binding.attention_decode_prefix(q, kc, kc.clone(), table, lens, 0)[0].shape == q.shape
    assert binding.attention_fwd_paged(q, kc, kc.clone(), table, lens)[0].shape == q.shape
    k = torch.zeros((0, 2, 1, 64), dtype=BF, device=DEV)
    assert binding.cache_append(q, k, k, kc, kc.clone(), table, lens).shape == q.shape
    q = torch.zeros((2, 4, 0, 64), dtype=BF, device=DEV)
    table, lens = torch.zeros((2, 2), dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    assert binding.attention_fwd_paged(q, kc, kc.clone(), table, lens)[0].shape == q.shape
    ok()


def _sweep(n, seed):
    g = np.random.default_rng(seed)
    cases = []
    for _ in range(n):
        Hkv, G = int(g.choice([1, 2, 4])), int(g.choice([1, 2, 3, 7, 8]))
        Nq = int(g.choice([x for x in (1, 2, 3, 4) if x * G <= 32]))
        P, d = int(g.choice([16, 32, 64, 128])), int(g.choice([64, 128]))
        B = int(g.integers(1, 40))
        prefix = P * int(g.integers(0, 1500 // P + 1))
        lens = tuple(int(prefix + Nq + g.integers(0, 200)) for _ in range(B))
        N = int(g.integers(1, 400))
        new = tuple(int(g.integers(0, min(N, L) + 1)) for L in lens[:3])
        cases.append((Hkv * G, Hkv, Nq, d, P, prefix, lens, N, new, BF if g.random() < 0.5 else FP))
    return cases


@pytest.mark.parametrize("case", _sweep(24, 515), ids=lambda c: f"B{len(c[6])}-H{c[0]}/{c[1]}-Nq{c[2]}-d{c[3]}-P{c[4]}"
                         f"-pre{c[5]}-N{c[7]}")
def test_random_shapes(case):
    Hq, Hkv, Nq, d, P, prefix, lens, N, new, dtype = case
    test_decode_prefix((Hq, Hkv, Nq, d, P, prefix, lens, dtype))
    test_fwd_paged((Hq, Hkv, N, d, P, lens[:3], new, dtype))
