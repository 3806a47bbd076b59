"""What the paged-cache operators are measured on.

Three operators of one serving path over a paged key/value cache
([pages][Hkv][page][d], found through a block table):

  append  new keys and values into the cache, keys (and queries) rotated by
          their position on the way
  prefix  decode of a batch whose sequences share a long prefix
  paged   forward pass of many new tokens against the cache that holds them

``run`` computes a pass in elementary torch operations (``own`` false) or
through the library's calls (``own`` true); ``exact`` is the definition in
64 bits.  Positions, page orders and lengths are drawn from the case alone,
values from the seed.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda"
_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one sequence: latency only
        dict(name="append_token", op="append", B=1, Hq=32, Hkv=8, N=1, d=128, P=16, dtype="bf16", rot=128,
             interleaved=False, base=10000.0, past=900, ragged=False, layout="dense", keep_k=False, lens_seed=1),
        # a decode step of a large batch, far into long contexts, pairs interleaved
        dict(name="append_batch", op="append", B=256, Hq=16, Hkv=16, N=1, d=128, P=64, dtype="fp16", rot=128,
             interleaved=True, base=500000.0, past=6000, ragged=False, layout="token", keep_k=False, lens_seed=2),
        # a padded batch of short prompts, half of each head rotated, read out
        # of the packed projection (one row holds q, k and v of a token)
        dict(name="append_ragged", op="append", B=13, Hq=12, Hkv=12, N=777, d=64, P=32, dtype="fp16", rot=32,
             interleaved=False, base=10000.0, past=0, ragged=True, layout="token", keep_k=True, lens_seed=3),
        # the prompt of a 16K-token grouped-query workload
        dict(name="append_prompt", op="append", B=1, Hq=32, Hkv=8, N=16384, d=128, P=64, dtype="bf16", rot=128,
             interleaved=False, base=500000.0, past=0, ragged=False, layout="dense", keep_k=True, lens_seed=4),

        # four requests behind a short system prompt: latency
        dict(name="prefix_few", op="prefix", B=4, Hq=32, Hkv=8, Nq=1, d=128, P=16, dtype="bf16", prefix=1024,
             own_max=100, lens_seed=5),
        # an ordinary batch behind a long document
        dict(name="prefix_document", op="prefix", B=32, Hq=32, Hkv=8, Nq=1, d=128, P=64, dtype="bf16", prefix=16384,
             own_max=512, lens_seed=6),
        # three tokens a step (drafted tokens to verify), multi-head, odd batch
        dict(name="prefix_drafts", op="prefix", B=50, Hq=12, Hkv=12, Nq=3, d=64, P=16, dtype="fp16", prefix=5008,
             own_max=300, lens_seed=7),
        # many samples of one 64K-token prompt: more query rows than one tile
        dict(name="prefix_samples", op="prefix", B=96, Hq=32, Hkv=8, Nq=1, d=128, P=128, dtype="bf16", prefix=65536,
             own_max=1000, lens_seed=8),

        # a short chunk of one sequence: latency
        dict(name="paged_short", op="paged", B=1, Hq=8, Hkv=2, N=40, d=128, P=16, dtype="bf16", past=300,
             ragged=False, lens_seed=9),
        # chunks of a few long sequences: few rows, many cached tokens
        dict(name="paged_chunk", op="paged", B=4, Hq=32, Hkv=8, N=64, d=128, P=64, dtype="bf16", past=16000,
             ragged=False, lens_seed=10),
        # a padded batch of prompts with nothing or little cached before them
        dict(name="paged_ragged", op="paged", B=8, Hq=12, Hkv=12, N=777, d=64, P=32, dtype="fp16", past=500,
             ragged=True, lens_seed=11),
        # long prompts behind a long cached context
        dict(name="paged_prompt", op="paged", B=2, Hq=32, Hkv=8, N=4096, d=128, P=64, dtype="bf16", past=8192,
             ragged=False, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "prefix", "paged"])
    Hq, Hkv = rng.choice([(32, 8), (16, 16), (12, 12), (8, 2), (8, 1), (6, 2), (5, 5), (28, 4)])
    c = dict(op=op, Hq=Hq, Hkv=Hkv, d=rng.choice([64, 128]), P=rng.choice([16, 32, 64, 128]),
             dtype=rng.choice(["bf16", "fp16"]), lens_seed=rng.randrange(1 << 20))
    if op == "append":
        tokens = _log_int(rng, 1, 200000)
        B = _log_int(rng, 1, min(256, tokens))
        c.update(B=B, N=max(1, tokens // B), rot=rng.choice([16, 32, c["d"] // 2, c["d"], c["d"]]),
                 interleaved=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0, 1000000.0]),
                 past=rng.choice([0, _log_int(rng, 1, 20000)]), ragged=rng.random() < 0.5,
                 layout=rng.choice(["dense", "token"]), keep_k=rng.random() < 0.5)
        # no more values moved than by the largest listed case, caches that fit
        cost = lambda: c["B"] * c["N"] * (Hq + 2 * Hkv) * c["d"]
        while cost() > 16384 * 48 * 128:
            c["N"] = c["N"] // 2
        while c["B"] * (c["past"] + c["N"]) * Hkv * c["d"] > (1 << 28):
            c["past"] //= 2
    elif op == "prefix":
        G = Hq // Hkv
        c.update(B=_log_int(rng, 1, 200), Nq=rng.choice([1, 1, 1, 2, 3, 4]),
                 prefix=c["P"] * max(1, _log_int(rng, 64, 65536) // c["P"]), own_max=_log_int(rng, 4, 1500))
        while c["B"] * G * c["Nq"] * Hkv * c["prefix"] * c["d"] > 96 * 32 * 65536 * 128:
            c["B"] = max(1, c["B"] // 2)
        while c["B"] * Hkv * c["own_max"] * c["d"] > 96 * 8 * 1000 * 128:
            c["own_max"] //= 2
    else:
        c.update(B=_log_int(rng, 1, 16), N=_log_int(rng, 1, 6000), past=rng.choice([0, _log_int(rng, 1, 30000)]),
                 ragged=rng.random() < 0.5)
        pairs = lambda: c["B"] * Hq * c["N"] * (c["past"] + c["N"]) * c["d"]
        while pairs() > 2 * 32 * 4096 * (8192 + 2048) * 128:
            c["N"] = max(1, c["N"] // 2)
            c["past"] = c["past"] * 3 // 4
    return c


# ------------------------------------------------------------------- lengths

def _lengths(case):
    """(cached tokens with the new ones, new tokens) of every sequence."""
    rng = random.Random(case["lens_seed"])
    total, new = [], []
    for b in range(case["B"]):
        if case["op"] == "prefix":
            new.append(case["Nq"])
            total.append(case["prefix"] + case["Nq"] + rng.randrange(case["own_max"]))
        else:
            n = rng.randint(1, case["N"]) if case["ragged"] and b > 0 else case["N"]
            past = rng.randint(case["past"] // 2, case["past"])
            new.append(n)
            total.append(past + n)
    return total, new


def _pages(case, total):
    """Block table rows (lists of physical pages) and the number of pages: in
    a shuffled pool, the prefix's pages shared by every sequence."""
    P = case["P"]
    shared = case["prefix"] // P if case["op"] == "prefix" else 0
    need = [-(-L // P) - shared for L in total]
    count = shared + sum(need) + 3
    pool = list(range(count))
    random.Random(case["lens_seed"] + 1).shuffle(pool)
    rows, used = [], shared
    for n in need:
        rows.append(pool[:shared] + pool[used:used + n])
        used += n
    return rows, count


# -------------------------------------------------------------------- inputs

def _inputs(case, seed):
    g = torch.Generator(DEVICE).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    B, Hq, Hkv, d, P = case["B"], case["Hq"], case["Hkv"], case["d"], case["P"]
    N = case["Nq"] if case["op"] == "prefix" else case["N"]
    total, new = _lengths(case)
    rows, count = _pages(case, total)
    width = max(len(r) for r in rows)
    randn = lambda *shape: torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32).to(dt)
    s = dict(
        case=case, total=total, new=new, width=width,
        table=torch.tensor([r + [-1] * (width - len(r)) for r in rows], dtype=torch.int32, device=DEVICE),
        lens=torch.tensor(total, dtype=torch.int32, device=DEVICE),
        new_lens=torch.tensor(new, dtype=torch.int32, device=DEVICE),
        k_cache=randn(count, Hkv, P, d), v_cache=randn(count, Hkv, P, d))
    if case["op"] != "append":
        s["q"] = randn(B, Hq, N, d)
        s["scale"] = 1.0 / math.sqrt(d)
        return s
    if case["layout"] == "token":
        # rows of a packed projection, [B][N][q heads, k heads, v heads][d]
        x = randn(B, N, Hq + 2 * Hkv, d).transpose(1, 2)
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        s["q"], s["k"], s["v"] = randn(B, Hq, N, d), randn(B, Hkv, N, d), randn(B, Hkv, N, d)
    half = case["rot"] // 2
    s["inv_freq"] = (case["base"] ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(DEVICE)
    s["q_out"] = torch.zeros(B, Hq, N, d, dtype=dt, device=DEVICE)
    s["k_out"] = torch.zeros(B, Hkv, N, d, dtype=dt, device=DEVICE) if case["keep_k"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "append":
        # sequence, token and cache slot of every new token, for the plain form
        b = [i for i, n in enumerate(s["new"]) for _ in range(n)]
        t = [j for n in s["new"] for j in range(n)]
        s["tok_b"] = torch.tensor(b, device=DEVICE)
        s["tok_t"] = torch.tensor(t, device=DEVICE)
        return s
    s["o"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(s["q"].shape[:3], dtype=torch.float32, device=DEVICE)
    if own:
        from exact_io_aware_bwd_b200 import binding
        B, Hq, N, d = s["q"].shape
        if case["op"] == "prefix":
            n = binding.fa_decode_prefix_workspace_bytes(B, Hq, case["Hkv"], N, d, case["P"], s["width"], case["prefix"])
        else:
            n = binding.fa_fwd_paged_workspace_bytes(B, Hq, case["Hkv"], N, d, case["P"], s["width"])
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEVICE)
    return s


# ---------------------------------------------------------------------- runs

def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _append_own, "prefix": _prefix_own, "paged": _paged_own}[op](s)
    return {"append": _append_plain, "prefix": _prefix_plain, "paged": _paged_plain}[op](s)


def _append_outputs(s):
    out = dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    if s["k_out"] is not None:
        out["k"] = s["k_out"]
    return out


def _append_own(s):
    from exact_io_aware_bwd_b200 import binding
    binding.fa_append_paged(s["q"], s["k"], s["v"], s["q_out"], s["k_out"], s["k_cache"], s["v_cache"], s["table"],
                            s["lens"], s["new_lens"], s["inv_freq"], s["case"]["interleaved"])
    return _append_outputs(s)


def _prefix_own(s):
    from exact_io_aware_bwd_b200 import binding
    binding.fa_decode_prefix(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["o"], s["lse"], s["scale"],
                             s["case"]["prefix"], s["workspace"])
    return s["o"], s["lse"]


def _paged_own(s):
    from exact_io_aware_bwd_b200 import binding
    binding.fa_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["new_lens"], s["o"], s["lse"],
                         s["scale"], s["workspace"])
    return s["o"], s["lse"]


def _rotate_plain(x, cos, sin, rot, interleaved):
    """x [tokens, heads, d] in 32 bits, cos and sin [tokens, 1, rot / 2]."""
    r = x[..., :rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _append_plain(s):
    case = s["case"]
    b, t = s["tok_b"], s["tok_t"]
    pos = s["lens"].long()[b] - s["new_lens"].long()[b] + t
    # angles of far positions lose their fraction in 32 bits
    angle = pos.double()[:, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    page, slot = s["table"].long()[b, pos // case["P"]], pos % case["P"]
    dt = s["k"].dtype
    rotated = lambda x: _rotate_plain(x[b, :, t].float(), cos, sin, case["rot"], case["interleaved"]).to(dt)
    kr = rotated(s["k"])
    s["q_out"][b, :, t] = rotated(s["q"])
    s["k_cache"][page, :, slot] = kr
    s["v_cache"][page, :, slot] = s["v"][b, :, t]
    if s["k_out"] is not None:
        s["k_out"][b, :, t] = kr
    return _append_outputs(s)


def _gather(cache, pages):
    """Rows of the given pages in order: [..., Hkv, keys, d] in 32 bits."""
    x = cache[pages]                      # [..., n, Hkv, P, d]
    x = x.movedim(-3, -4)                 # [..., Hkv, n, P, d]
    return x.flatten(-3, -2).float()


def _prefix_plain(s):
    case = s["case"]
    B, Hq, N, d = s["q"].shape
    Hkv, P, scale = case["Hkv"], case["P"], s["scale"]
    G, shared = Hq // Hkv, case["prefix"] // case["P"]
    table = s["table"].long()
    q = s["q"].float().view(B, Hkv, G * N, d)
    # the prefix, once for the rows of every sequence
    kp, vp = _gather(s["k_cache"], table[0, :shared]), _gather(s["v_cache"], table[0, :shared])
    qp = q.transpose(0, 1).reshape(Hkv, B * G * N, d)
    sp = (qp @ kp.transpose(1, 2)) * scale
    mp = sp.amax(-1, keepdim=True)
    pp = (sp - mp).exp()
    back = lambda x: x.reshape(Hkv, B, G * N, -1).transpose(0, 1)
    op, lp, mp = back(pp @ vp), back(pp.sum(-1, keepdim=True)), back(mp)
    # each sequence's own tokens, padded to the longest
    pages = table[:, shared:].clamp(min=0)
    ko, vo = _gather(s["k_cache"], pages), _gather(s["v_cache"], pages)
    so = (q @ ko.transpose(2, 3)) * scale
    key = case["prefix"] + torch.arange(so.shape[-1], device=DEVICE)
    last = s["lens"].long()[:, None] - N + torch.arange(N, device=DEVICE)         # [B, N]
    hidden = key > last.repeat(1, G)[:, None, :, None]
    so = so.masked_fill(hidden, float("-inf"))
    m = torch.maximum(mp, so.amax(-1, keepdim=True))
    po = (so - m).exp()
    w = (mp - m).exp()
    l = lp * w + po.sum(-1, keepdim=True)
    o = (op * w + po @ vo) / l
    lse = m + l.log()
    return o.reshape(B, Hq, N, d).to(s["q"].dtype), lse.reshape(B, Hq, N)


def _paged_plain(s):
    case = s["case"]
    B, Hq, N, d = s["q"].shape
    Hkv, P, G = case["Hkv"], case["P"], Hq // case["Hkv"]
    table = s["table"].long()
    for b in range(B):
        L, n = s["total"][b], s["new"][b]
        pages = table[b, :-(-L // P)]
        k, v = _gather(s["k_cache"], pages)[:, :L], _gather(s["v_cache"], pages)[:, :L]
        q = s["q"][b, :, :n].float().view(Hkv, G * n, d)
        x = (q @ k.transpose(1, 2)).view(Hkv, G, n, L) * s["scale"]
        row, key = torch.arange(n, device=DEVICE), torch.arange(L, device=DEVICE)
        x.masked_fill_(key > (L - n + row)[:, None], float("-inf"))
        m = x.amax(-1, keepdim=True)
        x = (x - m).exp_()
        l = x.sum(-1, keepdim=True)
        o = (x.view(Hkv, G * n, L) @ v).view(Hkv, G, n, d) / l
        s["o"][b, :, :n] = o.view(Hq, n, d).to(s["o"].dtype)
        s["lse"][b, :, :n] = (m + l.log()).view(Hq, n)
    return s["o"], s["lse"]


# ---------------------------------------------------------------------- work

def work(case):
    total, new = _lengths(case)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    rows = sum(new)
    if case["op"] == "append":
        moved = rows * d * 2 * (2 * Hq + 4 * Hkv + (Hkv if case["keep_k"] else 0))
        return {"bytes": moved + 4 * (sum(-(-L // case["P"]) for L in total) + 2 * case["B"]),
                "flops": 3 * rows * (Hq + Hkv) * case["rot"]}
    pairs = sum(n * L - n * (n - 1) // 2 for L, n in zip(total, new))
    if case["op"] == "prefix":
        keys = case["prefix"] + sum(L - case["prefix"] for L in total)
    else:
        keys = sum(total)
    return {"bytes": 2 * 2 * keys * Hkv * d + rows * Hq * (2 * 2 * d + 4), "flops": 4 * pairs * Hq * d}


# --------------------------------------------------------------------- exact

def exact(case, seed):
    s = _inputs(case, seed)
    return _append_exact(s) if case["op"] == "append" else _attention_exact(s)


def _append_exact(s):
    """Token by token of a sequence: the rotation as a complex product."""
    case = s["case"]
    rot, P = case["rot"], case["P"]
    out = {n: s[n].double() for n in ("k_cache", "v_cache")}
    out["q"] = s["q_out"].double()
    if s["k_out"] is not None:
        out["k"] = s["k_out"].double()
    f = s["inv_freq"].double()
    for b in range(case["B"]):
        L, n = s["total"][b], s["new"][b]
        pos = torch.arange(L - n, L, device=DEVICE)
        turn = torch.polar(torch.ones((n, rot // 2), dtype=torch.float64, device=DEVICE), pos.double()[:, None] * f)

        def rotated(x):
            x = x[b, :, :n].double()
            y = x.clone()
            if case["interleaved"]:
                z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * turn
                y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
            else:
                h = rot // 2
                z = torch.complex(x[..., :h].contiguous(), x[..., h:rot].contiguous()) * turn
                y[..., :h], y[..., h:rot] = z.real, z.imag
            return y

        k = rotated(s["k"])
        out["q"][b, :, :n] = rotated(s["q"])
        if "k" in out:
            out["k"][b, :, :n] = k
        pages = s["table"][b].long()[pos // P]
        out["k_cache"][pages, :, pos % P] = k.transpose(0, 1)
        out["v_cache"][pages, :, pos % P] = s["v"][b, :, :n].double().transpose(0, 1)
    return {n: out[n] for n in ("q", "k_cache", "v_cache", "k") if n in out}


def _attention_exact(s):
    """Sequence by sequence and kv head by kv head, every key gathered."""
    case = s["case"]
    B, Hq, N, d = s["q"].shape
    Hkv, P = case["Hkv"], case["P"]
    G = Hq // Hkv
    o = torch.zeros((B, Hq, N, d), dtype=torch.float64, device=DEVICE)
    lse = torch.zeros((B, Hq, N), dtype=torch.float64, device=DEVICE)
    for b in range(B):
        L, n = s["total"][b], s["new"][b]
        pages = s["table"][b, :-(-L // P)].long()
        seen = torch.arange(L, device=DEVICE) <= torch.arange(L - n, L, device=DEVICE)[:, None]
        for h in range(Hkv):
            k = s["k_cache"][pages, h].reshape(-1, d)[:L].double()
            v = s["v_cache"][pages, h].reshape(-1, d)[:L].double()
            heads = slice(h * G, (h + 1) * G)
            for t in range(0, n, 1024):  # rows in portions that fit
                rows = slice(t, min(n, t + 1024))
                x = torch.einsum("gnd,ld->gnl", s["q"][b, heads, rows].double(), k) * s["scale"]
                x = torch.where(seen[rows], x, -torch.inf)
                lse[b, heads, rows] = torch.logsumexp(x, -1)
                o[b, heads, rows] = torch.softmax(x, -1) @ v
    return o, lse
