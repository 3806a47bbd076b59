"""Steps of a server whose prefix has a pass of its own: append, prefix pass,
own keys and (where these are split) the join run one behind the other on
inputs that change from step to step, eager and captured; rows that are no
numbers on each path.  A test first makes sure that its sizes take the path it is
for: results are joined through the workspace then, and only then is one needed."""

import pytest
import torch

import paged_ref as pr
import test_paged_gpu as tp
from exact_io_aware_bwd_b200 import binding
from exact_io_aware_bwd_b200.build import build

pytestmark = pytest.mark.gpu

DEV, BF, FP = tp.DEV, tp.BF, tp.FP


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    binding.load()


def workspace(nbytes):
    assert nbytes > 0
    return torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)


def server(dtype, wide, **kw):
    """Behind a prefix of 1024 keys; wide: with room in the table for so many
    own keys that these are split, and joined by a third kernel."""
    s = tp.Server(dtype, prefix=1024, **kw)
    if wide:
        s.table = torch.cat([s.table, torch.full((len(s.prompts), 4096 // s.P), -1, dtype=torch.int32)], 1)
    sizes = lambda pages: (len(s.prompts), s.Hq, s.Hkv, 1, s.d, s.P, pages, s.prefix)
    narrow = binding.fa_decode_prefix_workspace_bytes(*sizes(s.prefix // s.P + 2))
    here = binding.fa_decode_prefix_workspace_bytes(*sizes(s.table.shape[1]))
    assert here > narrow > 0 if wide else here == narrow > 0
    return s


@pytest.mark.parametrize("wide", [False, True], ids=["own_unsplit", "own_split"])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_steps_behind_a_long_prefix(dtype, wide):
    server(dtype, wide).run()


@pytest.mark.parametrize("wide", [False, True], ids=["own_unsplit", "own_split"])
def test_captured_steps_behind_a_long_prefix(wide):
    """Append and decode captured as one graph; each step copies its tokens
    and lengths in and replays it."""
    state = {}

    def step(s, table, freq, q, k, v, lens):
        if not state:
            for n, t in dict(q=q, k=k, v=v, lens=lens).items():
                state[n] = t.clone()
            B, Hq, _, d = q.shape
            o, lse, q_rot = torch.empty_like(q), torch.empty((B, Hq, 1), device=DEV), torch.empty_like(q)
            ws = workspace(binding.fa_decode_prefix_workspace_bytes(B, Hq, s.Hkv, 1, d, s.P, table.shape[1], s.prefix))

            def work():
                binding.fa_append_paged(state["q"], state["k"], state["v"], q_rot, None, s.kc, s.vc, table, state["lens"],
                                        None, freq)
                binding.fa_decode_prefix(q_rot, s.kc, s.vc, table, state["lens"], o, lse, pr.default_scale(d), s.prefix, ws)

            work()  # outside the capture first: loads the kernels
            torch.cuda.synchronize()
            state["graph"] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(state["graph"]):
                work()
            state["out"] = (o, lse, q_rot, ws)
        for n, t in dict(q=q, k=k, v=v, lens=lens).items():
            state[n].copy_(t)
        state["graph"].replay()
        return state["out"][:2]

    server(BF, wide, steps=8).run(step)


@pytest.mark.parametrize("wide", [0, 300], ids=["own_unsplit", "own_split"])
def test_layers_in_a_row_equal_calls_apart(wide):
    """Three layers of a step, each layer's queries the output of the one
    before, all on one workspace: back to back, and replayed as a graph, they
    give bit for bit what they give with a wait for the GPU after every call."""
    B, Hq, Hkv, d, P, prefix, layers = 5, 8, 2, 128, 16, 1024, 3
    lens0 = [prefix + 20 + 9 * b for b in range(B)]
    g = torch.Generator().manual_seed(2)
    _, _, table, _ = pr.make_cache(1, Hkv, d, P, [n + 40 for n in lens0], BF, prefix=prefix, table_slack=1 + wide)
    pages = int(table.max()) + 1
    table, freq = table.to(DEV), pr.inv_freq(d).to(DEV)
    scale = pr.default_scale(d)
    ws = workspace(binding.fa_decode_prefix_workspace_bytes(B, Hq, Hkv, 1, d, P, table.shape[1], prefix))
    start = [torch.randn((layers, pages, Hkv, P, d), generator=g).to(BF).to(DEV) for _ in range(2)]
    steps = [[torch.randn((B, h, 1, d), generator=g).to(BF).to(DEV) for h in (Hq, Hkv, Hkv)] for _ in range(10)]
    lens = [torch.tensor([n + 1 + i for n in lens0], dtype=torch.int32, device=DEV) for i in range(len(steps))]

    def buffers():
        x = [t.clone() for t in steps[0]] + [lens[0].clone()] + [t.clone() for t in start]
        return x, torch.empty_like(steps[0][0]), [torch.empty_like(steps[0][0]) for _ in range(layers)], \
            torch.empty((layers, B, Hq, 1), device=DEV)

    def work(bufs, apart):
        (q, k, v, n, kc, vc), q_rot, outs, lse = bufs
        for i in range(layers):
            binding.fa_append_paged(q if i == 0 else outs[i - 1], k, v, q_rot, None, kc[i], vc[i], table, n, None, freq)
            if apart:
                torch.cuda.synchronize()
            binding.fa_decode_prefix(q_rot, kc[i], vc[i], table, n, outs[i], lse[i], scale, prefix, ws)
            if apart:
                torch.cuda.synchronize()

    def all_steps(go):
        bufs = buffers()
        results = []
        for tokens, n in zip(steps, lens):
            for dst, src in zip(bufs[0], tokens + [n]):
                dst.copy_(src)
            go(bufs)
            results.append(([o.clone() for o in bufs[2]], bufs[3].clone()))
        torch.cuda.synchronize()
        return results

    want = all_steps(lambda bufs: work(bufs, True))
    in_a_row = all_steps(lambda bufs: work(bufs, False))
    made = {}

    def replayed(bufs):
        if not made:
            made["graph"] = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(made["graph"]):
                work(bufs, False)
        made["graph"].replay()

    in_a_graph = all_steps(replayed)
    tp.ok()
    assert bool(torch.isfinite(want[-1][1]).all())
    for got in (in_a_row, in_a_graph):
        for (a, la), (b, lb) in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(la, lb)


NOT_NUMBERS = [
    # Hq, Hkv, N, d, P, prefix, lens, table slack, whether decode / the forward
    # pass join partial results, what is special
    (8, 2, 2, 128, 16, 32, (300, 40), 1, False, False, "decode in one kernel"),
    (8, 2, 3, 128, 64, 1024, (1100, 1030, 1500), 1, True, True, "prefix pass"),
    (4, 4, 1, 64, 32, 1280, (5000, 1400), 40, True, True, "own keys split"),
    (8, 2, 130, 64, 16, 0, (400, 190), 1, None, False, "forward, pairs"),
    (8, 2, 20, 128, 16, 0, (2000, 1500), 1, None, True, "forward, keys split"),
]


@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("case", NOT_NUMBERS, ids=lambda c: c[-1].replace(" ", "_"))
def test_a_query_that_is_no_number_shows(case, bad):
    """softmax over scores with a NaN or +inf among them is NaN: so are O and
    lse of that row (a score of inf in every key of one sign, which would leave
    only -inf, does not happen with this many keys); the other rows of its
    tile, warp and sequence stay right."""
    Hq, Hkv, N, d, P, prefix, lens, slack, joins, forward_joins, _ = case
    B = len(lens)
    kc, vc, table, tl = pr.make_cache(7, Hkv, d, P, lens, BF, prefix=prefix, table_slack=slack)
    q = torch.randn((B, Hq, N, d), generator=torch.Generator().manual_seed(5)).to(BF)
    ref = pr.attention(q, kc, vc, table, lens, [N] * B, pr.default_scale(d))
    hit = torch.zeros((B, Hq, N), dtype=torch.bool)
    hit[0, 1, N - 1] = hit[B - 1, Hq - 1, 0] = True
    q[hit, 3] = bad
    dev = [t.to(DEV) for t in (q, kc, vc, table, tl)]
    sizes = (B, Hq, Hkv, N, d, P, table.shape[1])
    assert (binding.fa_fwd_paged_workspace_bytes(*sizes) > 0) == forward_joins
    calls = [binding.attention_fwd_paged(*dev)]
    if joins is not None:
        assert (binding.fa_decode_prefix_workspace_bytes(*sizes, prefix) > 0) == joins
        calls.append(binding.attention_decode_prefix(*dev, prefix))
    tp.ok()
    for o, lse in calls:
        o, lse = o.cpu(), lse.cpu()
        assert bool(torch.isnan(o[hit]).all()) and bool(torch.isnan(lse[hit]).all())
        o[hit] = torch.from_numpy(ref[0])[hit].to(BF)
        lse[hit] = torch.from_numpy(ref[1])[hit].float()
        pr.check_attention(o, lse, ref, BF, [N] * B)


@pytest.mark.parametrize("new", [None, (1, 1, 1, 1, 1)], ids=["all_new", "new_lens"])
def test_queries_of_idle_and_refused_sequences_come_back_as_zeros(new):
    """cache_append's rows that no token of the call fills, in memory that held
    NaN before: sequence 1 is idle, sequence 3 longer than its table."""
    B, Hq, Hkv, d, P = 5, 8, 2, 128, 16
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn((B, h, 1, d), generator=g).to(BF).to(DEV) for h in (Hq, Hkv, Hkv))
    caches = [torch.zeros((2 * B, Hkv, P, d), dtype=BF, device=DEV) for _ in range(2)]
    table = torch.arange(2 * B, dtype=torch.int32, device=DEV).view(B, 2)
    lens = torch.tensor([3, 0, 20, 2 * P + 1, 32], dtype=torch.int32, device=DEV)
    nl = None if new is None else torch.tensor(new, dtype=torch.int32, device=DEV)
    freq = pr.inv_freq(d).to(DEV)
    for _ in range(3):
        held = [torch.full((B, Hq, 1, d), float("nan"), dtype=BF, device=DEV) for _ in range(64)]
        del held
        out = binding.cache_append(q, k, v, *caches, table, lens, freq, nl)
        assert binding.fa_get_device_status() == binding.FA_ERR_INVALID_ARG
        assert bool((out[1] == 0).all()) and bool((out[3] == 0).all())
        for b in (0, 2, 4):
            want, mag = pr.rotated(q[b].cpu(), lens[b:b + 1].cpu() - 1, pr.inv_freq(d), False)
            pr.check_rotated(out[b].cpu(), want, mag, f"q of sequence {b}")


APPEND_ID, PAGED_ID, OWN_ID = 15, 13, 14     # bits 8-15 of the status word: the kernel that met the error


@pytest.mark.parametrize("with_out", [False, True], ids=["cache_only", "q_out_k_out"])
@pytest.mark.parametrize("bad", ["page", "page_negative", "too_long", "new_too_many", "new_negative", "short"])
def test_a_refused_append_leaves_every_other_slot_alone(bad, with_out):
    """Both whole caches bit for bit: the good sequence's tokens, those of the
    bad one that sit on good pages (none when its lengths do not fit), nothing
    else; rows of q_out and k_out of a refused sequence as they were."""
    Hq, Hkv, N, d, P = 4, 2, 20, 64, 16
    kc, vc, table, tl = pr.make_cache(3, Hkv, d, P, [40, 30], BF)
    new = torch.tensor([20, 20], dtype=torch.int32)
    good_table = table.clone()
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
    q, k, v = (torch.randn((2, h, N, d), generator=g).to(BF) for h in (Hq, Hkv, Hkv))
    want_k, want_v = kc.clone(), vc.clone()
    by_page = bad.startswith("page")
    for b, pos in ((0, torch.arange(20, 40)), (1, torch.arange(10, 16 if by_page else 10))):
        t = pos - int(pos[0]) if len(pos) else pos
        page = good_table[b].long()[pos // P]
        want_k[page, :, pos % P], want_v[page, :, pos % P] = k[b, :, t].transpose(0, 1), v[b, :, t].transpose(0, 1)
    kd, vd = kc.to(DEV), vc.to(DEV)
    q_out, k_out = (torch.full((2, h, N, d), 7.0, dtype=BF, device=DEV) if with_out else None for h in (Hq, Hkv))
    binding.fa_append_paged(q.to(DEV) if with_out else None, k.to(DEV), v.to(DEV), q_out, k_out, kd, vd, table.to(DEV),
                            tl.to(DEV), new.to(DEV), None)
    assert binding.fa_peek_device_status_word() >> 8 & 255 == APPEND_ID
    assert binding.fa_get_device_status() == binding.FA_ERR_INVALID_ARG
    bits = lambda t: t.cpu().view(torch.int16)
    assert torch.equal(bits(kd), bits(want_k)) and torch.equal(bits(vd), bits(want_v))
    if with_out:
        for got, src in ((q_out, q), (k_out, k)):
            assert torch.equal(got[0].cpu(), src[0])
            assert torch.equal(got[1].cpu(), src[1]) if by_page else bool((got[1] == 7).all())


def test_the_status_word_names_the_kernel():
    kc, vc, table, tl = pr.make_cache(3, 2, 64, 16, [40, 30], BF)
    tl[1] = table.shape[1] * 16 + 1
    dev = [t.to(DEV) for t in (kc, vc, table, tl)]
    q = torch.ones((2, 4, 3, 64), dtype=BF, device=DEV)
    for call, kernel in ((lambda: binding.attention_fwd_paged(q, *dev), PAGED_ID),
                         (lambda: binding.attention_decode_prefix(q, *dev, 16), OWN_ID)):
        call()
        assert binding.fa_peek_device_status_word() >> 8 & 255 == kernel
        assert binding.fa_get_device_status() == binding.FA_ERR_INVALID_ARG
    tp.ok()


def joining_calls(seed, dtype):
    """Calls that all join partial results through a workspace, each with its
    reference: decode behind a prefix pass, the same with its own keys split,
    the forward pass with its keys split.  (name, inputs, prefix, reference,
    new tokens, bytes needed)"""
    Hq, Hkv, d, P = 8, 2, 128, 16
    calls = []
    for i, (prefix, lens, N, slack) in enumerate(((1024, (1100, 1030, 1500), 1, 1), (2048, (2100, 2050), 4, 300))):
        kc, vc, table, tl = pr.make_cache(seed + i, Hkv, d, P, lens, dtype, prefix=prefix, table_slack=slack)
        q = torch.randn((len(lens), Hq, N, d), generator=torch.Generator().manual_seed(seed + i)).to(dtype)
        ref = pr.attention(q, kc, vc, table, lens, [N] * len(lens), pr.default_scale(d))
        dev = [t.to(DEV) for t in (q, kc, vc, table, tl)]
        sizes = (len(lens), Hq, Hkv, N, d, P, table.shape[1])
        calls.append(("prefix", dev, prefix, ref, [N] * len(lens), binding.fa_decode_prefix_workspace_bytes(*sizes, prefix)))
        calls.append(("paged", dev, prefix, ref, [N] * len(lens), binding.fa_fwd_paged_workspace_bytes(*sizes)))
    assert all(c[5] > 0 for c in calls)
    return calls


def run_call(call, o, lse, ws, stream=None):
    name, dev, prefix, _, _, _ = call
    scale = pr.default_scale(dev[0].shape[3])
    if name == "prefix":
        binding.fa_decode_prefix(*dev, o, lse, scale, prefix, ws, stream)
    else:
        binding.fa_fwd_paged(*dev, None, o, lse, scale, ws, stream)


def outputs(call):
    q = call[1][0]
    return torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device=DEV)


def test_graphs_that_join_share_a_workspace():
    """Four captured calls over one workspace, replayed in turn: neither leaves
    anything the other depends on."""
    calls = joining_calls(1, BF)
    ws = workspace(max(c[5] for c in calls))
    graphs = []
    for c in calls:
        o, lse = outputs(c)
        run_call(c, o, lse, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run_call(c, o, lse, ws)
        graphs.append((graph, o, lse))
    for order in ((0, 1, 2, 3), (3, 1, 0, 2), (2, 2, 0, 0, 1, 3, 1)):
        for i in order:
            graphs[i][1].fill_(float("nan")), graphs[i][2].fill_(float("nan"))
        for i in order:
            graphs[i][0].replay()
        for i in set(order):
            pr.check_attention(graphs[i][1], graphs[i][2], calls[i][3], BF, calls[i][4])
    tp.ok()


def test_joining_calls_on_two_streams_do_not_meet():
    """Two streams, each with a workspace of its own that all its calls use in
    turn, a row of calls in flight on both."""
    sides = []
    for seed in (10, 20):
        calls = joining_calls(seed, FP)
        sides.append((torch.cuda.Stream(), calls, workspace(max(c[5] for c in calls))))
    torch.cuda.synchronize()
    results = [[[outputs(c) for c in calls] for _ in range(5)] for _, calls, _ in sides]
    torch.cuda.synchronize()
    for turn in range(5):
        for i in range(4):
            for side, (stream, calls, ws) in enumerate(sides):
                run_call(calls[i], *results[side][turn][i], ws, stream)
    torch.cuda.synchronize()
    for (_, calls, _), turns in zip(sides, results):
        for turn in turns:
            for c, (o, lse) in zip(calls, turn):
                pr.check_attention(o, lse, c[3], FP, c[4])
    tp.ok()


@pytest.mark.parametrize("prefix", [512, 768, 784, 1024])
@pytest.mark.parametrize("B,d", [(2, 128), (40, 128), (40, 64), (90, 64), (130, 128)])
def test_prefixes_with_and_without_a_pass_of_their_own(prefix, B, d):
    """Up to 768 keys, and up to 2^24 values of a head's keys in all that the
    blocks read, are taken with the own keys; idle sequences, ones shorter than
    the prefix or ending with it among the others."""
    Hq, Hkv, Nq, P = 4, 2, 2, 16
    lens = tuple((prefix + 2 + 7 * i, 0, prefix - 3 * i - 1, prefix, prefix + 1, 2)[i % 6 if i else 0] for i in range(B))
    kc, vc, table, tl = pr.make_cache(B, Hkv, d, P, lens, BF, prefix=prefix)
    alone = prefix <= 768 and B * Hkv * prefix * d <= 1 << 24
    assert (binding.fa_decode_prefix_workspace_bytes(B, Hq, Hkv, Nq, d, P, table.shape[1], prefix) == 0) == alone
    q = torch.randn((B, Hq, Nq, d), generator=torch.Generator().manual_seed(B)).to(BF)
    ref = pr.attention(q, kc, vc, table, lens, [Nq] * B, pr.default_scale(d))
    seen = table.clone()
    seen[1:, :prefix // P] = -1
    o, lse = binding.attention_decode_prefix(q.to(DEV), kc.to(DEV), vc.to(DEV), seen.to(DEV), tl.to(DEV), prefix)
    tp.ok()
    pr.check_attention(o, lse, ref, BF, [Nq] * B)


@pytest.mark.parametrize("items", [1, 2, 3, 16, 36, 37])
def test_own_keys_split_and_not(items):
    """The number of splits is read off the workspace: two blocks per SM, or
    the nearest number to it, and no split of fewer than 1024 keys."""
    Hq, Hkv, Nq, d, P, room = 16, 8, 1, 128, 128, 8192
    B = items
    splits = max(1, min((2 * 296 + B * Hkv) // (2 * B * Hkv), room // 1024))
    nbytes = binding.fa_decode_prefix_workspace_bytes(B, Hq, Hkv, Nq, d, P, room // P, 0)
    assert nbytes == (B * Hq * Nq * splits * (d + 2) * 4 if splits > 1 else 0)
    lens = tuple((1500, 1, 900, 0, 2100)[b % 5] for b in range(B))
    kc, vc, table, tl = pr.make_cache(items, Hkv, d, P, lens, FP, table_slack=room // P - 17)
    table = torch.cat([table, torch.full((B, room // P - table.shape[1]), -1, dtype=torch.int32)], 1)
    q = torch.randn((B, Hq, Nq, d), generator=torch.Generator().manual_seed(B)).to(FP)
    ref = pr.attention(q, kc, vc, table, lens, [Nq] * B, pr.default_scale(d))
    o, lse = binding.attention_decode_prefix(*[t.to(DEV) for t in (q, kc, vc, table, tl)], 0)
    tp.ok()
    pr.check_attention(o, lse, ref, FP, [Nq] * B)


def test_a_graph_of_copies_fills_a_fork_and_the_allocating_calls():
    """The calls that allocate, captured between what a program captures with
    them: copies of the step's inputs, a fill, a second stream that runs a
    prompt's pass beside decode and joins it.  Replayed on other inputs it
    gives bit for bit what the calls give one by one."""
    B, Hq, Hkv, d, P, prefix = 6, 8, 2, 128, 32, 1024
    lens = [prefix + 3 + 11 * b for b in range(B)]
    kc, vc, table, _ = pr.make_cache(4, Hkv, d, P, [n + 30 for n in lens], BF, prefix=prefix)
    g = torch.Generator().manual_seed(9)
    table, freq = table.to(DEV), pr.inv_freq(d).to(DEV)
    caches = [torch.nan_to_num(t).to(DEV) for t in (kc, vc)]
    N = 20
    sets = [[torch.randn((B, h, n, d), generator=g).to(BF).to(DEV) for h, n in ((Hq, 1), (Hkv, 1), (Hkv, 1), (Hq, N))]
            + [torch.tensor([n + 1 + i for n in lens], dtype=torch.int32, device=DEV)] for i in range(4)]
    here = [t.clone() for t in sets[0]]
    filled = torch.zeros((4, 2), device=DEV)
    side = torch.cuda.Stream()

    def work(given, kc, vc, apart):
        wait = torch.cuda.synchronize if apart else (lambda: None)
        for dst, src in zip(here, given):
            dst.copy_(src)
        q, k, v, prompt, n = here
        filled.zero_()
        wait()
        q_rot = binding.cache_append(q, k, v, kc, vc, table, n, freq)
        wait()
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            second = binding.attention_fwd_paged(prompt, kc, vc, table, n)
        wait()
        first = binding.attention_decode_prefix(q_rot, kc, vc, table, n, prefix)
        main.wait_stream(side)
        wait()
        return q_rot, *first, *second

    want = []
    own = [c.clone() for c in caches]
    for given in sets:
        want.append([t.clone() for t in work(given, *own, True)])
    torch.cuda.synchronize()
    own2 = [c.clone() for c in caches]
    from_here = [t.clone() for t in sets[0]]
    work(from_here, *[c.clone() for c in caches], False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work(from_here, *own2, False)
    for given, expected in zip(sets, want):
        for dst, src in zip(from_here, given):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, expected))
    assert all(torch.equal(a, b) for a, b in zip(own, own2))
    tp.ok()


def test_two_threads_call_at_once():
    """Each with its own stream, workspace and inputs."""
    import threading
    torch.cuda.synchronize()
    failures = []

    def run(seed):
        try:
            calls = joining_calls(seed, BF)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                ws = workspace(max(c[5] for c in calls))
                results = [[outputs(c) for c in calls] for _ in range(8)]
                stream.synchronize()
                for turn in results:
                    for c, (o, lse) in zip(calls, turn):
                        run_call(c, o, lse, ws, stream)
                stream.synchronize()
            for turn in results:
                for c, (o, lse) in zip(calls, turn):
                    pr.check_attention(o, lse, c[3], BF, c[4])
        except BaseException as e:
            failures.append(e)

    threads = [threading.Thread(target=run, args=(s,)) for s in (30, 40)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
    tp.ok()
