"""The operators on whole sequences where they are easily wrong: weights far below the largest,
infinities behind them, waits that give up, children whose rows still name pages, large batches."""
import pytest

import sequence_plain as sp

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rope_kv_cache_gb300 import build
    build.build_library()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prompt(q, k, v, nq, nk, **kw):
    """One sequence of nq queries that are the last of nk tokens: (out, lse)."""
    import rope_kv_cache_gb300 as rk
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device=DEV)
    rk.prompt_attention(q, k, v, i32([0, nq]), out, kv_starts=i32([0, nk]), lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def decode(q, k, v, **kw):
    """The same call of tree_attention: the keys lie in a contiguous cache."""
    import rope_kv_cache_gb300 as rk
    cache = torch.stack([k.transpose(0, 1), v.transpose(0, 1)])[None].contiguous()
    out, lse = torch.full_like(q, float("nan"))[None], torch.full(q.shape[:2], float("nan"), device=DEV)[None]
    rk.tree_attention(q[None].contiguous(), cache, i32([k.shape[0]]), out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out[0], lse[0]


def test_waits_that_run_out_leave_nan_in_every_row():
    """Calls that end as if a wait inside the kernel had run out at once. Nothing of an earlier call's rows
    or pieces may be left then: whole units, cut ones and their joins are all NaN."""
    import ctypes

    import rope_kv_cache_gb300 as rk
    fail = rk.load_serving_library().ropekv_sequence_fail
    fail.argtypes, fail.restype = [ctypes.c_int], ctypes.c_int
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).half()
    for D, Hq, Hkv, seqs in [(64, 8, 2, [(1, 1)]), (64, 8, 2, [(30, 30)] * 200), (128, 8, 2, [(3, 4000), (700, 900), (0, 9), (5, 2)]),
                             (128, 32, 8, [(300, 300)] * 32), (128, 6, 2, [(1, 30000)]), (256, 8, 1, [(70, 2000), (1, 9000), (129, 129)])]:
        nq, nk = sum(s[0] for s in seqs), sum(s[1] for s in seqs)
        start = lambda i: torch.tensor([1] + [s[i] for s in seqs], device=DEV).cumsum(0).int()
        q, k, v, qs, ks = r(nq + 2, Hq, D), r(nk + 2, Hkv, D), r(nk + 2, Hkv, D), start(0), start(1)
        ws = torch.zeros(rk.prompt_attention_workspace_size(q, k, v, qs, ks), dtype=torch.uint8, device=DEV)
        out, lse = torch.zeros_like(q), torch.zeros(nq + 2, Hq, device=DEV)
        call = lambda: rk.prompt_attention(q, k, v, qs, out, kv_starts=ks, lse=lse, workspace=ws)
        call()
        torch.cuda.synchronize()
        want, wl = out.clone(), lse.clone()
        assert want.isfinite().all() and not wl.isnan().any()
        assert fail(1) == 0
        try:
            call()
            torch.cuda.synchronize()
        finally:
            assert fail(0) == 1
        assert out[1:-1].isnan().all() and lse[1:-1].isnan().all(), (D, seqs[:3])
        assert (out[[0, -1]] == 0).all() and (lse[[0, -1]] == 0).all()
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    for D, S, cap, ends in [(64, 1, 260, [100 + b for b in range(100)]), (128, 26, 3000, [3000, 26, 1000, 0]), (256, 9, 5000, [5000])]:
        q, cache, lens = r(len(ends), S, 8, D), r(len(ends), 2, 2, cap, D), i32(ends)
        ws = torch.zeros(rk.tree_attention_workspace_size(q, cache), dtype=torch.uint8, device=DEV)
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device=DEV)
        call = lambda: rk.tree_attention(q, cache, lens, out, lse=lse, workspace=ws)
        call()
        torch.cuda.synchronize()
        want, wl = out.clone(), lse.clone()
        assert fail(1) == 0
        try:
            call()
            torch.cuda.synchronize()
        finally:
            fail(0)
        assert out.isnan().all() and lse.isnan().all()
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("lens,Hq,Hkv,D", [((40, 41), 8, 2, 64), ((5000, 5001), 8, 2, 64), ((2000, 700), 16, 2, 128),
                                           ((300, 1), 4, 1, 256)])
def test_a_million_empty_sequences_between_two(lens, Hq, Hkv, D):
    """What is shared out ends behind the first sequence, or goes on behind all the empty ones."""
    import rope_kv_cache_gb300 as rk
    B = 1 << 20
    g = torch.Generator(device=DEV).manual_seed(D)
    T = sum(lens)
    r = lambda H: torch.randn(T, H, D, generator=g, device=DEV).half()
    q, k, v, out = r(Hq), r(Hkv), r(Hkv), torch.full((T, Hq, D), float("nan"), dtype=torch.float16, device=DEV)
    lse = torch.full((T, Hq), float("nan"), device=DEV)
    starts = torch.full((B + 1,), lens[0], dtype=torch.int32, device=DEV)
    starts[0], starts[-1] = 0, T
    rk.prompt_attention(q, k, v, starts, out, lse=lse)
    torch.cuda.synchronize()
    for at in (slice(0, lens[0]), slice(lens[0], T)):
        n = at.stop - at.start
        o, l, to, tl = sp.attend(q[at], k[at], v[at], sp.causal(n, n, DEV))
        sp.check(out[at], o, to, "out")
        sp.check(lse[at], l, tl, "lse")


@pytest.mark.parametrize("D", [64, 128])
def test_both_tensor_core_attentions_in_turn(D):
    """A shared prefix's attention and one of many short prompts, launched one behind the other without a
    gap: kernels of half an SM that could start beside the other's."""
    import rope_kv_cache_gb300 as rk
    g = torch.Generator(device=DEV).manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).half()
    B, S, Hq, Hkv, tpp, P, M = 16, 3, 8, 2, 16, 600, 4
    prefix = P // tpp + 1
    pages = prefix + B * M
    pool, q1, att = r(2, pages, tpp, Hkv, D), r(B, S, Hq, D), torch.zeros(B, S, Hq, D, dtype=torch.float16, device=DEV)
    ids = torch.arange(pages, device=DEV).int()
    shared = torch.stack([ids[:prefix], ids[:prefix] + pages])
    own = ids[prefix:].view(B, 1, M)
    table = torch.cat([shared[0].expand(B, 1, -1), own], 2)
    table = torch.cat([table, table + pages], 1).contiguous()
    lens = (P + S + torch.arange(B, device=DEV) * 2).int()
    n = 250
    x, out = r(n * 30, Hq + 2 * Hkv, D), torch.zeros(n * 30, Hq, D, dtype=torch.float16, device=DEV)
    starts = (torch.arange(n + 1, device=DEV) * 30).int()

    def step(wait=lambda: None):
        for _ in range(3):
            rk.paged_attention_shared_prefix(q1, pool, shared, P, table, lens, att)
            wait()
            rk.prompt_attention(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], starts, out)
            wait()
    step(torch.cuda.synchronize)
    want = att.clone(), out.clone()
    assert all(w.isfinite().all() and w.abs().sum() > 0 for w in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        att.zero_()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(att, want[0]) and torch.equal(out, want[1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("distance", [10, 12, 14, 16])
@pytest.mark.parametrize("nq,nk", [(3000, 3000), (40, 3000), (4, 20000)])
def test_many_small_weights_beside_a_large_one(nq, nk, distance, D):
    """The first token holds most of the weight and has a zero V, all others score `distance` lower. A
    weight is rounded to FP16 as 2^7 times what it is relative to the largest (or more, where the
    running maximum lags): 2^-11 of itself, or 2^-25 of 2^-7 below FP16's normal range. To that come
    2^-17 for what roundings of scores up to 16 (five of 2^-24) and ex2 (2^-22) do to a weight, the sums'
    N 2^-23 (of O and l) and the result's rounding, 2^-11 or 2^-25. lse: ten roundings of at most 24 2^-24
    in log2 units, and the sum's."""
    g = torch.Generator(device=DEV).manual_seed(distance)
    q = torch.zeros(nq, 4, D, dtype=torch.float16, device=DEV)
    q[..., 0] = 1
    k = torch.zeros(nk, 2, D, dtype=torch.float16, device=DEV)
    k[0, :, 0] = distance
    v = (100 * (1 + torch.rand(nk, 2, D, generator=g, device=DEV))).half()
    v[0] = 0
    n = nk - nq + 1 + torch.arange(nq, device=DEV, dtype=torch.float64)          # keys of each row
    sums = v.double().cumsum(0)[nk - nq:].repeat_interleave(2, 1)                  # of the V of those but the first
    w = torch.tensor(-float(distance), dtype=torch.float64, device=DEV).exp()
    L = (1 + (n - 1) * w)[:, None, None]
    want = w * sums / L
    tol = sums / L * max(2.0 ** -11 * w, 2.0 ** -32) + want * (2.0 ** -11 + 2.0 ** -17 + 2 * n[:, None, None] * 2.0 ** -23) + 2.0 ** -25
    for call in (lambda: prompt(q, k, v, nq, nk, sm_scale=1.0), lambda: decode(q, k, v, sm_scale=1.0)):
        out, lse = call()
        sp.check(out, want, tol, "out")
        sp.check(lse, (distance + L[..., 0].log()).expand(nq, 4), torch.full((1, 1), 2.0 ** -16, dtype=torch.float64, device=DEV) + n[:, None] * 2.0 ** -23, "lse")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq,nk", [(300, 300), (5, 1200), (1, 20000), (90, 91)])
def test_infinities_of_any_weight_reach_the_rows_that_see_them(nq, nk, D):
    """Tokens that score 20 to 2000 lower than the others: their weights are positive all the same,
    so that an infinity among their V is one in out (two of both signs: NaN)."""
    g = torch.Generator(device=DEV).manual_seed(D + nq)
    q = torch.randn(nq, 4, D, generator=g, device=DEV).half()
    k, v = (torch.randn(nk, 2, D, generator=g, device=DEV).half() for _ in range(2))
    q[..., 0], k[..., 0] = 1, 0
    lower = [20, 60, 100, 300, 2000]
    for i, d in enumerate(lower):
        at = [0, nk // 3, nk // 2, nk - 2, nk - 1][i]
        k[at, :, 0] = -d
        v[at, i % 2, 7 * i + 1] = float("inf") if i != 2 else -float("inf")
        v[at, 1, 50] = float("inf")
        if i == 4:
            v[at, 1, 50] = -float("inf")
    o, l, to, tl = sp.attend(q, k, v, sp.causal(nq, nk, DEV), 0.5)
    for call in (lambda: prompt(q, k, v, nq, nk, sm_scale=0.5), lambda: decode(q, k, v, sm_scale=0.5)):
        out, lse = call()
        sp.check(out, o, to, "out")
        sp.check(lse, l, tl, "lse")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinities_before_scores_that_rise_far(D):
    """Infinities that O holds when the running maximum rises by more than FP32's exponents."""
    nk = 700
    q = torch.zeros(nk, 2, D, dtype=torch.float16, device=DEV)
    q[..., 0] = 8
    k = torch.zeros(nk, 1, D, dtype=torch.float16, device=DEV)
    k[:, 0, 0] = torch.linspace(0, 1000, nk, device=DEV).half()
    v = torch.randn(nk, 1, D, generator=torch.Generator(device=DEV).manual_seed(D), device=DEV).half()
    v[3, 0, 5], v[200, 0, 6], v[400, 0, 7] = float("inf"), -float("inf"), float("nan")
    o, l, to, tl = sp.attend(q, k, v, sp.causal(nk, nk, DEV))
    for call in (lambda: prompt(q, k, v, nk, nk), lambda: decode(q, k, v)):
        out, lse = call()
        sp.check(out, o, to, "out")
        sp.check(lse, l, tl, "lse")


@pytest.mark.parametrize("fmt", ["f16", "int8"])
def test_a_child_whose_row_still_names_pages_gives_them_up(fmt):
    """Sequences of length 0 with mapped pages, as no accepted draft leaves them: a fork counts their old
    entries down, and afterwards every count is the number of table entries that name the page."""
    import rope_kv_cache_gb300 as rk
    B, M, P, tpp, S = 7, 4, 30, 16, 20
    dt = torch.float16 if fmt == "f16" else torch.int8
    cache = torch.randint(-100, 100, (2, P, tpp, 2, 64), device=DEV, dtype=torch.int8).to(dt)
    scales = None if fmt == "f16" else torch.rand(2, P, 2, tpp, device=DEV)
    table = torch.full((B, 2, M), -1, dtype=torch.int32)
    rows = {0: [3, 9, 4], 1: [3, 11], 2: [20, 21], 3: [22, 23, 24], 4: [3, 9, 25, 26], 5: [27]}
    for b, r in rows.items():
        table[b, 0, :len(r)] = torch.tensor(r)
        table[b, 1, :len(r)] = torch.tensor(r) + P
    table[4, 0, 3], table[4, 1, 3] = 999, -7                  # names no page
    count = lambda t: torch.bincount(t[:, 0][(t[:, 0] >= 0) & (t[:, 0] < P)].long().flatten().cpu(), minlength=P).int()
    refs = count(table).to(DEV)
    table = table.to(DEV)
    lens = i32([40, 20, S, S, S, S, 0])
    # nothing of the drafts is accepted: lengths of 0, pages still mapped
    rk.paged_kv_accept_drafts(cache, table, lens, S, torch.zeros(B, 0, dtype=torch.int32, device=DEV),
                              i32([0] * B), lens, kv_scales=scales)
    assert lens.tolist() == [20, 0, 0, 0, 0, 0, 0]
    lens[1] = 20                                              # sequences 0 and 1 go on
    # 3 and 4 from sequence 0 (of whose pages 4 shares two), 2 and 6 from 1; 5 twice: skipped
    before, bits = table.clone(), cache.clone()
    rk.paged_kv_fork(cache, table, lens, refs, i32([0, 0, 1, 1, 0, 1]), i32([3, 4, 2, 6, 5, 5]), kv_scales=scales)
    torch.cuda.synchronize()
    assert torch.equal(count(table), refs.cpu()), "counts are not the numbers of entries"
    assert lens.tolist() == [20, 20, 20, 20, 20, 0, 20] and torch.equal(table[[0, 1, 5]], before[[0, 1, 5]])
    # the free pages before the call, the lowest first, one for each fork's partly filled page
    assert table[:, 0].tolist()[2:5] + table[6:, 0].tolist() == [[3, 2, -1, -1], [3, 0, -1, -1], [3, 1, -1, -1], [3, 5, -1, -1]]
    assert torch.equal(cache[:, [2, 5], :4], bits[:, [11, 11], :4]) and torch.equal(cache[:, [0, 1], :4], bits[:, [9, 9], :4])
    for p in (20, 21, 22, 23, 24, 25):
        assert refs[p] == 0, f"page {p} is nobody's and not free"
    rk.paged_kv_free(table, lens, refs, i32(list(range(B))))
    torch.cuda.synchronize()
    assert (refs == 0).all() and (table == -1).all()


def test_forks_of_batches_of_very_different_sizes_at_once():
    """Host threads, each with a stream and tensors of its own: batches that need from 48 to 96 KB of
    shared memory for their plans. (By ctypes, which lets the calls overlap.)"""
    import ctypes
    import threading

    import rope_kv_cache_gb300 as rk
    lib, failures = rk.load_serving_library(), []

    class Batch:
        def __init__(self, B):
            self.B, self.stream = B, torch.cuda.Stream()
            self.table = torch.full((B, 2, 2), -1, dtype=torch.int32, device=DEV)
            self.table[0, :, 0] = i32([1, 9])
            self.lens, self.refs = torch.zeros(B, dtype=torch.int32, device=DEV), i32([0, 1, 0, 0, 0, 0, 0, 0])
            self.lens[0] = 3
            self.cache = torch.randn(2, 8, 4, 1, 64, device=DEV).half()
            self.parent, self.kid = i32([0]), i32([B - 1])
            self.ws = torch.empty(rk.paged_kv_fork_workspace_size(1, B), dtype=torch.uint8, device=DEV)

        def fork(self):
            p = lambda t: ctypes.c_void_p(t.data_ptr())
            return lib.paged_kv_fork(p(self.cache), None, p(self.table), p(self.lens), p(self.refs), p(self.parent),
                                     p(self.kid), p(self.ws), self.ws.numel(), 1, self.B, 1, 64, 8, 2, 4, 0,
                                     ctypes.c_void_p(self.stream.cuda_stream))

    def work(b):
        for _ in range(20000):                       # (after the first: the child is not empty, nothing to do)
            rc = b.fork()
            if rc != 0:
                failures.append((b.B, rc))
                return
    batches = [Batch(B) for B in (1 << 18, 200000, 150000, 140000)]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(b,)) for b in batches]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    for b in batches:
        assert b.lens[b.B - 1] == 3 and b.table[b.B - 1, 0].tolist() == [0, -1] and b.refs.tolist()[:2] == [1, 1]
        assert torch.equal(b.cache[:, 0, :3], b.cache[:, 1, :3])


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
def test_forked_pages_copied_away_in_a_graph(fmt):
    """Free, fork, copy the forks' own pages away, launched without a gap: the copies take what the forks
    have just written. Before every replay, pages written by forks and copies are filled with other bits."""
    import rope_kv_cache_gb300 as rk
    B, M, P, tpp, Hkv, D, live = 40, 8, 400, 16, 2, 64, 10
    g = torch.Generator(device=DEV).manual_seed(5)
    dt = {"f16": torch.float16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[fmt]
    raw = torch.randint(0, 256, (2, P, tpp, Hkv, D * (2 if fmt == "f16" else 1)), generator=g, device=DEV, dtype=torch.uint8)
    cache = raw.view(dt)
    scales = None if fmt == "f16" else torch.rand(2, P, Hkv, tpp, generator=g, device=DEV)
    table, lens = torch.full((B, 2, M), -1, dtype=torch.int32), [0] * B
    refs = torch.zeros(P, dtype=torch.int32)
    refs[300:] = 1                                     # where the copies go: nobody's to fork into
    for b in range(live):
        lens[b] = 16 * (b % M) + 1 + b                 # none is a multiple of a page
        ids = torch.arange(8 * b + 100, 8 * b + 100 + -(-lens[b] // tpp))
        table[b, 0, :len(ids)], table[b, 1, :len(ids)] = ids.int(), ids.int() + P
        refs[ids] += 1
        assert (refs[:300] <= 1).all()
    table, lens, refs = table.to(DEV), i32(lens), refs.to(DEV)
    kids, parents = i32(list(range(live, B))), i32([(7 * i) % live for i in range(B - live)])
    n = B - live                                       # the forks' pages: the lowest free ones, 0 .. n - 1
    src, dst = i32(list(range(n)) + [100]), i32(list(range(300, 300 + n + 1)))
    ws = torch.empty(rk.paged_kv_fork_workspace_size(n, B), dtype=torch.uint8, device=DEV)

    def step(wait=lambda: None):
        rk.paged_kv_free(table, lens, refs, kids)
        wait()
        rk.paged_kv_fork(cache, table, lens, refs, parents, kids, kv_scales=scales, workspace=ws)
        wait()
        rk.paged_kv_copy_pages(cache, src, dst, kv_scales=scales)
        wait()

    def spoil(x):
        raw[:, :n] = raw[:, 300:301 + n][:, :n] = x
        raw[:, 300 + n] = x
        if scales is not None:
            scales[:, :n] = scales[:, 300:300 + n] = scales[:, 300 + n:301 + n] = float(x)
    spoil(1)
    step(torch.cuda.synchronize)
    state = [t.clone() for t in (table, lens, refs)]
    # by hand: the forks' pages and their copies hold the first tokens of the parents' last pages
    for i in range(n):
        b = int(parents[i])
        full, rest = divmod(int(lens[b]), tpp)
        tail = int(table[b, 0, full])
        for p in (i, 300 + i):
            assert torch.equal(raw[:, p, :rest], raw[:, tail, :rest]) and (raw[:, p, rest:] == 1).all()
            assert scales is None or torch.equal(scales[:, p, :, :rest], scales[:, tail, :, :rest])
    assert torch.equal(raw[:, 300 + n], raw[:, 100])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in range(2, 30):
        spoil(x)
        torch.cuda.synchronize()
        want, wscales = raw.clone(), None if scales is None else scales.clone()
        for i in range(n):
            b = int(parents[i])
            full, rest = divmod(int(lens[b]), tpp)
            tail = int(table[b, 0, full])
            for p in (i, 300 + i):
                want[:, p, :rest] = raw[:, tail, :rest]
                if scales is not None:
                    wscales[:, p, :, :rest] = scales[:, tail, :, :rest]
        want[:, 300 + n] = raw[:, 100]
        if scales is not None:
            wscales[:, 300 + n] = scales[:, 100]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(raw, want) and (scales is None or torch.equal(scales, wscales))
        assert all(torch.equal(a, b) for a, b in zip((table, lens, refs), state))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_whose_scores_are_all_minus_infinity(D):
    """Tokens 0 to 149 score -infinity for every query: a zero row and an lse of -infinity before token 150,
    without them behind, in whole units and in cut ones."""
    g = torch.Generator(device=DEV).manual_seed(D)
    for nq, nk in ((300, 300), (160, 9000)):
        q, k, v = (torch.randn(n, H, D, generator=g, device=DEV).half() for n, H in ((nq, 4), (nk, 2), (nk, 2)))
        q[..., 0] = 1
        hidden = nk - nq + 150
        k[:hidden, :, 0] = -float("inf")
        i, t = torch.arange(nq, device=DEV)[:, None] + nk - nq, torch.arange(nk, device=DEV)[None]
        clean = k.clone()
        clean[:hidden] = 0
        o, l, to, tl = sp.attend(q, clean, v, (t <= i) & (t >= hidden))
        for out, lse in (prompt(q, k, v, nq, nk), decode(q, k, v)):
            assert (out[:150] == 0).all() and (lse[:150] == -float("inf")).all()
            sp.check(out, o, to, "out")
            sp.check(lse, l, tl, "lse")
