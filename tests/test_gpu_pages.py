"""Rows of accepted drafts moved, pages copied, forked and freed, against plain lists; every byte
of the caches that is not named stays as it was."""
import random

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


def pool(pages, tpp, Hkv, D, fmt, seed):
    """Random bits: (cache, scales, the cache as bits)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = {"f16": torch.float16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[fmt]
    raw = torch.randint(0, 256, (2, pages, tpp, Hkv, D * (2 if fmt == "f16" else 1)), generator=g, device=DEV, dtype=torch.uint8)
    scales = None if fmt == "f16" else torch.rand(2, pages, Hkv, tpp, generator=g, device=DEV)
    return raw.view(dt), scales, raw


def paths(rng, B, S, A):
    """Accepted nodes: ascending paths, some with entries that are skipped."""
    acc, lens = [], []
    for b in range(B):
        row = sorted(rng.sample(range(S), min(A, S))) + [rng.randrange(-3, S + 3) for _ in range(max(0, A - S))]
        if b % 4 == 3:
            row = [rng.randrange(-2, S + 2) for _ in range(A)]
        acc.append(row)
        lens.append(rng.choice([0, 1, A, A, rng.randrange(-1, A + 3)]))
    return acc, lens


@pytest.mark.parametrize("B,S,A,Hkv,D,cap", [(1, 1, 1, 1, 64, 5), (5, 16, 5, 2, 64, 60), (9, 61, 8, 8, 128, 100),
                                             (7, 40, 23, 3, 256, 64), (3, 300, 300, 1, 128, 310), (4, 4, 9, 2, 64, 12)])
def test_accepted_drafts_of_a_contiguous_cache(B, S, A, Hkv, D, cap):
    import rope_kv_cache_gb300 as rk
    rng = random.Random(S)
    acc, n = paths(rng, B, S, A)
    lens = [rng.choice([S, cap, rng.randrange(0, cap + 4), S // 2]) for _ in range(B)]
    cache = torch.randint(-32768, 32768, (B, 2, Hkv, cap, D), device=DEV, dtype=torch.int16).view(torch.float16)
    before = cache.view(torch.int16).clone()
    new, want_lens = sp.accept(lambda b, p: before[b, :, :, p], lens, S, acc, n, cap)
    # a source that an earlier entry of the call overwrote would be one at or before it: there is none
    out = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    rk.kv_accept_drafts(cache, i32(lens), S, i32(acc), i32(n), out)
    torch.cuda.synchronize()
    for (b, p), x in new.items():
        before[b, :, :, p] = x
    assert torch.equal(cache.view(torch.int16), before)
    assert out.tolist() == [w if l >= S else -7 for w, l in zip(want_lens, lens)]
    ends = i32(lens)
    rk.kv_accept_drafts(cache, ends, S, i32([[j for j in range(A)]] * B), i32(n), ends)     # nothing moves
    torch.cuda.synchronize()
    assert torch.equal(cache.view(torch.int16), before) and ends.tolist() == want_lens


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("B,S,A,Hkv,D,tpp,M", [(1, 1, 1, 1, 64, 16, 1), (6, 16, 5, 2, 64, 16, 4), (9, 61, 8, 8, 128, 64, 3),
                                               (5, 20, 20, 3, 256, 7, 9), (3, 300, 260, 1, 128, 32, 10)])
def test_accepted_drafts_of_a_paged_cache(B, S, A, Hkv, D, tpp, M, fmt):
    import rope_kv_cache_gb300 as rk
    rng = random.Random(S + tpp)
    acc, n = paths(rng, B, S, A)
    P = B * M + 3
    ids, vids = rng.sample(range(P), B * M), rng.sample(range(P, 2 * P), B * M)
    table = [[ids[b * M:(b + 1) * M], vids[b * M:(b + 1) * M]] for b in range(B)]
    for b in range(0, B, 3):                    # unmapped and wrong pages, each plane on its own
        table[b][rng.randrange(2)][rng.randrange(M)] = rng.choice([-1, -9, 2 * P, P if False else 2 * P + 5])
    lens = [rng.choice([S, M * tpp, rng.randrange(0, M * tpp + 4)]) for _ in range(B)]
    cache, scales, raw = pool(P, tpp, Hkv, D, fmt, S)
    want, wscales = raw.clone(), None if scales is None else scales.clone()
    for plane in (0, 1):
        def rows(b, p, plane=plane):
            i = table[b][plane][p // tpp] - plane * P
            return (i, p % tpp) if 0 <= i < P else None
        new, want_lens = sp.accept(rows, lens, S, acc, n, M * tpp)
        for (b, p), (i, r) in new.items():
            to, tr = rows(b, p)
            want[plane, to, tr] = raw[plane, i, r]
            if scales is not None:
                wscales[plane, to, :, tr] = scales[plane, i, :, r]
    out = i32(lens)
    rk.paged_kv_accept_drafts(cache, i32(table), out, S, i32(acc), i32(n), out, kv_scales=scales)
    torch.cuda.synchronize()
    assert torch.equal(raw, want) and out.tolist() == want_lens
    assert scales is None or torch.equal(scales, wscales)


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("N,tpp,Hkv,D", [(1, 1, 1, 64), (3, 16, 2, 64), (40, 64, 8, 128), (7, 5, 3, 256), (300, 32, 1, 128)])
def test_page_copies(N, tpp, Hkv, D, fmt):
    import rope_kv_cache_gb300 as rk
    rng = random.Random(N)
    P = 2 * N + 3
    cache, scales, raw = pool(P, tpp, Hkv, D, fmt, N)
    order = rng.sample(range(P), 2 * N)
    src, dst = order[:N], order[N:]
    src[0], dst[-1] = rng.choice([src[0], -1, P]), rng.choice([dst[-1], -5, P, 2 * P])
    if N > 2:
        src[1] = dst[1]                          # onto itself
        src[2] = src[N - 1]                      # one source for two
    want, wscales = raw.clone(), None if scales is None else scales.clone()
    for s, d in zip(src, dst):
        if 0 <= s < P and 0 <= d < P:
            want[:, d] = raw[:, s]
            if scales is not None:
                wscales[:, d] = scales[:, s]
    rk.paged_kv_copy_pages(cache, i32(src), i32(dst), kv_scales=scales)
    torch.cuda.synchronize()
    assert torch.equal(raw, want) and (scales is None or torch.equal(scales, wscales))


class Pool:
    """B sequences over P pages, some shared; the plain lists beside the tensors."""

    def __init__(self, rng, B, M, P, tpp, Hkv, D, fmt, live):
        self.tpp, self.B, self.P = tpp, B, P
        self.cache, self.scales, self.raw = pool(P, tpp, Hkv, D, fmt, B)
        free = rng.sample(range(P), P)
        self.table, self.lens, self.refs = [[[-1] * M, [-1] * M] for _ in range(B)], [0] * B, [0] * P
        for b in live:
            n = rng.choice([0, 1, tpp, M * tpp, rng.randrange(0, M * tpp + 1), M * tpp + 3 if b == live[0] else 1])
            n = min(n, (len(free) - 2) * tpp) if n <= M * tpp else n
            for col in range(min(M, -(-n // tpp))):
                p = free.pop()
                self.refs[p] += 1
                self.table[b][0][col], self.table[b][1][col] = p, p + P
            self.lens[b] = n
        self.g = [i32(self.table), i32(self.lens), i32(self.refs)]

    def fork(self, parents, children, **kw):
        import rope_kv_cache_gb300 as rk
        want, ws = self.raw.clone(), None if self.scales is None else self.scales.clone()
        for s, d, n in sp.fork(self.table, self.lens, self.refs, parents, children, self.tpp):
            want[:, d, :n] = self.raw[:, s, :n]
            if ws is not None:
                ws[:, d, :, :n] = self.scales[:, s, :, :n]
        rk.paged_kv_fork(self.cache, *self.g, i32(parents), i32(children), kv_scales=self.scales, **kw)
        torch.cuda.synchronize()
        assert torch.equal(self.raw, want) and (ws is None or torch.equal(self.scales, ws))
        self.same()

    def free(self, sequences, keep=None):
        import rope_kv_cache_gb300 as rk
        sp.free(self.table, self.lens, self.refs, sequences, keep, self.tpp)
        rk.paged_kv_free(*self.g, i32(sequences), tokens_per_page=self.tpp, keep_lens=None if keep is None else i32(keep))
        torch.cuda.synchronize()
        self.same()

    def same(self):
        assert self.g[0].tolist() == self.table
        assert self.g[1].tolist() == self.lens
        assert self.g[2].tolist() == self.refs


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("B,M,P,tpp,Hkv,D", [(4, 3, 20, 16, 2, 64), (30, 6, 120, 64, 8, 128), (12, 1, 40, 5, 3, 256),
                                             (40, 300, 2000, 4, 1, 64), (6, 4, 25, 32, 1, 128)])
def test_forks_and_frees(B, M, P, tpp, Hkv, D, fmt):
    rng = random.Random(B + M)
    half = B // 2
    s = Pool(rng, B, M, P, tpp, Hkv, D, fmt, list(range(half)))
    kids = list(range(half, B))
    s.fork([rng.randrange(half) for _ in kids], kids)
    s.fork([rng.randrange(half) for _ in kids], kids)                    # not empty: skipped
    s.free(kids[::2] + kids[:1] + [-1, B, B + 7])                        # one named twice, some out of range
    s.free([0, kids[-1]], keep=[tpp + 1, 1])
    s.fork([kids[-1]] * len(kids[::2]), kids[::2])                       # a fork of a fork
    s.free(list(range(B)))
    assert all(x == 0 for x in s.refs)


def test_forks_that_are_skipped():
    rng = random.Random(3)
    s = Pool(rng, 12, 4, 40, 16, 2, 64, "f16", [0, 1, 2])
    s.lens[1] = 20
    s.g[1][1] = 20
    #  twice named, a parent too, out of range, itself
    s.fork([0, 1, 1, 4, 1, -1, 1, 12, 2], [5, 5, 6, 7, 4, 8, 12, 9, 2])
    s.fork([0, 1], [-5, 40])
    s.fork([1], [10])


def test_forks_without_free_pages():
    """Three forks with a partly filled page and two free pages: the third ends with its last whole page."""
    import rope_kv_cache_gb300 as rk
    s = Pool(random.Random(1), 6, 4, 5, 16, 1, 64, "int8", [])
    s.table[0] = [[4, 1, -1, -1], [9, 6, -1, -1]]
    s.lens[0], s.refs[:] = 20, [0, 1, 3, 0, 1]
    s.table[5], s.lens[5] = [[4, -1, -1, -1], [9, -1, -1, -1]], 24       # its partly filled page is unmapped
    s.g = [i32(s.table), i32(s.lens), i32(s.refs)]
    ws = torch.full((rk.paged_kv_fork_workspace_size(4, 6),), 0xff, dtype=torch.uint8, device=DEV)
    s.fork([5, 0, 0, 0], [4, 3, 2, 1], workspace=ws)
    assert s.lens == [20, 16, 20, 20, 16, 24]
    with pytest.raises(rk.RopeKVError):
        rk.paged_kv_fork(s.cache, *s.g, i32([0]), i32([1]), kv_scales=s.scales, workspace=ws[:16])


def test_page_0_is_a_page_like_any_other():
    """Page 0 is free and goes to the first fork; the forks behind it have no partly filled page."""
    s = Pool(random.Random(2), 6, 3, 8, 16, 2, 64, "f16", [])
    s.table[0], s.lens[0] = [[5, 2, -1], [13, 10, -1]], 20
    s.table[1], s.lens[1] = [[7, -1, -1], [15, -1, -1]], 16
    s.refs[:] = [0, 1, 1, 1, 1, 1, 0, 1]
    s.g = [i32(s.table), i32(s.lens), i32(s.refs)]
    s.fork([0, 1, 1, 0], [2, 3, 4, 5])
    assert s.table[2][0] == [5, 0, -1] and s.table[5][0] == [5, 6, -1] and s.table[3][0] == [7, -1, -1]


def test_many_forks_over_a_large_pool():
    """More forks than one scan takes, free pages far up among 70000."""
    import rope_kv_cache_gb300 as rk
    N, P, tpp = 2500, 70001, 2
    table = torch.full((N + 1, 2, 2), -1, dtype=torch.int32, device=DEV)
    table[0, :, 0], table[0, 0, 1], table[0, 1, 1] = i32([7, 7 + P]), 9, 9 + P
    lens, refs = torch.zeros(N + 1, dtype=torch.int32, device=DEV), torch.ones(P, dtype=torch.int32, device=DEV)
    lens[0] = 3
    free = torch.arange(16, P, 25, device=DEV)
    refs[free] = 0
    cache = torch.randn(2, P, tpp, 1, 64, device=DEV).half()
    want = cache.clone()
    want[:, free[:N], :1] = cache[:, 9:10, :1]
    kids = torch.randperm(N, device=DEV).int() + 1
    rk.paged_kv_fork(cache, table, lens, refs, torch.zeros(N, dtype=torch.int32, device=DEV), kids)
    torch.cuda.synchronize()
    assert torch.equal(cache, want) and (lens[1:] == 3).all() and int(refs[7]) == N + 1 and int(refs[9]) == 1
    assert torch.equal(table[kids.long(), 0, 1].long(), free[:N]) and torch.equal(table[1:, 1, 1], table[1:, 0, 1] + P)
    assert (refs[free[:N]] == 1).all() and (refs[free[N:]] == 0).all()


def test_frees_forks_and_copies_follow_one_another_in_a_graph():
    """Launched without a gap: free the children, fork them anew, copy their pages away; every
    replay finds the state of the one before."""
    import rope_kv_cache_gb300 as rk
    s = Pool(random.Random(9), 40, 8, 400, 16, 2, 64, "e4m3", list(range(10)))
    kids = list(range(10, 40))
    parents = [(7 * i) % 10 for i in range(30)]
    k, p = i32(kids), i32(parents)
    src, dst = i32(list(range(0, 200))), i32(list(range(200, 400)))
    ws = torch.empty(rk.paged_kv_fork_workspace_size(30, 40), dtype=torch.uint8, device=DEV)

    def step(wait=lambda: None):
        rk.paged_kv_free(*s.g, k)
        wait()
        rk.paged_kv_fork(s.cache, *s.g, p, k, kv_scales=s.scales, workspace=ws)
        wait()
    step(torch.cuda.synchronize)
    want = [x.clone() for x in s.g]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(4):
            step()
    for _ in range(30):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s.g, want))
    del src, dst
