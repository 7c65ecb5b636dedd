"""The operators on whole sequences together with the writes around them, as a serving loop
uses them: launched one behind another without a gap (each a dependent of the one before), from a
graph too, and compared with the same calls that were waited for and with the 64-bit form."""
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


def table(rows, r):
    ang = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * 1e4 ** (-2.0 * torch.arange(r // 2, device=DEV) / r)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


class Loop:
    """Prompt, a tree of drafts, its accepted path, and a decode step over the contiguous cache."""

    def __init__(self, B, S0, S, Hq, Hkv, D, seed):
        import rope_kv_cache_gb300 as rk
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.B, self.S0, self.S, self.Hq, self.Hkv, self.D, self.cap = B, S0, S, Hq, Hkv, D, S0 + 2 * S + 3
        r = lambda n: torch.randn(B, n, Hq + 2 * Hkv, D, generator=g, device=DEV).half()
        self.first, self.drafts, self.one = r(S0), r(S), r(1)
        self.cs = table(self.cap, D)[None].contiguous()
        parents = [[-1] + [max(0, i - 1 - (i * 7 + b) % 3) for i in range(1, S)] for b in range(B)]
        depth = [[0] * S for _ in range(B)]
        for b in range(B):
            for i in range(1, S):
                depth[b][i] = depth[b][parents[b][i]] + 1
        self.mask = rk.tree_mask_from_parents(parents).to(DEV)
        # the path down to the last node
        paths = []
        for b in range(B):
            p, i = [], S - 1
            while i >= 0:
                p.insert(0, i)
                i = parents[b][i]
            paths.append(p)
        A = max(map(len, paths))
        self.accepted, self.counts = i32([p + [0] * (A - len(p)) for p in paths]), i32([len(p) for p in paths])
        self.pos = (S0 + torch.tensor(depth, device=DEV)).int()
        self.starts = (torch.arange(B + 1, device=DEV) * S0).int()
        self.end_tree, self.ends, self.end_one = i32([S0 + S] * B), i32([0] * B), i32([0] * B)
        e = lambda n: torch.zeros(B, n, Hq, D, dtype=torch.float16, device=DEV)
        self.o1, self.o2, self.o3, self.q2, self.q3 = e(S0), e(S), e(1), e(S), e(1)
        self.cache = torch.zeros(B, 2, Hkv, self.cap, D, dtype=torch.float16, device=DEV)
        self.packed = torch.empty_like(self.first)

    def run(self, wait=lambda: None):
        import rope_kv_cache_gb300 as rk
        B, S0, Hq, Hkv, D = self.B, self.S0, self.Hq, self.Hkv, self.D
        self.packed.copy_(self.first)
        rk.rope_write_kv_packed(self.cs, self.packed, self.cache, Hq, Hkv)
        wait()
        x = self.packed.view(B * S0, Hq + 2 * Hkv, D)
        rk.prompt_attention(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], self.starts, self.o1.view(B * S0, Hq, D))
        wait()
        rk.rope_write_kv_tree(self.cs, self.end_tree, self.pos, self.drafts, self.cache, self.q2, Hq, Hkv)
        wait()
        rk.tree_attention(self.q2, self.cache, self.end_tree, self.o2, tree_mask=self.mask)
        wait()
        rk.kv_accept_drafts(self.cache, self.end_tree, self.S, self.accepted, self.counts, self.ends)
        wait()
        torch.add(self.ends, 1, out=self.end_one)
        rk.rope_write_kv_continuous(self.cs, self.end_one, self.one, self.cache, self.q3, Hq, Hkv)
        wait()
        rk.tree_attention(self.q3, self.cache, self.end_one, self.o3)
        wait()
        return [t.clone() for t in (self.o1, self.o2, self.o3, self.cache, self.end_one)]


@pytest.mark.parametrize("B,S0,S,Hq,Hkv,D", [(3, 200, 26, 8, 2, 64), (2, 700, 61, 32, 8, 128), (5, 33, 9, 6, 2, 256)])
def test_prompt_drafts_acceptance_and_decode(B, S0, S, Hq, Hkv, D):
    c = Loop(B, S0, S, Hq, Hkv, D, seed=S)
    want = c.run(torch.cuda.synchronize)
    for _ in range(5):
        c.cache.zero_()
        got = c.run()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = c.run()
    for _ in range(10):
        c.cache.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # against the 64-bit form, from what the writes left
    x = c.packed
    ends = c.ends.tolist()
    for b in range(B):
        o, _, tol, _ = sp.attend(x[b, :, :Hq], x[b, :, Hq:Hq + Hkv], x[b, :, Hq + Hkv:], sp.causal(S0, S0, DEV))
        sp.check(c.o1[b], o, tol, f"prompt {b}")
        n = ends[b] + 1
        assert n == S0 + c.counts[b].item() + 1
        k, v = c.cache[b, :, :, :n].transpose(1, 2)
        o, _, tol, _ = sp.attend(c.q3[b], k, v, torch.ones(1, n, dtype=torch.bool, device=DEV))
        sp.check(c.o3[b], o, tol, f"decode {b}")
    # the accepted path, written again as a chain of its own, leaves the same cache
    import rope_kv_cache_gb300 as rk
    for b in range(B):
        n = c.counts[b].item()
        path = c.accepted[b, :n].long()
        again = c.cache[b:b + 1].clone()
        again[:, :, :, S0:S0 + n] = 0
        rk.rope_write_kv_continuous(c.cs, i32([S0 + n]), c.drafts[b:b + 1, path].contiguous(), again,
                                    torch.zeros(1, n, Hq, D, dtype=torch.float16, device=DEV), Hq, Hkv)
        torch.cuda.synchronize()
        assert torch.equal(again[:, :, :, :S0 + n], c.cache[b:b + 1, :, :, :S0 + n])


@pytest.mark.parametrize("fmt", ["f16", "int8", "e4m3"])
def test_chunks_forks_and_frees_of_a_paged_cache(fmt):
    """A prompt in two chunks over a paged cache (written, read back, attended to), two forks that
    decode on, and everything given back."""
    import rope_kv_cache_gb300 as rk
    g = torch.Generator(device=DEV).manual_seed(3)
    Hq, Hkv, D, tpp, n1, n2, P, M = 8, 2, 128, 16, 70, 51, 40, 9
    n = n1 + n2
    dt = {"f16": torch.float16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[fmt]
    pool = torch.zeros(2, P, tpp, Hkv, D, dtype=torch.uint8 if fmt == "e4m3" else dt, device=DEV).view(dt)
    scales = None if fmt == "f16" else torch.zeros(2, P, Hkv, tpp, device=DEV)
    cs = table(256, D)
    page_table = torch.full((3, 2, M), -1, dtype=torch.int32, device=DEV)
    pages = torch.randperm(P, generator=g, device=DEV)[:8].int()
    page_table[0, 0, :8], page_table[0, 1, :8] = pages, pages + P
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    refs[pages.long()] = 1
    lens = i32([n, 0, 0])
    x = torch.randn(n, Hq + 2 * Hkv, D, generator=g, device=DEV).half()
    q_out = torch.zeros(n, Hq, D, dtype=torch.float16, device=DEV)
    out = torch.zeros_like(q_out)
    rows = lambda m: torch.zeros(m, Hkv, D, dtype=torch.float16, device=DEV)

    def write(x, seq, first, q_out):
        pos = first + torch.arange(x.shape[0], device=DEV)
        slots = page_table[seq, 0][pos // tpp].long() * tpp + pos % tpp
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        if fmt == "f16":
            rk.rope_write_kv_slot_mapping(cs, pos, q, k, v, slots, pool[0], pool[1], q_out)
        else:
            rk.rope_write_kv_slot_mapping_quant(cs, pos, q, k, v, slots, pool[0], pool[1], scales[0], scales[1], q_out)
    for lo, hi in ((0, n1), (n1, n)):
        write(x[lo:hi], 0, lo, q_out[lo:hi])
        k, v = rows(hi), rows(hi)
        rk.paged_kv_read(pool, page_table, torch.arange(hi, device=DEV).int(), i32([0] * hi), k, v, kv_scales=scales)
        rk.prompt_attention(q_out[lo:hi], k, v, i32([0, hi - lo]), out[lo:hi], kv_starts=i32([0, hi]))
    torch.cuda.synchronize()
    o, _, tol, _ = sp.attend(q_out, k, v, sp.causal(n, n, DEV))
    sp.check(out, o, tol, "chunks")
    # two forks, each with one more token of its own
    rk.paged_kv_fork(pool, page_table, lens, refs, i32([0, 0]), i32([1, 2]), kv_scales=scales)
    new = torch.randn(2, 1, Hq + 2 * Hkv, D, generator=g, device=DEV).half()
    q1 = torch.zeros(3, 1, Hq, D, dtype=torch.float16, device=DEV)
    parent = [t.clone() for t in ((pool.view(torch.uint8)[:, pages.long()],) if scales is None else
                                  (pool.view(torch.uint8)[:, pages.long()], scales[:, pages.long()]))]
    for b in (1, 2):
        write(new[b - 1], b, n, q1[b])
    att = torch.zeros_like(q1)
    kv = i32([0, n + 1, n + 1])
    rk.paged_attention_shared_prefix(q1, pool, None, 0, page_table, kv, att, kv_scales=scales)
    torch.cuda.synchronize()
    now = (pool.view(torch.uint8)[:, pages.long()],) + (() if scales is None else (scales[:, pages.long()],))
    assert all(torch.equal(a, b) for a, b in zip(parent, now)), "a fork's write reached its parent"
    assert lens.tolist() == [n, n, n] and sorted(refs[pages.long()].tolist()) == [1] + [3] * 7
    for b in (1, 2):
        k, v = rows(n + 1), rows(n + 1)
        rk.paged_kv_read(pool, page_table, torch.arange(n + 1, device=DEV).int(), i32([b] * (n + 1)), k, v, kv_scales=scales)
        # the same attention as a chunk of one token over the rows read back
        one = torch.zeros(1, Hq, D, dtype=torch.float16, device=DEV)
        rk.prompt_attention(q1[b], k, v, i32([0, 1]), one, kv_starts=i32([0, n + 1]))
        torch.cuda.synchronize()
        o, _, tol, _ = sp.attend(q1[b], k, v, torch.ones(1, n + 1, dtype=torch.bool, device=DEV))
        sp.check(one, o, tol, f"fork {b} by its rows")
        # 8-bit: the attention decodes exactly, the rows read back were rounded to FP16 (2^-11 of each)
        more = 0 if fmt == "f16" else 4 * 2.0 ** -11 * (1 + q1[b].abs().max().item() * k.abs().max().item() * D ** 0.5) * v.abs().max().item()
        sp.check(att[b], o, tol + more, f"fork {b} by its pages")
    rk.paged_kv_free(page_table, lens, refs, i32([1, 2]), tokens_per_page=tpp, keep_lens=i32([n1, 0]))
    rk.paged_kv_free(page_table, lens, refs, i32([0]))
    torch.cuda.synchronize()
    assert lens.tolist() == [0, n1, 0] and (page_table[[0, 2]] == -1).all() and (page_table[1, :, -(-n1 // tpp):] == -1).all()
    assert sorted(refs[pages.long()].tolist()) == [0] * 3 + [1] * 5 and int(refs.sum()) == 5
