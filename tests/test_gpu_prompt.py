"""prompt_attention against the plain 64-bit form: lengths, head layouts, contexts, strides,
values that are not finite, streams, graphs, workspaces."""
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


class Case:
    """Sequences of (queries, keys) tokens, `lead` rows before the first and `trail` behind the last,
    whose contents (and those of out) are NaN."""

    def __init__(self, seqs, Hq, Hkv, D, seed=0, lead=0, trail=0, packed=False, q_scale=2.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.seqs, self.Hq, self.Hkv, self.D = seqs, Hq, Hkv, D
        nq, nk = [s[0] for s in seqs], [s[1] for s in seqs]
        T, Tk = sum(nq) + lead + trail, sum(nk) + lead + trail
        start = lambda n: torch.tensor([lead] + n, device=DEV).cumsum(0).int()
        self.qs, self.ks = start(nq), start(nk)
        nan = float("nan")
        if packed:
            assert nq == nk
            x = torch.full((T, Hq + 2 * Hkv, D), nan, dtype=torch.float16, device=DEV)
            self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            self.q = torch.full((T, Hq, D), nan, dtype=torch.float16, device=DEV)
            self.k, self.v = torch.full((Tk, Hkv, D), nan, dtype=torch.float16, device=DEV), \
                torch.full((Tk, Hkv, D), nan, dtype=torch.float16, device=DEV)
        r = lambda n, H: torch.randn(n, H, D, generator=g, device=DEV)
        self.q[lead:lead + sum(nq)] = (r(sum(nq), Hq) * q_scale).half()
        self.k[lead:lead + sum(nk)], self.v[lead:lead + sum(nk)] = r(sum(nk), Hkv).half(), r(sum(nk), Hkv).half()
        self.out = torch.full((T, Hq, D), nan, dtype=torch.float16, device=DEV)
        self.lse = torch.full((T, Hq), nan, device=DEV)

    def run(self, **kw):
        import rope_kv_cache_gb300 as rk
        rk.prompt_attention(self.q, self.k, self.v, self.qs, self.out, kv_starts=self.ks, lse=self.lse, **kw)

    def verify(self, scale=None):
        torch.cuda.synchronize()
        qs, ks = self.qs.tolist(), self.ks.tolist()
        left = torch.ones(self.out.shape[0], dtype=torch.bool, device=DEV)
        for b, (nq, nk) in enumerate(self.seqs):
            if nq == 0:
                continue
            at, kt = slice(qs[b], qs[b] + nq), slice(ks[b], ks[b] + nk)
            o, l, to, tl = sp.attend(self.q[at], self.k[kt], self.v[kt], sp.causal(nq, nk, DEV), scale)
            sp.check(self.out[at], o, to, f"out of sequence {b}")
            sp.check(self.lse[at], l, tl, f"lse of sequence {b}")
            left[at] = False
        assert self.out[left].isnan().all() and self.lse[left].isnan().all(), "rows of no sequence were written"


same = lambda *n: [(x, x) for x in n]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seqs", [same(1), same(2), same(31, 33), same(63, 64, 65), same(127), same(128), same(129),
                                  same(255, 256, 257), same(1, 300, 0, 5, 0, 64), same(515), same(1030)])
def test_lengths(seqs, D):
    c = Case(seqs, 4, 2, D, seed=D, lead=3, trail=2)
    c.run()
    c.verify()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (3, 1), (5, 1), (10, 2), (7, 1), (8, 1), (16, 1), (16, 2), (12, 2),
                                    (71, 1), (128, 1), (129, 1), (300, 1), (9, 3), (257, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_heads(Hq, Hkv, D):
    c = Case(same(70, 1, 131), Hq, Hkv, D, seed=Hq, lead=1, trail=1, packed=Hq % 2 == 0)
    c.run()
    c.verify()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seqs", [[(1, 1000)], [(1, 129), (17, 128), (3, 64)], [(100, 1000), (1, 1), (200, 201)],
                                  [(300, 1200)], [(5, 3), (300, 20), (1, 0), (130, 0), (2, 1)], [(0, 77), (4, 77)],
                                  [(257, 400), (0, 0), (64, 640)]])
def test_chunks_behind_a_context_and_queries_that_see_nothing(seqs, D):
    c = Case(seqs, 8, 2, D, seed=len(seqs), lead=2, trail=5)
    c.run()
    c.verify()


@pytest.mark.parametrize("lens", [[3] * 200, [1] * 500, [0] * 40 + [9] + [0] * 70 + [130, 0], list(range(70)),
                                  [(7 * b) % 4 for b in range(2000)], [0] * 900 + [300] + [0] * 900])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_sequences(lens, D):
    c = Case(same(*lens), 4, 1, D, seed=len(lens), lead=1, trail=1)
    c.run()
    c.verify()


@pytest.mark.parametrize("D,scale", [(64, 0.0), (64, -0.125), (128, 1.0), (256, -1.0), (128, 1e-30), (64, 30.0)])
def test_scales(D, scale):
    c = Case(same(200, 40), 4, 2, D, seed=3, q_scale=1.0 if abs(scale) < 2 else 0.25)
    c.run(sm_scale=scale)
    c.verify(scale)


def test_growing_scores():
    """Every key scores higher than those before by more than the running maximum may lag."""
    c = Case(same(700), 2, 1, 128, seed=9)
    ramp = torch.linspace(0, 40, 700, device=DEV)
    c.q[:] = 0
    c.q[..., 0] = 8
    c.k[:, 0, 0] = ramp.half()
    c.run()
    c.verify()
    c.k[:, 0, 0] = ramp.flip(0).half()
    c.run()
    c.verify()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_values(D):
    c = Case(same(300, 77), 4, 2, D, seed=5)
    c.v.copy_(torch.where(c.v > 0, 65504.0, -65504.0).half())
    c.v[:, 1] = 65504.0
    c.run()
    c.verify()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("where", [0, 63, 130, 200, 299])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(D, where):
    c = Case(same(300, 260), 4, 2, D, seed=where, lead=1)
    c.v[1 + where, 0, 5] = float("inf")
    c.v[1 + where, 1, D - 1] = float("nan")
    c.v[1 + 300 + min(where, 259), 0, 7] = float("-inf")
    c.run()
    c.verify()


@pytest.mark.parametrize("D", [64, 128])
def test_values_that_are_not_finite_in_many_short_sequences(D):
    c = Case([(20, 20 + 60 * (b % 3)) for b in range(50)], 8, 2, D, seed=D, lead=1, trail=2)
    for b in range(0, 50, 7):
        at = c.ks[b].item() + c.seqs[b][1] - 10
        c.v[at, b % 2, 3 * b % D] = [float("inf"), float("nan"), float("-inf")][b % 3]
    c.run()
    c.verify()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seqs", [same(400, 131), [(30, 90)] * 40, [(5, 1200)]])
def test_values_that_are_not_finite_in_many_places(D, seqs):
    # in one column: of a row, seen ones and others; weights are far above FP16's least
    c = Case(seqs, 8, 2, D, seed=D, lead=1, trail=2, q_scale=1.0)
    g = torch.Generator(device=DEV).manual_seed(D)
    at = torch.rand(c.v.shape, generator=g, device=DEV)
    for x, bad in enumerate(["nan", "inf", "-inf"]):
        c.v[(at > x * 1e-3) & (at < x * 1e-3 + 5e-4)] = float(bad)
    c.run()
    c.verify()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_keys_that_are_not_finite_do_not_reach_rows_before_them(D, bad):
    c = Case(same(200, 150), 4, 2, D, seed=1)
    c.k[130] = bad
    c.run()
    torch.cuda.synchronize()
    got, lse = c.out.clone(), c.lse.clone()
    c.k[130] = 0
    c.run()
    c.verify()
    assert torch.equal(got[:130], c.out[:130]) and torch.equal(lse[:130], c.lse[:130])
    assert torch.equal(got[200:], c.out[200:]) and torch.equal(lse[200:], c.lse[200:])
    if bad != bad:
        assert got[130:200].isnan().all() and lse[130:200].isnan().all()


def test_queries_that_are_not_finite_stay_in_their_rows():
    c = Case(same(200), 4, 2, 128, seed=2)
    c.run()
    torch.cuda.synchronize()
    want = c.out.clone()
    c.q[77, 1] = float("nan")
    c.run()
    torch.cuda.synchronize()
    assert c.out[77, 1].isnan().all()
    c.out[77, 1] = want[77, 1]
    assert torch.equal(c.out, want)


@pytest.mark.parametrize("starts", [[0, 10, 5, 40], [-7, 3, 50], [20, 90, 1000], [2000, 3000], [5, 4, 3]])
def test_starts_out_of_range_read_and_write_within_the_tensors(starts):
    import rope_kv_cache_gb300 as rk
    c = Case(same(64), 4, 2, 64, seed=4)
    s = torch.tensor(starts, dtype=torch.int32, device=DEV)
    guard = torch.full((64 + 2, 4, 64), 7.0, dtype=torch.float16, device=DEV)
    rk.prompt_attention(c.q, c.k, c.v, s, guard[1:65], kv_starts=s)
    torch.cuda.synchronize()
    assert (guard[0] == 7).all() and (guard[65] == 7).all() and guard.isfinite().all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_out_at_every_multiple_of_16_bytes(D):
    c = Case(same(70, 200), 4, 2, D, seed=8)
    c.run()
    c.verify()
    want = c.out
    for off in (8, 16, 24):
        flat = torch.full((c.out.numel() + 64,), 7.0, dtype=torch.float16, device=DEV)
        c.out = flat[off:off + want.numel()].view(want.shape)
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want) and (flat[:off] == 7).all() and (flat[off + want.numel():] == 7).all()


def test_nothing_to_do():
    import rope_kv_cache_gb300 as rk
    e = lambda *s: torch.empty(*s, dtype=torch.float16, device=DEV)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    rk.prompt_attention(e(0, 4, 64), e(0, 2, 64), e(0, 2, 64), z, e(0, 4, 64))
    out = torch.full((5, 4, 64), 3.0, dtype=torch.float16, device=DEV)
    rk.prompt_attention(e(5, 4, 64), e(5, 2, 64), e(5, 2, 64), z, out)                  # no sequence
    two = torch.tensor([1, 4], dtype=torch.int32, device=DEV)
    rk.prompt_attention(torch.zeros_like(out), e(0, 2, 64), e(0, 2, 64), two, out, kv_starts=two)   # no keys at all
    torch.cuda.synchronize()
    assert (out[1:4] == 0).all() and (out[0] == 3).all() and (out[4] == 3).all()


def test_default_starts_streams_and_workspaces():
    import rope_kv_cache_gb300 as rk
    c = Case(same(300, 41), 8, 2, 128, seed=6, packed=True)
    c.run()
    c.verify()
    size = rk.prompt_attention_workspace_size(c.q, c.k, c.v, c.qs)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(c.out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rk.prompt_attention(c.q, c.k, c.v, c.qs, out, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, c.out)
    with pytest.raises(rk.RopeKVError):
        rk.prompt_attention(c.q, c.k, c.v, c.qs, out, workspace=ws[:size - 16])


def test_equal_calls_give_equal_bits_from_graphs_too():
    import rope_kv_cache_gb300 as rk
    c = Case([(700, 900), (3, 3000), (129, 129)], 8, 2, 128, seed=7)
    c.run()
    c.verify()
    want, wl = c.out.clone(), c.lse.clone()
    ws = torch.empty(rk.prompt_attention_workspace_size(c.q, c.k, c.v, c.qs, c.ks), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            c.run(workspace=ws)
    for _ in range(20):
        c.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want) and torch.equal(c.lse, wl)
    # the same graph with other lengths: the launch depends on the sizes alone
    c.seqs = [(1, 1), (800, 4000), (31, 28)]
    c.qs.copy_(torch.tensor([0, 1, 801, 832]))
    c.ks.copy_(torch.tensor([0, 1, 4001, 4029]))
    c.out.fill_(float("nan"))
    c.lse.fill_(float("nan"))
    g.replay()
    c.verify()


def test_random_calls():
    import random
    rng = random.Random(11)
    for seed in range(40):
        D, Hkv, G = rng.choice([64, 128, 256]), rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 4, 5, 8, 14])
        seqs = []
        for _ in range(rng.choice([1, 1, 2, 5, 17])):
            nq = int(2 ** rng.uniform(0, 9.5)) - (rng.random() < 0.1)
            nk = nq if rng.random() < 0.5 else max(0, nq + int(2 ** rng.uniform(0, 11)) - rng.choice([0, 0, 50]))
            seqs.append((nq, nk))
        c = Case(seqs, Hkv * G, Hkv, D, seed=seed, lead=rng.choice([0, 1]), trail=rng.choice([0, 4]))
        c.run()
        c.verify()
