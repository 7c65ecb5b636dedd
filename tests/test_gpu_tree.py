"""tree_attention against the plain 64-bit form: chains and trees, lengths, head layouts, slots out
of range, values that are not finite, long caches, graphs."""
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


def trees(B, S, g):
    """Random trees as mask words; the words' unused bits are random too."""
    import rope_kv_cache_gb300 as rk
    parents = [[-1] + [int(torch.randint(max(0, i - 9), i, (1,), generator=g)) for i in range(1, S)] for _ in range(B)]
    mask = rk.tree_mask_from_parents(parents)
    if S % 32:
        junk = torch.randint(-2 ** 31, 2 ** 31, mask[..., -1].shape, generator=g)
        keep = (1 << S % 32) - 1
        word = mask[..., -1].long() & 0xffffffff & keep | (junk & 0xffffffff & ~keep)
        mask[..., -1] = torch.where(word >= 2 ** 31, word - 2 ** 32, word).int()
    return mask.to(DEV)


class Case:
    """ends[b]: where sequence b ends with its S new tokens; slots that no token sees hold NaN."""

    def __init__(self, ends, S, Hq, Hkv, D, cap, tree, seed=0, q_scale=2.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        B = len(ends)
        self.ends, self.S, self.cap = ends, S, cap
        self.lens = torch.tensor(ends, dtype=torch.int32, device=DEV)
        self.cache = torch.randn(B, 2, Hkv, cap, D, generator=g, device=DEV).half()
        for b, e in enumerate(ends):
            self.cache[b, :, :, max(0, min(e, cap)):] = float("nan")
        self.q = (torch.randn(B, S, Hq, D, generator=g, device=DEV) * q_scale).half()
        self.mask = trees(B, S, torch.Generator().manual_seed(seed)) if tree else None
        self.out = torch.full((B, S, Hq, D), float("nan"), dtype=torch.float16, device=DEV)
        self.lse = torch.full((B, S, Hq), float("nan"), device=DEV)

    def run(self, **kw):
        import rope_kv_cache_gb300 as rk
        rk.tree_attention(self.q, self.cache, self.lens, self.out, tree_mask=self.mask, lse=self.lse, **kw)

    def verify(self, scale=None, only=None):
        torch.cuda.synchronize()
        for b, e in enumerate(self.ends):
            if only is not None and b not in only:
                continue
            n = max(0, min(e, self.cap))
            j = torch.arange(n, device=DEV) - (e - self.S)                 # number of the new token at each slot
            new = sp.tree_sees(self.mask[b], self.S) if self.mask is not None else \
                torch.ones(self.S, self.S, dtype=torch.bool, device=DEV).tril()
            sees = (j < 0)[None] | ((j >= 0)[None] & new[:, j.clamp(0, self.S - 1)])
            k, v = self.cache[b, :, :, :n].transpose(1, 2)
            o, l, to, tl = sp.attend(self.q[b], k, v, sees, scale)
            sp.check(self.out[b], o, to, f"out of sequence {b}")
            sp.check(self.lse[b], l, tl, f"lse of sequence {b}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("S,tree", [(1, False), (1, True), (2, False), (7, True), (26, True), (31, False), (32, True),
                                    (33, True), (61, True), (64, False), (65, True), (100, True), (129, True), (200, False)])
def test_new_tokens(S, tree, D):
    c = Case([S, S + 1, S + 60, S + 128, 500], S, 8, 2, D, max(500, S + 130), tree, seed=S)
    c.run()
    c.verify()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (3, 1), (5, 1), (14, 2), (8, 1), (64, 1), (71, 1), (200, 1), (257, 1)])
def test_heads(Hq, Hkv, D):
    for S, tree in ((1, False), (6, True)):
        c = Case([300, 6, 77], S, Hq, Hkv, D, 300, tree, seed=Hq)
        c.run()
        c.verify()


@pytest.mark.parametrize("tree", [False, True])
def test_ends_out_of_range(tree):
    """Inactive sequences, fewer slots than new tokens, ends behind the cache and far outside."""
    S = 5
    c = Case([0, 1, 3, 5, 64, 66, 70, 2000, 2 ** 31 - 1, -3, -2 ** 31], S, 4, 2, 64, 64, tree, seed=8)
    c.run()
    c.verify()


def test_masks_that_hide_everything_or_name_later_tokens():
    c = Case([9, 200, 131, 64], 9, 4, 2, 128, 200, True, seed=1)
    c.mask[0] = 0                       # no context either: nothing is seen
    c.mask[1] = 0
    c.mask[2] = -1                      # all see all
    c.mask[3, :4] = 0x100
    c.run()
    c.verify()
    assert (c.out[0] == 0).all() and (c.lse[0] == -float("inf")).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("S", [1, 8, 40])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(S, D):
    c = Case([S + 100, S + 3, 300], S, 8, 2, D, 300, S > 1, seed=S)
    c.cache[0, 1, 0, 100 + S // 2, 3] = float("inf")        # a new token
    c.cache[1, 1, 1, S + 2, D - 1] = float("nan")
    c.cache[2, 1, 1, 17, 0] = float("-inf")                 # the context
    c.run()
    c.verify()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("S", [1, 12, 70])
def test_values_that_are_not_finite_in_many_places(S, D):
    c = Case([S + 900, S + 3, 300], S, 8, 2, D, 1000, True, seed=S, q_scale=1.0)
    g = torch.Generator(device=DEV).manual_seed(D)
    at = torch.rand(c.cache[:, 1].shape, generator=g, device=DEV)
    for x, bad in enumerate(["nan", "inf", "-inf"]):
        c.cache[:, 1][(at > x * 1e-3) & (at < x * 1e-3 + 5e-4)] = float(bad)
    c.run()
    c.verify()


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales(scale):
    c = Case([300, 44], 7, 4, 2, 128, 300, True, seed=2, q_scale=1.0)
    c.run(sm_scale=scale)
    c.verify(scale)


def test_large_values_and_growing_scores():
    c = Case([900, 300], 3, 4, 2, 64, 900, False, seed=3)
    c.cache[:, 1].copy_(torch.where(c.cache[:, 1] > 0, 65504.0, -65504.0).half())
    c.q[:] = 0
    c.q[..., 0] = 8
    c.cache[0, 0, :, :, 0] = torch.linspace(0, 60, 900, device=DEV).half()
    c.run()
    c.verify()


@pytest.mark.parametrize("B,S,cap,D", [(1, 1, 9000, 128), (2, 1, 40000, 64), (1, 61, 20000, 128), (3, 4, 7000, 256),
                                       (40, 1, 3000, 128), (200, 1, 260, 64), (200, 1, 260, 128), (60, 9, 400, 128),
                                       (60, 9, 2000, 64), (30, 26, 700, 64)])
def test_long_and_many(B, S, cap, D):
    ends = [cap if b == 0 else S + (b * 7919) % (cap - S) for b in range(B)]
    c = Case(ends, S, 8, 2, D, cap, S > 1, seed=B)
    c.run()
    c.verify(only=set(range(0, B, max(1, B // 8))))


def test_offsets_past_32_bits():
    """4.3 G elements: the last sequences' rows lie past 2^32 elements."""
    import rope_kv_cache_gb300 as rk
    B, Hkv, cap, D, S = 9, 8, 131072, 256, 2
    cache = torch.empty(B, 2, Hkv, cap, D, dtype=torch.float16, device=DEV)
    assert cache.numel() > 2 ** 32
    ends = [500, 7, 2, 300, 9, 77, 64, 1, 600]
    small = Case(ends, S, 8, Hkv, D, 600, False, seed=4)
    for b, e in enumerate(ends):
        cache[b, :, :, :e] = small.cache[b, :, :, :e]
        cache[b, :, :, e:e + 300] = float("nan")
    small.run()
    small.verify()
    out = torch.empty_like(small.out)
    rk.tree_attention(small.q, cache, small.lens, out)
    torch.cuda.synchronize()
    small.out.copy_(out)
    rk.tree_attention(small.q, cache, small.lens, out, lse=small.lse)
    small.verify()
    # one sequence that ends at the cache's last slots
    small2 = Case([130], S, 8, Hkv, D, 130, False, seed=5)
    cache[8, :, :, cap - 200:cap - 70] = 0
    lens = small.lens.clone()
    lens[8] = cap
    cache[8] = 0
    cache[8, 0, :, :, 0] = -1
    cache[8, 0, :, cap - 64:, 0] = 100
    cache[8, 1, :, cap - 64:] = 3
    q = torch.zeros_like(small.q)
    q[..., 0] = 8
    rk.tree_attention(q, cache, lens, out)
    torch.cuda.synchronize()
    assert (out[8] == 3).all()


def test_graphs_streams_and_workspaces():
    import rope_kv_cache_gb300 as rk
    c = Case([3000, 61, 400, 0], 61, 8, 2, 128, 3000, True, seed=6)
    c.run()
    c.verify()
    want, wl = c.out.clone(), c.lse.clone()
    size = rk.tree_attention_workspace_size(c.q, c.cache)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            c.run(workspace=ws)
    for _ in range(20):
        c.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want) and torch.equal(c.lse, wl)
    c.ends = [61, 3000, 62, 1000]
    c.cache.nan_to_num_(0.25)
    c.lens.copy_(torch.tensor(c.ends))
    g.replay()
    c.verify()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want.copy_(c.out)
    c.out.fill_(0)
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    assert torch.equal(c.out, want)


def test_nothing_to_do():
    import rope_kv_cache_gb300 as rk
    e = lambda *s: torch.empty(*s, dtype=torch.float16, device=DEV)
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    rk.tree_attention(e(0, 1, 4, 64), e(0, 2, 2, 8, 64), z, e(0, 1, 4, 64))
    out = torch.full((2, 1, 4, 64), 3.0, dtype=torch.float16, device=DEV)
    rk.tree_attention(torch.zeros_like(out), e(2, 2, 2, 0, 64), torch.ones(2, dtype=torch.int32, device=DEV), out)
    torch.cuda.synchronize()
    assert (out == 0).all()
