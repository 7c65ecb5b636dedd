"""Serving calls that follow one another on a stream without a gap, each reading what the
one before it has just overwritten: read, 8-bit write, read again, as one graph, so that
several of the launches (each a dependent of the one before) are on the GPU at once."""
import numpy as np
import pytest

import serving_plain as sp

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rope_kv_cache_gb300 import build
    build.build_library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T,Hkv,D", [(1, 8, 128), (40, 8, 128), (300, 2, 64), (600, 8, 128), (1216, 8, 128), (700, 4, 256)])
def test_reads_between_writes_see_the_newest_codes_and_scales(T, Hkv, D, fmt):
    import rope_kv_cache_gb300 as rk
    rng = np.random.Generator(np.random.PCG64(T + D))
    Hq, bs, steps = Hkv, 16, 12
    blocks = -(-T // bs) + 1
    dtype = torch.float8_e4m3fn if fmt == "e4m3" else torch.int8
    pool = torch.zeros(2, blocks, bs, Hkv, D, dtype=torch.uint8, device=DEV).view(dtype)
    scales = torch.zeros(2, blocks, Hkv, bs, device=DEV)
    perm = rng.permutation(blocks)
    p = np.arange(T)
    slots, pos = dev(perm[p // bs] * bs + p % bs), dev(p)
    rpos, rseq = dev(p.astype(np.int32)), dev(np.zeros(T, np.int32))
    table = dev(np.stack([perm, perm + blocks])[None].astype(np.int32))
    tab = dev(sp.table(T, D))
    # rows of very different sizes, so that an old scale or an old code shows
    rows = [dev((rng.standard_normal((T, Hq + 2 * Hkv, D)) * 4.0 ** (i % 5)).astype(np.float16)) for i in range(steps)]
    q_out = torch.empty(T, Hq, D, dtype=torch.float16, device=DEV)

    def write(x):
        rk.rope_write_kv_slot_mapping_quant(tab, pos, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots, pool[0],
                                            pool[1], scales[0], scales[1], q_out)

    def read(out):
        rk.paged_kv_read(pool, table, rpos, rseq, out[0], out[1], kv_scales=scales)
    want = torch.empty(steps, 2, T, Hkv, D, dtype=torch.float16, device=DEV)
    for i, x in enumerate(rows):
        write(x)
        torch.cuda.synchronize()
        read(want[i])
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    got = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i, x in enumerate(rows):
            write(x)
            read(got[i])
    for _ in range(40):
        got.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("N", [64, 1200, 6000, 40000])
def test_many_reads_of_few_tokens_between_their_writes(N, fmt):
    """Every SM reads the same four tokens, whose write is one small launch: the next read
    begins to launch while the last rows of the one before are still on their way."""
    import rope_kv_cache_gb300 as rk
    rng = np.random.Generator(np.random.PCG64(N))
    T, Hkv, D, bs, steps = 4, 8, 128, 16, 16
    dtype = torch.float8_e4m3fn if fmt == "e4m3" else torch.int8
    pool = torch.zeros(2, 1, bs, Hkv, D, dtype=torch.uint8, device=DEV).view(dtype)
    scales = torch.zeros(2, 1, Hkv, bs, device=DEV)
    slots, table = dev(np.arange(T)), dev(np.array([[[0], [1]]], np.int32))
    p = dev((np.arange(N) % T).astype(np.int32))
    seq = dev(np.zeros(N, np.int32))
    tab = dev(sp.table(T, D))
    rows = [dev((rng.standard_normal((T, 3 * Hkv, D)) * 4.0 ** (i % 5)).astype(np.float16)) for i in range(steps)]
    q_out = torch.empty(T, Hkv, D, dtype=torch.float16, device=DEV)

    def write(x):
        rk.rope_write_kv_slot_mapping_quant(tab, slots, x[:, :Hkv], x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:], slots, pool[0],
                                            pool[1], scales[0], scales[1], q_out)

    def read(out, n=N):
        rk.paged_kv_read(pool, table, p[:n], seq[:n], out[0], out[1], kv_scales=scales)
    want = torch.empty(steps, 2, T, Hkv, D, dtype=torch.float16, device=DEV)
    for i, x in enumerate(rows):
        write(x)
        torch.cuda.synchronize()
        read(want[i], T)
        torch.cuda.synchronize()
    got = torch.empty(steps, 2, N, Hkv, D, dtype=torch.float16, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i, x in enumerate(rows):
            write(x)
            read(got[i])
    for _ in range(20):
        got.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.view(steps, 2, N // T, T, Hkv, D), want[:, :, None].expand(-1, -1, N // T, -1, -1, -1))


def test_metadata_reads_and_metadata_again():
    """The row lists of a read are written by the launch before it, over those of the last read."""
    import rope_kv_cache_gb300 as rk
    rng = np.random.Generator(np.random.PCG64(5))
    B, width, Hkv, D, tpp, M, steps = 40, 8, 2, 128, 16, 4, 16
    pages = B * M
    pool = dev(rng.standard_normal((2, pages, tpp, Hkv, D)).astype(np.float16))
    ids = rng.permutation(pages).reshape(B, M)
    table = dev(np.stack([ids, ids + pages], 1).astype(np.int32))
    old = [dev(rng.integers(0, M * tpp - width, B).astype(np.int32)) for _ in range(steps)]
    n = [dev(rng.integers(0, width + 1, B).astype(np.int32)) for _ in range(steps)]
    pos, seq = torch.empty(B * width, dtype=torch.int32, device=DEV), torch.empty(B * width, dtype=torch.int32, device=DEV)

    def step(i, out):
        rk.dflash_prepare_delta_metadata(old[i], n[i], width, pos, seq)
        rk.paged_kv_read(pool, table, pos, seq, out[0], out[1])
    want = torch.zeros(steps, 2, B * width, Hkv, D, dtype=torch.float16, device=DEV)
    for i in range(steps):
        step(i, want[i])
        torch.cuda.synchronize()
    got = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(steps):
            step(i, got[i])
    for _ in range(40):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
