"""The operators on whole sequences: exports of include/ropekv_sequence.h, refusals on the host
(no GPU: only calls that must be rejected before any CUDA call, or that have nothing to do),
and the binding's refusals, each by its own message."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

import rope_kv_cache_gb300 as rk
from rope_kv_cache_gb300 import _serving, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, MIS, NUL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0)
FAR = ctypes.c_void_p(0x100000000)          # not overlapping what lies at A
OK, NULL, MISALIGNED, HEAD_DIM, HEADS, SHAPE, CAPACITY, STYLE = 0, -1, -2, -3, -5, -6, -8, -9


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_library()
    return rk.load_serving_library()


def test_header_and_exports(lib):
    text = open(os.path.join(ROOT, "include", "ropekv_sequence.h")).read()
    names = re.findall(r"ROPEKV_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)
    assert set(names) == {"prompt_attention_workspace_size", "prompt_attention", "tree_attention_workspace_size",
                          "tree_attention", "kv_accept_drafts", "paged_kv_accept_drafts", "paged_kv_copy_pages",
                          "paged_kv_fork_workspace_size", "paged_kv_fork", "paged_kv_free"}
    for n in names:
        assert hasattr(lib, n) and (n in rk.__all__), n


def pdims(**kw):
    d = dict(numTokens=100, numKVTokens=100, batch=4, numQHeads=32, numKVHeads=8, headDim=128)
    d.update(kw)
    return _serving.ropekv_prompt_dims(**d)


def prompt(lib, ptrs=None, qs=48 * 128, ks=48 * 128, vs=48 * 128, size=1 << 40, scale=0.1, **kw):
    #          q  k  v  q_starts kv_starts out lse workspace
    p = ptrs or [A, A, A, A, A, FAR, A, A]
    # (the inputs may lie over one another)
    return lib.prompt_attention(p[0], qs, p[1], ks, p[2], vs, *p[3:], size, ctypes.byref(pdims(**kw)), scale, NUL)


def test_prompt_refuses_bad_arguments(lib):
    assert prompt(lib, headDim=96) == HEAD_DIM
    assert prompt(lib, numQHeads=30) == HEADS and prompt(lib, numKVHeads=0) == HEADS
    for kw in (dict(numTokens=-1), dict(numKVTokens=-1), dict(batch=-1), dict(numTokens=(1 << 28) + 1),
               dict(numKVTokens=(1 << 28) + 1), dict(batch=(1 << 20) + 1), dict(numTokens=1 << 27), dict(qs=32 * 128 - 8),
               dict(ks=8 * 128 - 8), dict(vs=100), dict(qs=48 * 128 + 4), dict(ks=(1 << 36) + 8), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert prompt(lib, **kw) == SHAPE, kw
    for i in range(8):
        ptrs = [A, A, A, A, A, FAR, A, A]
        ptrs[i] = MIS
        assert prompt(lib, ptrs=ptrs) == MISALIGNED, i
        ptrs[i] = NUL
        if i not in (4, 6):                  # kv_starts and lse may be NULL
            assert prompt(lib, ptrs=ptrs) == NULL, i
    assert prompt(lib, ptrs=[A] * 8) == SHAPE                                   # out over q
    last = ctypes.c_void_p(0x10000 + 2 * (99 * 48 + 31) * 128)                  # over q's last head alone
    assert prompt(lib, ptrs=[A, FAR, FAR, A, A, last, A, A]) == SHAPE
    assert prompt(lib, ptrs=[FAR, A, FAR, A, A, A, A, A]) == SHAPE and prompt(lib, ptrs=[FAR, FAR, A, A, A, A, A, A]) == SHAPE
    need = lib.prompt_attention_workspace_size(ctypes.byref(pdims(numTokens=1000, numKVTokens=1000)))
    assert need > 0 and prompt(lib, numTokens=1000, numKVTokens=1000, size=need - 1) == CAPACITY
    assert prompt(lib, numTokens=0, ptrs=[NUL] * 8, size=0) == OK and prompt(lib, batch=0, ptrs=[NUL] * 8, size=0) == OK
    assert lib.prompt_attention(A, 0, A, 0, A, 0, A, A, FAR, A, A, 0, None, 0.1, NUL) == NULL
    size = lib.prompt_attention_workspace_size
    assert size(None) == NULL and size(ctypes.byref(pdims(headDim=32))) == HEAD_DIM and size(ctypes.byref(pdims(batch=0))) == 0


def tdims(**kw):
    d = dict(batch=4, seqLen=7, numQHeads=32, numKVHeads=8, headDim=128, kvCapacity=512)
    d.update(kw)
    return _serving.ropekv_tree_dims(**d)


def tree(lib, ptrs=None, size=1 << 40, scale=0.1, **kw):
    #          q  cache lens mask out lse workspace
    p = ptrs or [A, A, A, A, FAR, A, A]
    return lib.tree_attention(*p, size, ctypes.byref(tdims(**kw)), scale, NUL)


def test_tree_refuses_bad_arguments(lib):
    assert tree(lib, headDim=80) == HEAD_DIM and tree(lib, numQHeads=31) == HEADS and tree(lib, numQHeads=0) == HEADS
    for kw in (dict(batch=-1), dict(seqLen=-1), dict(seqLen=(1 << 15) + 1), dict(kvCapacity=-1), dict(kvCapacity=(1 << 28) + 1),
               dict(batch=1 << 20, seqLen=1 << 10), dict(kvCapacity=1 << 28, numKVHeads=8), dict(batch=1 << 20, seqLen=1, kvCapacity=1 << 20), dict(scale=float("nan"))):
        assert tree(lib, **kw) == SHAPE, kw
    for i in range(7):
        ptrs = [A, A, A, A, FAR, A, A]
        ptrs[i] = MIS
        assert tree(lib, ptrs=ptrs) == MISALIGNED, i
        ptrs[i] = NUL
        if i not in (3, 5):                  # tree_mask and lse may be NULL
            assert tree(lib, ptrs=ptrs) == NULL, i
    assert tree(lib, ptrs=[A] * 7) == SHAPE and tree(lib, ptrs=[A, FAR, A, A, A, A, A]) == SHAPE     # out over q
    assert tree(lib, ptrs=[FAR, A, A, A, A, A, A]) == SHAPE                     # out over the cache
    need = lib.tree_attention_workspace_size(ctypes.byref(tdims()))
    assert need > 0 and tree(lib, size=need - 1) == CAPACITY
    for kw in (dict(batch=0), dict(seqLen=0)):
        assert tree(lib, ptrs=[NUL] * 7, size=0, **kw) == OK
    assert lib.tree_attention_workspace_size(None) == NULL
    assert lib.tree_attention_workspace_size(ctypes.byref(tdims(seqLen=0))) == 0


def accept(lib, ptrs=None, B=4, S=7, n=5, Hkv=8, D=128, cap=100):
    return lib.kv_accept_drafts(*(ptrs or [A] * 5), B, S, n, Hkv, D, cap, NUL)


def paged_accept(lib, ptrs=None, B=4, S=7, n=5, Hkv=8, D=128, P=16, M=8, tpp=64, fmt=1):
    return lib.paged_kv_accept_drafts(*(ptrs or [A] * 7), B, S, n, Hkv, D, P, M, tpp, fmt, NUL)


def copy(lib, ptrs=None, n=5, Hkv=8, D=128, P=16, tpp=64, fmt=1):
    return lib.paged_kv_copy_pages(*(ptrs or [A] * 4), n, Hkv, D, P, tpp, fmt, NUL)


def fork(lib, ptrs=None, size=1 << 30, n=5, B=4, Hkv=8, D=128, P=16, M=8, tpp=64, fmt=1):
    return lib.paged_kv_fork(*(ptrs or [A] * 8), size, n, B, Hkv, D, P, M, tpp, fmt, NUL)


def free(lib, ptrs=None, n=5, B=4, P=16, M=8, tpp=64):
    return lib.paged_kv_free(*(ptrs or [A] * 5), n, B, P, M, tpp, NUL)


@pytest.mark.parametrize("call,pointers,optional", [(accept, 5, {4}), (paged_accept, 7, {6}), (copy, 4, set()),
                                                    (fork, 8, set()), (free, 5, {4})])
def test_rows_and_pages_refuse_bad_pointers(lib, call, pointers, optional):
    for i in range(pointers):
        ptrs = [A] * pointers
        ptrs[i] = MIS
        assert call(lib, ptrs=ptrs) == MISALIGNED, i
        ptrs[i] = NUL
        if i not in optional:
            assert call(lib, ptrs=ptrs) == NULL, i


def test_rows_and_pages_refuse_bad_sizes(lib):
    for call in (accept, paged_accept, copy, fork):
        assert call(lib, D=96) == HEAD_DIM and call(lib, Hkv=0) == HEADS and call(lib, n=-1) == SHAPE
    for call in (paged_accept, copy, fork):
        assert call(lib, fmt=3) == STYLE and call(lib, fmt=-1) == STYLE
        assert call(lib, P=-1) == SHAPE and call(lib, tpp=0) == SHAPE and call(lib, P=1 << 24) == SHAPE
    for call in (accept, paged_accept):
        assert call(lib, B=-1) == SHAPE and call(lib, S=-1) == SHAPE and call(lib, S=40000) == SHAPE and call(lib, n=40000) == SHAPE
        assert call(lib, B=0, ptrs=[NUL] * (5 if call is accept else 7)) == OK
    assert accept(lib, cap=-1) == SHAPE
    for call in (paged_accept, fork, free):
        assert call(lib, M=-1) == SHAPE and call(lib, M=1 << 25) == SHAPE and call(lib, B=-1) == SHAPE
    assert fork(lib, n=(1 << 20) + 1) == SHAPE and fork(lib, B=(1 << 18) + 1) == SHAPE
    assert fork(lib, size=lib.paged_kv_fork_workspace_size(5, 4) - 1) == CAPACITY
    assert copy(lib, n=0, ptrs=[NUL] * 4) == OK and fork(lib, n=0, ptrs=[NUL] * 8, size=0) == OK
    assert free(lib, n=-1) == SHAPE and free(lib, P=-1) == SHAPE and free(lib, tpp=0) == SHAPE
    assert free(lib, n=0, ptrs=[NUL] * 5) == OK and free(lib, B=0, ptrs=[NUL] * 5) == OK
    assert copy(lib, ptrs=[A, NUL, A, A], fmt=1) == NULL                       # scales of an 8-bit pool
    with pytest.raises(rk.RopeKVError):
        rk.paged_kv_fork_workspace_size(-1, 4)


def test_tree_masks():
    m = rk.tree_mask_from_parents([[-1, 0, 0, 1], [-1, -1, 1, 2]])
    assert m.dtype == torch.int32 and m[:, :, 0].tolist() == [[1, 3, 5, 11], [1, 2, 6, 14]]
    m = rk.tree_mask_from_parents([[-1] + list(range(39))])
    assert m.shape == (1, 40, 2) and m[0, 31].tolist() == [-1, 0] and m[0, 39].tolist() == [-1, 255]
    assert rk.tree_mask_from_parents([]).shape == (0, 0, 0)
    for bad in ([[0]], [[-1, 1]], [[-2]], [[-1], [-1, 0]]):
        with pytest.raises(ValueError):
            rk.tree_mask_from_parents(bad)


def h(*s):
    return torch.zeros(*s, dtype=torch.float16)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def refused(fn, good, kw, error, match):
    a = dict(good)
    a.update(kw)
    with pytest.raises(error, match=match):
        fn(**a)


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "expected a CUDA device"),
    (dict(kv_starts=i32(4), k=h(9, 2, 64), v=h(9, 2, 64)), ValueError, "expected a CUDA device"),
    (dict(q=h(5, 4)), ValueError, r"q \[T,Hq,D\]"),
    (dict(k=h(5, 2, 128)), ValueError, r"k, v \[Tk,Hkv,D\]"),
    (dict(v=h(6, 2, 64)), ValueError, r"k, v \[Tk,Hkv,D\]"),
    (dict(k=h(6, 2, 64), v=h(6, 2, 64)), ValueError, "kv_starts is needed"),
    (dict(q_starts=i32(0)), ValueError, "q_starts"),
    (dict(q_starts=i32(2, 2)), ValueError, "q_starts"),
    (dict(kv_starts=i32(3)), ValueError, "kv_starts"),
    (dict(out=h(5, 2, 64)), ValueError, "out .* lse"),
    (dict(lse=torch.zeros(5, 3)), ValueError, "out .* lse"),
    (dict(q=h(5, 4, 64).float()), TypeError, "q: dtype Float"),
    (dict(sm_scale="1"), TypeError, "real number"),
    (dict(q_starts=[0, 5]), TypeError, "q_starts must be a torch.Tensor"),
])
def test_prompt_binding(kw, error, match):
    refused(rk.prompt_attention, dict(q=h(5, 4, 64), k=h(5, 2, 64), v=h(5, 2, 64), q_starts=i32(4), out=h(5, 4, 64)), kw,
            error, match)


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "expected a CUDA device"),
    (dict(tree_mask=i32(3, 5, 1), lse=torch.zeros(3, 5, 4)), ValueError, "expected a CUDA device"),
    (dict(q=h(3, 4, 64)), ValueError, r"q \[B,S,Hq,D\]"),
    (dict(kv_cache=h(2, 2, 2, 9, 64)), ValueError, "kv_cache"),
    (dict(kv_cache=h(3, 1, 2, 9, 64)), ValueError, "kv_cache"),
    (dict(kv_cache=h(3, 2, 2, 9, 128)), ValueError, "kv_cache"),
    (dict(kv_cache_end_lens=i32(4)), ValueError, "kv_cache_end_lens"),
    (dict(out=h(3, 5, 2, 64)), ValueError, "out"),
    (dict(lse=torch.zeros(3, 5)), ValueError, "lse"),
    (dict(tree_mask=i32(3, 5, 2)), ValueError, "tree_mask"),
    (dict(tree_mask=i32(3, 5)), ValueError, "tree_mask"),
    (dict(kv_cache=torch.zeros(3, 2, 2, 9, 64)), ValueError, "CUDA"),
])
def test_tree_binding(kw, error, match):
    refused(rk.tree_attention, dict(q=h(3, 5, 4, 64), kv_cache=h(3, 2, 2, 9, 64), kv_cache_end_lens=i32(3), out=h(3, 5, 4, 64)),
            kw, error, match)


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "expected a CUDA device"),
    (dict(kv_cache=h(3, 2, 9, 64)), ValueError, r"kv_cache \[B,2,Hkv,cap,D\]"),
    (dict(accepted=i32(3)), ValueError, r"accepted \[B,A\]"),
    (dict(accepted=i32(2, 4)), ValueError, r"accepted \[B,A\]"),
    (dict(accepted_lens=i32(2)), ValueError, "accepted_lens"),
    (dict(kv_cache_end_lens=i32(2)), ValueError, "kv_cache_end_lens"),
    (dict(end_lens_out=i32(2)), ValueError, "end_lens_out"),
    (dict(seq_len=2 ** 40), ValueError, "seq_len is too large"),
])
def test_accept_binding(kw, error, match):
    refused(rk.kv_accept_drafts, dict(kv_cache=h(3, 2, 2, 9, 64), kv_cache_end_lens=i32(3), seq_len=5, accepted=i32(3, 4),
                                      accepted_lens=i32(3)), kw, error, match)


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "expected a CUDA device"),
    (dict(page_table=i32(3, 1, 2)), ValueError, "page_table"),
    (dict(kv_lens=i32(2)), ValueError, "kv_lens"),
    (dict(kv_lens_out=i32(2)), ValueError, "kv_lens_out"),
    (dict(accepted=i32(2, 4)), ValueError, "accepted"),
    (dict(kv_scales=torch.zeros(2, 4, 2, 16)), ValueError, "no kv_scales"),
    (dict(kv_cache=torch.zeros(2, 4, 16, 2, 64, dtype=torch.int8)), ValueError, "kv_scales .* expected"),
])
def test_paged_accept_binding(kw, error, match):
    refused(rk.paged_kv_accept_drafts, dict(kv_cache=h(2, 4, 16, 2, 64), page_table=i32(3, 2, 2), kv_lens=i32(3), seq_len=5,
                                            accepted=i32(3, 4), accepted_lens=i32(3)), kw, error, match)


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "expected a CUDA device"),
    (dict(kv_cache=h(4, 16, 2, 64)), ValueError, r"kv_cache \[2,P,TPP,Hkv,D\]"),
    (dict(dst_pages=i32(4)), ValueError, "src_pages, dst_pages"),
    (dict(src_pages=i32(3, 1)), ValueError, "src_pages, dst_pages"),
    (dict(kv_scales=torch.zeros(2, 4, 2, 16)), ValueError, "no kv_scales"),
    (dict(kv_cache=torch.zeros(2, 4, 16, 2, 64, dtype=torch.int8), kv_scales=torch.zeros(2, 4, 16, 2)), ValueError, "kv_scales .* expected"),
    (dict(kv_cache=torch.zeros(2, 4, 16, 2, 64)), TypeError, "kv_cache: dtype Float"),
])
def test_copy_binding(kw, error, match):
    refused(rk.paged_kv_copy_pages, dict(kv_cache=h(2, 4, 16, 2, 64), src_pages=i32(3), dst_pages=i32(3)), kw, error, match)


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "expected a CUDA device"),
    (dict(kv_lens=i32(2)), ValueError, "kv_lens"),
    (dict(ref_counts=i32(5)), ValueError, "ref_counts"),
    (dict(children=i32(3)), ValueError, "parents, children"),
    (dict(page_table=i32(3, 2)), ValueError, "page_table"),
])
def test_fork_binding(kw, error, match):
    refused(rk.paged_kv_fork, dict(kv_cache=h(2, 4, 16, 2, 64), page_table=i32(3, 2, 2), kv_lens=i32(3), ref_counts=i32(4),
                                   parents=i32(2), children=i32(2)), kw, error, match)


@pytest.mark.parametrize("kw,error,match", [
    (dict(), ValueError, "expected a CUDA device"),
    (dict(page_table=i32(3, 2)), ValueError, "page_table"),
    (dict(kv_lens=i32(2)), ValueError, "kv_lens"),
    (dict(sequences=i32(2, 1)), ValueError, "sequences, keep_lens"),
    (dict(keep_lens=i32(3), tokens_per_page=16), ValueError, "sequences, keep_lens"),
    (dict(keep_lens=i32(2)), ValueError, "tokens_per_page is needed"),
])
def test_free_binding(kw, error, match):
    refused(rk.paged_kv_free, dict(page_table=i32(3, 2, 2), kv_lens=i32(3), ref_counts=i32(4), sequences=i32(2)), kw, error, match)


@pytest.mark.gpu
@pytest.mark.parametrize("kw,error,match", [
    (dict(q_starts="cpu"), ValueError, "q_starts is on cpu"),
    (dict(q_starts=torch.int64), TypeError, "q_starts: dtype Long"),
    (dict(k=torch.bfloat16), TypeError, "k: dtype BFloat16"),
    (dict(lse=torch.float16), TypeError, "lse: dtype Half"),
    (dict(q="strided"), ValueError, "q: heads and dims must be dense"),
    (dict(out="strided"), ValueError, "out must be contiguous"),
    (dict(workspace=torch.float32), TypeError, "workspace: dtype Float"),
])
def test_prompt_on_the_device(kw, error, match):
    """One argument of another device, type or layout; nothing is launched."""
    a = dict(q=h(5, 4, 64), k=h(5, 2, 64), v=h(5, 2, 64), q_starts=torch.tensor([0, 2, 5], dtype=torch.int32), out=h(5, 4, 64),
             lse=torch.zeros(5, 4), workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    a = {n: t.to("cuda:0") for n, t in a.items()}
    rk.prompt_attention(**a)
    for n, how in kw.items():
        a[n] = a[n].cpu() if how == "cpu" else torch.stack([a[n], a[n]], -1)[..., 0] if how == "strided" else a[n].to(how)
    with pytest.raises(error, match=match):
        rk.prompt_attention(**a)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_outputs_over_inputs_are_refused():
    q = torch.zeros(5, 4, 64, dtype=torch.float16, device="cuda:0")
    starts = torch.tensor([0, 5], dtype=torch.int32, device="cuda:0")
    with pytest.raises(rk.RopeKVError):
        rk.prompt_attention(q, q, q, starts, q)
    cache, lens = torch.zeros(5, 2, 2, 9, 64, dtype=torch.float16, device="cuda:0"), torch.ones(5, dtype=torch.int32, device="cuda:0")
    with pytest.raises(rk.RopeKVError):
        rk.tree_attention(q[:, None], cache, lens, q[:, None])


def test_scales_that_fp32_does_not_hold_in_binary_digits_are_refused(lib):
    for scale in (3e38, -3e38):
        assert prompt(lib, scale=scale) == SHAPE and tree(lib, scale=scale) == SHAPE
    # one that it does hold: the next check is reached
    assert prompt(lib, scale=2e38, ptrs=[A] * 3 + [NUL] + [A] * 4) == NULL and tree(lib, scale=-2e38, ptrs=[NUL] * 7) == NULL
