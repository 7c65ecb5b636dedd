"""Cases of the operators on whole sequences: what each reads, writes and
computes, in a plain form (elementary torch operations) and through the
package's entry points.

  prompt   prompt_attention: causal attention of packed sequences of different
           lengths, of whole prompts or of chunks behind a context.
  tree     tree_attention: attention of the new tokens of every sequence (one, a
           chain or a tree of drafts) over the contiguous KV cache.
  accept   kv_accept_drafts, paged_kv_accept_drafts: the rows of accepted drafts
           moved to the front, in a contiguous and in a paged cache.
  copy     paged_kv_copy_pages: pages of a paged cache copied.
  beam     paged_kv_free and paged_kv_fork: sequences given up and made anew as
           copies of others that share their pages.

``own = False`` runs the plain forms, ``own = True`` the library's kernels.
"""
import math

import torch

own = False

DEV = "cuda:0"
E4M3_MAX, INT8_MAX = 448.0, 127.0


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # a few short prompts at once: latency
        _prompt("prompt_small", B=3, lo=1, hi=100, ctx=0, Hq=8, Hkv=2, D=64, packed=True),
        # a batch of prompts of very different lengths, half of them chunks behind a context
        _prompt("prompt_ragged", B=24, lo=1, hi=1200, ctx=1000, Hq=32, Hkv=8, D=128, packed=False),
        # one long prompt, Q, K and V views of one packed projection
        _prompt("prompt_long", B=1, lo=12001, hi=12001, ctx=0, Hq=32, Hkv=8, D=128, packed=True),
        # a tree of drafts of one sequence
        _tree("tree_small", B=1, S=26, lo=900, hi=900, Hq=8, Hkv=2, D=64, chain=False),
        # a decode step of a large batch: one new token per sequence
        _tree("decode_batch", B=128, S=1, lo=1, hi=4000, Hq=32, Hkv=8, D=128, chain=True),
        # verification of a tree of 61 drafts per sequence
        _tree("tree_draft", B=16, S=61, lo=500, hi=6000, Hq=32, Hkv=8, D=128, chain=False),
        # accepted drafts of a small batch
        _accept("accept_small", paged=False, B=4, S=16, A=5, Hkv=2, D=64, length=300, tpp=1, format="f16"),
        # accepted drafts of a large batch over an INT8 pool
        _accept("accept_paged_int8", paged=True, B=128, S=61, A=8, Hkv=8, D=128, length=900, tpp=64, format="int8"),
        # copy on write of a few pages
        _copy("copy_small_e4m3", N=6, Hkv=2, D=64, tpp=16, format="e4m3"),
        # many pages copied, as sequences move to another part of the pool
        _copy("copy_many", N=1200, Hkv=8, D=128, tpp=32, format="f16"),
        # a beam search step of one request
        _beam("beam_small", parents=4, children=4, lo=1, hi=200, Hkv=2, D=64, tpp=16, format="f16"),
        # several samples of each of many requests
        _beam("beam_batch", parents=64, children=192, lo=1, hi=2000, Hkv=8, D=128, tpp=64, format="f16"),
    ]


def _prompt(name, **c):
    return dict(name=name, op="prompt", **c)


def _tree(name, **c):
    return dict(name=name, op="tree", **c)


def _accept(name, **c):
    return dict(name=name, op="accept", **c)


def _copy(name, **c):
    return dict(name=name, op="copy", **c)


def _beam(name, **c):
    return dict(name=name, op="beam", **c)


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "accept", "copy", "beam"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8])
    tpp = rng.choice([16, 32, 64])
    fmt = rng.choice(["f16", "f16", "e4m3", "int8"])
    if op == "prompt":
        hi = _log_int(rng, 1, 12001)
        return _fit(dict(op=op, B=_log_int(rng, 1, 64), lo=rng.choice([1, hi]), hi=hi,
                         ctx=rng.choice([0, 0, _log_int(rng, 1, 8192)]), Hq=Hkv * G, Hkv=Hkv, D=D,
                         packed=rng.random() < 0.5), "hi", "B", "ctx")
    if op == "tree":
        S = rng.choice([1, 1, 1, 4, 7, 26, 61, 128])
        hi = _log_int(rng, 1, 16384)
        return _fit(dict(op=op, B=_log_int(rng, 1, 256), S=S, lo=rng.choice([0, hi // 2, hi]), hi=hi,
                         Hq=Hkv * G, Hkv=Hkv, D=D, chain=S == 1 or rng.random() < 0.3), "hi", "B")
    if op == "accept":
        paged = rng.random() < 0.5
        S = rng.choice([1, 8, 26, 61])
        return _fit(dict(op=op, paged=paged, B=_log_int(rng, 1, 256), S=S, A=min(S, rng.choice([2, 5, 8])),
                         Hkv=Hkv, D=D, length=_log_int(rng, 61, 1000), tpp=tpp if paged else 1,
                         format=fmt if paged else "f16"), "B", "length")
    if op == "copy":
        return _fit(dict(op=op, N=_log_int(rng, 1, 4000), Hkv=Hkv, D=D, tpp=tpp, format=fmt), "N")
    return _fit(dict(op=op, parents=_log_int(rng, 1, 64), children=_log_int(rng, 1, 256), lo=1,
                     hi=_log_int(rng, 1, 4000), Hkv=Hkv, D=D, tpp=tpp, format=fmt), "hi", "children", "parents")


def _cost(c):
    """What bounds a case's plain form and its memory: bytes of the caches and of the scores."""
    if c["op"] == "prompt":
        return 4.0 * c["B"] * c["Hq"] * c["hi"] * (c["hi"] + c["ctx"]) * max(1.0, c["D"] / 128)
    if c["op"] == "tree":
        return c["B"] * (c["hi"] + c["S"]) * (4.0 * c["Hkv"] * c["D"] + 2.0 * c["Hq"] * c["S"])
    e = _esize(c.get("format", "f16"))
    if c["op"] == "accept":
        return 2.0 * e * c["B"] * (c["length"] + c["S"] + c["tpp"]) * c["Hkv"] * c["D"]
    if c["op"] == "copy":
        return 2.0 * e * c["N"] * c["tpp"] * c["Hkv"] * c["D"]
    return 2.0 * e * (c["parents"] * (c["hi"] + c["tpp"]) + c["children"] * c["tpp"]) * c["Hkv"] * c["D"]


#: The largest listed cost of each kind, which drawn cases stay below.
_MOST = {"prompt": 4.0 * 32 * 12001 ** 2, "tree": 128 * 4001 * 4.0 * 1024 + 1, "accept": 290e6, "copy": 160e6,
         "beam": 610e6}


def _fit(case, *shrink):
    """Shrink the named sizes in turn until the case costs no more than the listed ones."""
    k = 0
    while _cost(case) > _MOST[case["op"]]:
        name = shrink[k % len(shrink)]
        case[name] = max(min(case[name], 61 if name == "length" else 1), case[name] * 2 // 3)
        if "lo" in case:
            case["lo"] = min(case["lo"], case["hi"])
        k += 1
    return case


def _esize(fmt):
    return 2 if fmt == "f16" else 1


def _spread(n, lo, hi, shift=0.0):
    """n whole numbers spread over [lo, hi], the first of them hi; the same for equal sizes."""
    return [hi if b == 0 else lo + int(((b * 0.6180339887 + shift) % 1.0) * (hi - lo + 1)) for b in range(n)]


def _prompt_lens(c):
    """Query tokens of each sequence, and the context tokens before them (every other sequence has some)."""
    q = _spread(c["B"], c["lo"], c["hi"])
    return q, [x if b % 2 else 0 for b, x in enumerate(_spread(c["B"], 0, c["ctx"], 0.3))]


def work(case):
    c = case
    if c["op"] == "prompt":
        nq, ctx = _prompt_lens(c)
        rows, keys = sum(nq), sum(nq) + sum(ctx)
        seen = sum(n * x + n * (n + 1) / 2.0 for n, x in zip(nq, ctx))
        return {"bytes": 4.0 * rows * c["Hq"] * c["D"] + 4.0 * keys * c["Hkv"] * c["D"] + 4.0 * rows * c["Hq"],
                "flops": 4.0 * seen * c["Hq"] * c["D"]}
    if c["op"] == "tree":
        ctx = sum(_spread(c["B"], c["lo"], c["hi"]))
        rows = c["B"] * c["S"]
        mask = 0 if c["chain"] else rows * 4 * ((c["S"] + 31) // 32)
        return {"bytes": rows * c["Hq"] * (4.0 * c["D"] + 4) + 4.0 * (ctx + rows) * c["Hkv"] * c["D"] + mask,
                "flops": 4.0 * c["D"] * c["Hq"] * (c["S"] * ctx + rows * (c["S"] + 1) / 2.0)}
    row = 2.0 * c["Hkv"] * (c["D"] * _esize(c["format"]) + (0 if c["format"] == "f16" else 4))
    if c["op"] == "accept":
        # about half of the most, in mean, and the first stays where it is
        return {"bytes": c["B"] * (2 * row * (c["A"] - 1) / 2.0 + 4 * c["A"] + 12), "flops": 0}
    if c["op"] == "copy":
        return {"bytes": c["N"] * (2 * row * c["tpp"] + 8), "flops": 0}
    # half a page per child is copied in mean, and its table row is read and written
    lens = sum(_spread(c["parents"], c["lo"], c["hi"])) / c["parents"]
    return {"bytes": c["children"] * (row * c["tpp"] + 16.0 * lens / c["tpp"] + 24), "flops": 0}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float16)


def _starts(lens):
    return torch.tensor([0] + lens, device=DEV).cumsum(0).int()


def _pool(pages, tpp, Hkv, D, fmt, g):
    """A filled pool [2, pages, tpp, Hkv, D] and, for 8-bit formats, its scales [2, pages, Hkv, tpp]."""
    x = _randn(g, 2, pages, tpp, Hkv, D)
    if fmt == "f16":
        return x, None
    big = E4M3_MAX if fmt == "e4m3" else INT8_MAX
    scale = x.abs().amax(-1).float() / big
    codes = x / scale[..., None].clamp(min=1e-20)
    codes = codes.to(torch.float8_e4m3fn) if fmt == "e4m3" else codes.round_().to(torch.int8)
    return codes, scale.transpose(2, 3).contiguous()


def _tree_mask(B, S, g):
    """Random trees over S nodes each, node 0 the root: [B, S, ceil(S/32)] int32, bit j of row i set
    where node j is i or an ancestor of i."""
    u = torch.rand(B, S, generator=g, device=DEV)
    sees = torch.eye(S, dtype=torch.bool, device=DEV).repeat(B, 1, 1)
    b = torch.arange(B, device=DEV)
    for i in range(1, S):
        parent = (u[:, i] * min(i, 12)).long() + max(0, i - 12)
        sees[:, i] |= sees[b, parent]
    words = torch.nn.functional.pad(sees, (0, -S % 32)).view(B, S, -1, 32).long()
    return (words << torch.arange(32, device=DEV)).sum(-1).int().contiguous()


def _accepted(c, g):
    """Accepted nodes of each sequence: a path of 1 to A nodes down a tree numbered level by level,
    so that a node that moves comes from behind all accepted ones."""
    B, S, A = c["B"], c["S"], c["A"]
    width = max(1, (S - 1) // max(1, A - 1))
    level = torch.arange(A, device=DEV)
    pick = (torch.rand(B, A, generator=g, device=DEV) * width).long()
    node = torch.where(level == 0, 0, 1 + (level - 1) * width + pick)
    node = torch.where(node < A, level, node)
    lens = torch.randint(1, A + 1, (B,), generator=g, device=DEV)
    return node.int().contiguous(), lens.int()


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "prompt":
        nq, ctx = _prompt_lens(c)
        nk = [n + x for n, x in zip(nq, ctx)]
        s["q_starts"], s["kv_starts"] = _starts(nq), _starts(nk)
        s["most"] = (max(nq), max(nk))
        Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
        if c["packed"] and c["ctx"] == 0:
            x = _randn(g, sum(nq), Hq + 2 * Hkv, D)
            s["q"], s["k"], s["v"] = x[:, :Hq].mul_(2), x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            s["q"] = _randn(g, sum(nq), Hq, D).mul_(2)
            s["k"], s["v"] = _randn(g, sum(nk), Hkv, D), _randn(g, sum(nk), Hkv, D)
        s["out"] = torch.zeros(sum(nq), Hq, D, dtype=torch.float16, device=DEV)
        s["lse"] = torch.zeros(sum(nq), Hq, device=DEV)
    elif c["op"] == "tree":
        B, S = c["B"], c["S"]
        ctx = _spread(B, c["lo"], c["hi"])
        s["end_lens"] = (torch.tensor(ctx, device=DEV) + S).int()
        s["cache"] = _randn(g, B, 2, c["Hkv"], c["hi"] + S, c["D"])
        s["q"] = _randn(g, B, S, c["Hq"], c["D"]).mul_(2)
        s["mask"] = None if c["chain"] else _tree_mask(B, S, g)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(B, S, c["Hq"], device=DEV)
    elif c["op"] == "accept":
        B, S, tpp = c["B"], c["S"], c["tpp"]
        s["accepted"], s["accepted_lens"] = _accepted(c, g)
        s["lens"] = S + torch.randint(0, c["length"] + 1, (B,), generator=g, device=DEV).int()
        s["lens_out"] = torch.zeros_like(s["lens"])
        if c["paged"]:
            cols = -(-(c["length"] + S) // tpp)
            order = torch.randperm(B * cols, generator=g, device=DEV).int().view(B, 1, cols)
            s["page_table"] = torch.cat([order, order + B * cols], 1).contiguous()
            s["cache"], s["scales"] = _pool(B * cols, tpp, c["Hkv"], c["D"], c["format"], g)
        else:
            s["cache"], s["scales"] = _randn(g, B, 2, c["Hkv"], c["length"] + S, c["D"]), None
    elif c["op"] == "copy":
        order = torch.randperm(2 * c["N"] + 3, generator=g, device=DEV).int()
        s["src"], s["dst"] = order[:c["N"]].contiguous(), order[c["N"]:2 * c["N"]].clone()
        s["cache"], s["scales"] = _pool(2 * c["N"] + 3, c["tpp"], c["Hkv"], c["D"], c["format"], g)
    else:
        P, N, tpp = c["parents"], c["children"], c["tpp"]
        lens = _spread(P, c["lo"], c["hi"])
        cols = -(-c["hi"] // tpp)
        need = torch.tensor([-(-n // tpp) for n in lens], device=DEV)
        used = sum(-(-n // tpp) for n in lens)
        pages = used + N + 5
        order = torch.randperm(pages, generator=g, device=DEV).int()
        mapped = torch.arange(cols, device=DEV)[None] < need[:, None]
        at = (mapped.flatten().cumsum(0) - 1).clamp(min=0).view(mapped.shape)
        s["page_table"] = torch.full((P + N, 2, cols), -1, dtype=torch.int32, device=DEV)
        s["page_table"][:P, 0] = torch.where(mapped, order[at], -1)
        s["page_table"][:P, 1] = torch.where(mapped, order[at] + pages, -1)
        s["ref_counts"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
        s["ref_counts"][order[:used].long()] = 1
        s["kv_lens"] = torch.tensor(lens + [0] * N, device=DEV).int()
        s["parents"] = torch.randint(0, P, (N,), generator=g, device=DEV).int()
        s["children"] = (P + torch.randperm(N, generator=g, device=DEV)).int()
        s["cache"], s["scales"] = _pool(pages, tpp, c["Hkv"], c["D"], c["format"], g)
    return s


# ------------------------------------------------------------ plain forms --

def _softmax_sum(score, sees, v):
    """One softmax over the last axis of score, masked by sees, and the sums of v: (out, lse)."""
    score = score.masked_fill(~sees, -math.inf)
    m = score.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    p = torch.exp(score - m)
    l = p.sum(-1, keepdim=True)
    out = torch.where(l > 0, (p @ v) / l, 0.0)
    return out, (m + torch.log(l))[..., 0]


def _plain_prompt(s):
    c = s["case"]
    B, Hq, Hkv, D, (nq, nk) = c["B"], c["Hq"], c["Hkv"], c["D"], s["most"]
    qs, ks = s["q_starts"].long(), s["kv_starts"].long()
    lq, lk = torch.diff(qs), torch.diff(ks)
    i, t = torch.arange(nq, device=DEV), torch.arange(nk, device=DEV)
    # every sequence padded to the longest
    rows = (qs[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    keys = (ks[:-1, None] + t).clamp(max=s["k"].shape[0] - 1)
    q = (s["q"][rows].float() / math.sqrt(D)).view(B, nq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    k = s["k"][keys].float().permute(0, 2, 3, 1)[:, :, None]
    v = s["v"][keys].float().permute(0, 2, 1, 3)[:, :, None]
    sees = t <= ((lk - lq)[:, None] + i)[..., None]
    out, lse = _softmax_sum(q @ k, (sees & (t < lk[:, None, None]))[:, None, None], v)
    live = i < lq[:, None]
    out = out.permute(0, 3, 1, 2, 4).reshape(B, nq, Hq, D)[live]
    s["out"].copy_(out)
    s["lse"].copy_(lse.permute(0, 3, 1, 2).reshape(B, nq, Hq)[live])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_tree(s):
    c = s["case"]
    B, S, Hq, Hkv, D = (c[n] for n in ("B", "S", "Hq", "Hkv", "D"))
    G, cap = Hq // Hkv, s["cache"].shape[3]
    # node j of a sequence is at slot end - S + j: what a row sees there says its mask
    j = torch.arange(cap, device=DEV)[None] - (s["end_lens"].long()[:, None] - S)         # [B, cap]
    if s["mask"] is None:
        sees = j[:, None] <= torch.arange(S, device=DEV)[None, :, None]
    else:
        at = j.clamp(0, S - 1)[:, None].expand(B, S, cap)
        bit = (torch.gather(s["mask"].long(), 2, at // 32) >> (at % 32)) & 1
        sees = (j[:, None] < 0) | ((j[:, None] < S) & (bit == 1))
    q = (s["q"].float() / math.sqrt(D)).view(B, S, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, S * G, D)
    kv = s["cache"].float()
    sees = sees.repeat_interleave(G, 1)[:, None]
    out, lse = _softmax_sum(q @ kv[:, 0].transpose(2, 3), sees, kv[:, 1])
    s["out"].copy_(out.view(B, Hkv, S, G, D).permute(0, 2, 1, 3, 4).reshape(B, S, Hq, D))
    s["lse"].copy_(lse.view(B, Hkv, S, G).permute(0, 2, 1, 3).reshape(B, S, Hq))
    return {"out": s["out"], "lse": s["lse"]}


def _bits(cache):
    return cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache


def _plain_accept(s):
    c = s["case"]
    B, S, A, tpp = (c[n] for n in ("B", "S", "A", "tpp"))
    b, j = torch.arange(B, device=DEV)[:, None], torch.arange(A, device=DEV)[None]
    base = s["lens"].long()[:, None] - S
    # entries past a sequence's count stay where they are
    src = base + torch.where(j < s["accepted_lens"][:, None], s["accepted"].long(), j)
    dst = base + j
    s["lens_out"].copy_(base[:, 0] + s["accepted_lens"])
    cache = _bits(s["cache"])
    if not c["paged"]:
        cache[b, :, :, dst] = cache[b, :, :, src]
        return {"cache": s["cache"], "lens": s["lens_out"]}
    table = s["page_table"][:, 0].long()
    from_, to = table[b, src // tpp], table[b, dst // tpp]
    cache[:, to, dst % tpp] = cache[:, from_, src % tpp]
    if s["scales"] is not None:
        s["scales"][:, to, :, dst % tpp] = s["scales"][:, from_, :, src % tpp]
    return {"cache": s["cache"], "scales": s["scales"], "lens": s["lens_out"]}


def _plain_copy(s):
    cache, src, dst = _bits(s["cache"]), s["src"].long(), s["dst"].long()
    cache[:, dst] = cache[:, src]
    if s["scales"] is not None:
        s["scales"][:, dst] = s["scales"][:, src]
    return {"cache": s["cache"], "scales": s["scales"]}


def _plain_beam(s):
    c = s["case"]
    tpp, table, refs, lens = c["tpp"], s["page_table"], s["ref_counts"], s["kv_lens"]
    pages, cols = refs.shape[0], table.shape[2]
    children, parents = s["children"].long(), s["parents"].long()
    # free: every mapped page of the children loses one reference
    old = table[children, 0]
    refs.index_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).flatten().int())
    table[children] = -1
    lens[children] = 0
    # fork: whole pages are shared, a partly filled last one is copied to the lowest free page
    n = lens[parents].long()
    whole, rest = n // tpp, n % tpp
    part = rest > 0
    free = torch.argsort((refs != 0).int(), stable=True)
    new = free[(part.cumsum(0) - 1).clamp(min=0)]
    col = torch.arange(cols, device=DEV)
    share = col < whole[:, None]
    row = torch.where(share, table[parents, 0], torch.where((col == whole[:, None]) & part[:, None], new[:, None].int(), -1))
    tail = table[parents, 0].gather(1, whole.clamp(max=cols - 1)[:, None])[:, 0].long()
    refs.index_add_(0, row.clamp(min=0).flatten().long(), (row >= 0).flatten().int())
    table[children, 0], table[children, 1] = row, torch.where(row >= 0, row + pages, -1)
    lens[children] = n.int()
    # a fork without a partly filled page copies nothing: its page onto itself
    src = torch.where(part, tail, 0)
    dst = torch.where(part, new, 0)
    cache, keep = _bits(s["cache"]), torch.arange(tpp, device=DEV) < rest[:, None]
    cache[:, dst] = torch.where(keep[None, :, :, None, None], cache[:, src], cache[:, dst])
    if s["scales"] is not None:
        s["scales"][:, dst] = torch.where(keep[None, :, None], s["scales"][:, src], s["scales"][:, dst])
    return {"cache": s["cache"], "scales": s["scales"], "table": table, "lens": lens, "refs": refs}


# -------------------------------------------------------------- own calls --

def _own(s):
    import rope_kv_cache_gb300 as rk
    c = s["case"]
    if c["op"] == "prompt":
        rk.prompt_attention(s["q"], s["k"], s["v"], s["q_starts"], s["out"], kv_starts=s["kv_starts"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "tree":
        rk.tree_attention(s["q"], s["cache"], s["end_lens"], s["out"], tree_mask=s["mask"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "accept":
        if not c["paged"]:
            rk.kv_accept_drafts(s["cache"], s["lens"], c["S"], s["accepted"], s["accepted_lens"], s["lens_out"])
            return {"cache": s["cache"], "lens": s["lens_out"]}
        rk.paged_kv_accept_drafts(s["cache"], s["page_table"], s["lens"], c["S"], s["accepted"],
                                  s["accepted_lens"], s["lens_out"], kv_scales=s["scales"])
        return {"cache": s["cache"], "scales": s["scales"], "lens": s["lens_out"]}
    if c["op"] == "copy":
        rk.paged_kv_copy_pages(s["cache"], s["src"], s["dst"], kv_scales=s["scales"])
        return {"cache": s["cache"], "scales": s["scales"]}
    rk.paged_kv_free(s["page_table"], s["kv_lens"], s["ref_counts"], s["children"])
    rk.paged_kv_fork(s["cache"], s["page_table"], s["kv_lens"], s["ref_counts"], s["parents"], s["children"],
                     kv_scales=s["scales"])
    return {"cache": s["cache"], "scales": s["scales"], "table": s["page_table"], "lens": s["kv_lens"],
            "refs": s["ref_counts"]}


def run(state):
    if own:
        return _own(state)
    return {"prompt": _plain_prompt, "tree": _plain_tree, "accept": _plain_accept, "copy": _plain_copy,
            "beam": _plain_beam}[state["case"]["op"]](state)


# -------------------------------------------------- the definition, 64 bits --

def _attend(q, k, v, first):
    """Rows of [n, H, D] against [t, H, D] keys, row i seeing the first `first` + i + 1; 64 bits."""
    score = torch.einsum("nhd,thd->hnt", q, k) / q.shape[-1] ** 0.5
    hidden = torch.arange(k.shape[0], device=DEV) > (first + torch.arange(q.shape[0], device=DEV))[:, None]
    score[:, hidden] = -math.inf
    return (torch.einsum("hnt,thd->nhd", torch.softmax(score, -1), v), torch.logsumexp(score, -1).t())


def exact(case, seed):
    c = case
    if c["op"] not in ("prompt", "tree"):
        return None  # copies: nothing is computed
    s = prepare(case, seed)
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    if c["op"] == "prompt":
        q0 = k0 = 0
        for n, x in zip(*_prompt_lens(c)):
            for h in range(c["Hkv"]):
                k, v = (s[w][k0:k0 + n + x, h].double()[:, None].expand(-1, G, -1) for w in ("k", "v"))
                for lo in range(0, n, 2048):
                    hi = min(n, lo + 2048)
                    o, l = _attend(s["q"][q0 + lo:q0 + hi, h * G:(h + 1) * G].double(), k[:x + hi], v[:x + hi], x + lo)
                    out[q0 + lo:q0 + hi, h * G:(h + 1) * G], lse[q0 + lo:q0 + hi, h * G:(h + 1) * G] = o, l
            q0, k0 = q0 + n, k0 + n + x
        return {"out": out, "lse": lse}
    for b, end in enumerate(s["end_lens"].tolist()):
        k, v = (s["cache"][b, p, :, :end].double().repeat_interleave(G, 0) for p in (0, 1))       # [Hq, end, D]
        score = torch.einsum("shd,htd->hst", s["q"][b].double(), k) / c["D"] ** 0.5
        for i in range(c["S"]):
            for w in range(0, c["S"], 32):
                word = (1 << max(0, min(32, i + 1 - w))) - 1 if s["mask"] is None else int(s["mask"][b, i, w // 32])
                hide = [t for t in range(min(32, c["S"] - w)) if not word >> t & 1]
                if hide:
                    score[:, i, end - c["S"] + w + torch.tensor(hide, device=DEV)] = -math.inf
        lse[b] = torch.logsumexp(score, -1).t()
        out[b] = torch.einsum("hst,htd->shd", torch.softmax(score, -1), v)
    return {"out": out, "lse": lse}
