"""Cases of the serving operators over the paged KV cache: what each reads,
writes and computes, in a plain form (elementary torch operations) and through
the package's entry points.

  mrope      rope_write_kv_mrope: rotary positions with several axes (time,
             height, width), rotated Q out, K and V into their cache slots.
  quant      rope_write_kv_slot_mapping_quant: rotated K and V quantised to 8
             bits with one scale per token and head as they are written.
  read       paged_kv_read: rows of a paged cache (FP16 or 8 bits) read back as
             dense FP16 rows.
  chunk      quant and read one after the other, as a chunked prefill does that
             keeps its context in 8 bits and attends to FP16 rows.
  attention  paged_attention_shared_prefix: attention of a batch whose
             sequences share a long prefix that is read and multiplied once
             for all of them.

``own = False`` runs the plain forms, ``own = True`` the library's kernels.
"""
import math

import torch

own = False

DEV = "cuda:0"
NEOX, GPTJ = 0, 1
E4M3_MAX, INT8_MAX = 448.0, 127.0


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step of 256 text sequences in a multimodal batch: all axes agree
        _mrope("mrope_decode", T=256, Hq=32, Hkv=8, D=128, r=128, style=NEOX, interleaved=False,
               text=1.0, strided=True, bs=64),
        # a prefill of video frames and text: patches carry (time, height, width)
        _mrope("mrope_video", T=8192, Hq=32, Hkv=8, D=128, r=128, style=NEOX, interleaved=True,
               text=0.25, strided=True, bs=64),
        # one decode step into an E4M3 cache
        _quant("quant_decode_e4m3", T=256, Hq=32, Hkv=8, D=128, r=128, style=NEOX, bs=64),
        # a prefill into an E4M3 cache, Q, K and V views of one packed projection
        _quant("quant_prefill_e4m3", T=8192, Hq=32, Hkv=8, D=128, r=128, style=NEOX, bs=64),
        # a chunk of a long prompt: written to an INT8 cache, the context read back in FP16
        _chunk("chunk_int8", T=2050, context=6100, Hq=32, Hkv=8, D=128, r=64, style=GPTJ, bs=32),
        # reading one short sequence's pages back, a few rows of padding
        _read("read_small_int8", N=77, B=3, Hkv=2, D=64, tpp=16, format="int8"),
        # reading a batch's context back
        _read("read_context_e4m3", N=65521, B=128, Hkv=8, D=128, tpp=64, format="e4m3"),
        # a few sequences behind a short system prompt: latency
        _attn("attention_small", B=3, S=1, Hq=8, Hkv=2, D=64, tpp=16, prefix=500, lo=1, hi=100,
              format="f16"),
        # a decode step of a large batch behind a long shared prompt
        _attn("attention_batch", B=256, S=1, Hq=32, Hkv=8, D=128, tpp=64, prefix=8192, lo=1, hi=512,
              format="f16"),
        # the same kind of batch with an E4M3 cache and long answers
        _attn("attention_e4m3", B=128, S=1, Hq=32, Hkv=8, D=128, tpp=64, prefix=4097, lo=1, hi=2048,
              format="e4m3"),
        # verification of seven drafted tokens per sequence over an INT8 cache
        _attn("attention_draft_int8", B=61, S=7, Hq=32, Hkv=8, D=128, tpp=32, prefix=2000, lo=7,
              hi=700, format="int8"),
        # wide heads, one KV head per group of eight
        _attn("attention_wide", B=40, S=1, Hq=16, Hkv=2, D=256, tpp=64, prefix=3001, lo=1, hi=900,
              format="f16"),
    ]


def _mrope(name, **c):
    return dict(name=name, op="mrope", **c)


def _quant(name, **c):
    return dict(name=name, op="quant", format="e4m3", **c)


def _chunk(name, **c):
    return dict(name=name, op="chunk", format="int8", **c)


def _read(name, **c):
    return dict(name=name, op="read", **c)


def _attn(name, **c):
    return dict(name=name, op="attention", **c)


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["mrope", "quant", "chunk", "read", "attention", "attention", "attention"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8])
    r = rng.choice([x for x in (32, 64, 128, 256) if x <= D])
    style = rng.choice([NEOX, GPTJ])
    bs = rng.choice([16, 32, 64])
    heads = dict(Hq=Hkv * G, Hkv=Hkv, D=D)
    if op == "mrope":
        return _fit(dict(op=op, T=_log_int(rng, 1, 8192), r=r, style=style, bs=bs,
                         interleaved=rng.random() < 0.5, text=rng.choice([0.0, 0.25, 1.0]),
                         strided=rng.random() < 0.5, **heads), "T")
    if op == "quant":
        return _fit(dict(op=op, format="e4m3", T=_log_int(rng, 1, 8192), r=r, style=style, bs=bs,
                         **heads), "T")
    if op == "chunk":
        return _fit(dict(op=op, format="int8", T=_log_int(rng, 1, 4096),
                         context=_log_int(rng, 1, 16384), r=r, style=style, bs=bs, **heads),
                    "context", "T")
    if op == "read":
        B = _log_int(rng, 1, 128)
        return _fit(dict(op=op, N=_log_int(rng, B, 65536), B=B, Hkv=Hkv, D=D,
                         tpp=bs, format=rng.choice(["f16", "e4m3", "int8"])), "N")
    S = rng.choice([1, 1, 1, 1, 2, 4, 7, 16])
    return _fit(dict(op=op, B=_log_int(rng, 1, 256), S=S, tpp=bs,
                     prefix=_log_int(rng, 16, 16384), lo=S, hi=S + _log_int(rng, 1, 2048),
                     format=rng.choice(["f16", "f16", "e4m3", "int8"]), **heads),
                "hi", "prefix", "B")


#: What the largest listed case of each kind costs, which drawn cases stay below.
_MOST = {"mrope": 206e6, "quant": 190e6, "chunk": 120e6, "read": 390e6, "attention": 270e6}


def _fit(case, *shrink):
    """Halve the named sizes in turn until the case costs no more than the listed ones."""
    def cost(c):
        w = work(c)
        if c["op"] == "attention":
            # the padded suffix counts in full: the plain form lays it out
            w["bytes"] += c["B"] * c["hi"] * c["Hkv"] * c["D"] * 2
        return max(w["bytes"], w["flops"] / 130)
    k = 0
    while cost(case) > _MOST[case["op"]]:
        name = shrink[k % len(shrink)]
        floor = case["lo"] if name == "hi" else case["B"] if name == "N" else 1
        case[name] = max(floor, case[name] * 2 // 3)
        k += 1
    return case


def _esize(fmt):
    return 2 if fmt == "f16" else 1


def work(case):
    c = case
    if c["op"] == "attention":
        suffix = c["B"] * (c["lo"] + c["hi"]) / 2.0
        rows = c["B"] * c["S"]
        row_bytes = 2 * c["Hkv"] * (c["D"] * _esize(c["format"]) + (0 if c["format"] == "f16" else 4))
        qo = rows * c["Hq"] * (4 * c["D"] + 4)
        return {"bytes": qo + (c["prefix"] + suffix) * row_bytes,
                "flops": 4.0 * c["D"] * c["Hq"] * c["S"] * (c["B"] * c["prefix"] + suffix)}
    if c["op"] == "read":
        row = c["Hkv"] * c["D"]
        per = 2 * (row * (_esize(c["format"]) + 2) + (0 if c["format"] == "f16" else 4 * c["Hkv"])) + 8
        return {"bytes": c["N"] * per, "flops": 2.0 * c["N"] * row}
    q, kv = c["Hq"] * c["D"], c["Hkv"] * c["D"]
    if c["op"] == "mrope":
        # the rows of cos and sin: one of r floats in all, whichever axes they come from
        per = 2 * (q + 2 * kv) + 4 * c["r"] + 2 * (q + 2 * kv) + 8 * 4
        return {"bytes": c["T"] * per, "flops": 6.0 * c["T"] * (c["Hq"] + c["Hkv"]) * c["r"] / 2}
    per = 2 * (q + 2 * kv) + 4 * c["r"] + 2 * q + 2 * kv + 8 * c["Hkv"] + 8 * 2
    flops = c["T"] * (3.0 * (c["Hq"] + c["Hkv"]) * c["r"] + 4.0 * kv)
    if c["op"] == "quant":
        return {"bytes": c["T"] * per, "flops": flops}
    # chunk: the context's rows, the chunk's own among them, come back as FP16
    rows = c["context"] + c["T"]
    return {"bytes": c["T"] * per + rows * (2 * (3 * kv + 4 * c["Hkv"]) + 8),
            "flops": flops + 2.0 * rows * kv}


# ----------------------------------------------------------------- inputs --

def _table(rows, r, theta=5e5):
    """[rows, r] FP32: cos then sin of pos * theta^(-2i/r)."""
    ang = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] \
        * theta ** (-2.0 * torch.arange(r // 2, device=DEV, dtype=torch.float64) / r)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _qkv(c, g, strided=True):
    """Q, K, V of T tokens: views of one packed projection, or tensors of their own."""
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV).half()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    return (q, k, v) if strided else (q.contiguous(), k.contiguous(), v.contiguous())


def _sections(r, axes=3):
    """r/2 frequencies over time, height and width: about a quarter for time."""
    rest = (r // 2 * 3 // 8)
    return [r // 2 - 2 * rest, rest, rest] if axes == 3 else [r // 2]


def _freq_axis(c):
    """Axis of each frequency, chunked or interleaved (host tensor)."""
    n, sec = c["r"] // 2, _sections(c["r"])
    if not c["interleaved"]:
        return torch.tensor([a for a in range(3) for _ in range(sec[a])], dtype=torch.int32)
    i = torch.arange(n)
    axis = torch.where((i % 3 == 1) & (i < 3 * sec[1]), 1, 0)
    return torch.where((i % 3 == 2) & (i < 3 * sec[2]), 2, axis).to(torch.int32)


def _mrope_positions(c, g):
    """Text runs (equal axes) and 14 x 14 patch frames (time, row, column), as a
    prompt of alternating runs has them; [3, T] int64."""
    T = c["T"]
    t = torch.arange(T, device=DEV)
    frame, cell = t // 196, t % 196
    vis = torch.stack([frame, cell // 14, cell % 14]) + 64
    txt = torch.randint(0, 16384, (1, T), generator=g, device=DEV).expand(3, T) if T <= 256 else \
        (t + 64).expand(3, T)
    is_text = torch.rand(T // 196 + 1, generator=g, device=DEV)[frame] < c["text"]
    return torch.where(is_text, txt, vis).contiguous()


def _slots(T, bs, g):
    """T distinct slots: whole blocks in random order, filled in order."""
    blocks = -(-T // bs) + 8
    order = torch.randperm(blocks, generator=g, device=DEV)
    t = torch.arange(T, device=DEV)
    return blocks, order[t // bs] * bs + t % bs


def _page_ids(n, g):
    """K page ids 0..n-1 and V page ids n..2n-1, each in random order, int32."""
    return (torch.randperm(n, generator=g, device=DEV).int(),
            torch.randperm(n, generator=g, device=DEV).int() + n)


def _tables(n_pages_of, cols, g, spare=3):
    """Page table [B, 2, cols] over a shuffled pool; sequence b maps its first
    n_pages_of[b] columns. Returns (table, number of pages)."""
    mapped = torch.arange(cols, device=DEV)[None] < n_pages_of[:, None]
    total = int(mapped.sum()) + spare
    kid, vid = _page_ids(total, g)
    at = (mapped.flatten().cumsum(0) - 1).clamp(min=0).view(mapped.shape)
    none = torch.full((), -1, dtype=torch.int32, device=DEV)
    return torch.stack([torch.where(mapped, kid[at], none), torch.where(mapped, vid[at], none)],
                       1).contiguous(), total


def _pool(pages, tpp, Hkv, D, fmt, g):
    """A filled pool [2, pages, tpp, Hkv, D] and, for 8-bit formats, its scales
    [2, pages, Hkv, tpp]."""
    x = torch.randn(2, pages, tpp, Hkv, D, generator=g, device=DEV, dtype=torch.float16)
    if fmt == "f16":
        return x, None
    big = E4M3_MAX if fmt == "e4m3" else INT8_MAX
    scale = x.abs().amax(-1).float() / big
    codes = x / scale[..., None].clamp(min=1e-20)
    del x
    codes = codes.to(torch.float8_e4m3fn) if fmt == "e4m3" else codes.round_().to(torch.int8)
    return codes, scale.transpose(2, 3).contiguous()


def _empty_cache(c, blocks, fmt):
    shape = (blocks, c["bs"], c["Hkv"], c["D"])
    dt = {"f16": torch.float16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[fmt]
    return torch.zeros(shape, dtype=torch.uint8 if fmt == "e4m3" else dt, device=DEV).view(dt)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "mrope":
        s["q"], s["k"], s["v"] = _qkv(c, g, c["strided"])
        s["cos_sin"], s["positions"] = _table(16384, c["r"]), _mrope_positions(c, g)
        s["freq_axis"] = _freq_axis(c)
        blocks, s["slots"] = _slots(c["T"], c["bs"], g)
        s["key_cache"], s["value_cache"] = _empty_cache(c, blocks, "f16"), _empty_cache(c, blocks, "f16")
        s["q_out"] = torch.zeros(c["T"], c["Hq"], c["D"], dtype=torch.float16, device=DEV)
    elif c["op"] in ("quant", "chunk"):
        T, ctx = c["T"], c.get("context", 0)
        s["q"], s["k"], s["v"] = _qkv(c, g)
        s["cos_sin"] = _table(max(16384, ctx + T), c["r"])
        s["positions"] = torch.randint(0, 16384, (T,), generator=g, device=DEV) if ctx == 0 and T <= 256 \
            else ctx + torch.arange(T, device=DEV)
        s["q_out"] = torch.zeros(T, c["Hq"], c["D"], dtype=torch.float16, device=DEV)
        if c["op"] == "quant":
            pages, s["slots"] = _slots(T, c["bs"], g)
            shape = (2, pages, c["Hkv"], c["bs"])
            s["scales"] = torch.zeros(shape, device=DEV)
            s["cache"] = torch.stack([_empty_cache(c, pages, c["format"]).view(torch.uint8)] * 2) \
                .view(torch.float8_e4m3fn)
        else:
            # one sequence: its context is in the cache, the chunk follows it
            cols = -(-(ctx + T) // c["bs"])
            n = torch.tensor([cols], device=DEV)
            s["page_table"], pages = _tables(n, cols, g)
            # the slot mapping names one block for K and V alike
            s["page_table"][:, 1] = s["page_table"][:, 0] + pages
            s["cache"], s["scales"] = _pool(pages, c["bs"], c["Hkv"], c["D"], "int8", g)
            pos = ctx + torch.arange(T, device=DEV)
            s["slots"] = s["page_table"][0, 0][pos // c["bs"]].long() * c["bs"] + pos % c["bs"]
            s["row_positions"] = torch.arange(ctx + T, device=DEV, dtype=torch.int32)
            s["row_sequences"] = torch.zeros(ctx + T, device=DEV, dtype=torch.int32)
            s["k_out"] = torch.zeros(ctx + T, c["Hkv"], c["D"], dtype=torch.float16, device=DEV)
            s["v_out"] = torch.zeros_like(s["k_out"])
    elif c["op"] == "read":
        N, B, tpp = c["N"], c["B"], c["tpp"]
        # N rows over B sequences of random lengths, in order; about 5 % of the rows are padding
        cut = torch.randperm(max(N - 1, 1), generator=g, device=DEV)[:B - 1].sort().values + 1
        lens = torch.diff(cut, prepend=cut.new_zeros(1), append=cut.new_tensor([N])) if N > 1 else cut.new_ones(1)
        seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), lens)
        pos = torch.arange(N, device=DEV) - (lens.cumsum(0) - lens)[seq]
        cols = int(-(-lens.max() // tpp))
        s["page_table"], pages = _tables(-(-lens // tpp), cols, g)
        pad = torch.rand(N, generator=g, device=DEV) < 0.05
        s["row_positions"] = torch.where(pad, -1, pos).int()
        s["row_sequences"] = torch.where(pad, -1, seq).int()
        s["cache"], s["scales"] = _pool(pages, tpp, c["Hkv"], c["D"], c["format"], g)
        s["k_out"] = torch.zeros(N, c["Hkv"], c["D"], dtype=torch.float16, device=DEV)
        s["v_out"] = torch.zeros_like(s["k_out"])
    else:
        B, S, P, tpp = c["B"], c["S"], c["prefix"], c["tpp"]
        s["q"] = (torch.randn(B, S, c["Hq"], c["D"], generator=g, device=DEV) * 2).half()
        own_len = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g, device=DEV)
        own_len[0] = c["hi"]
        s["kv_lens"] = (P + own_len).int()
        shared, first = -(-P // tpp), P // tpp
        cols = -(-(P + c["hi"]) // tpp)
        # one pool: the prefix's pages, then each sequence's own behind its first full page
        n_own = -(-(P + own_len) // tpp) - first
        own_table, pages = _tables(torch.cat([n_own.new_tensor([shared]), n_own]),
                                   max(shared, cols - first), g)
        s["prefix_table"] = own_table[0, :, :shared].contiguous()
        table = torch.full((B, 2, cols), -1, dtype=torch.int32, device=DEV)
        table[:, :, :first] = s["prefix_table"][:, :first]
        table[:, :, first:] = own_table[1:, :, :cols - first]
        s["page_table"] = table
        s["cache"], s["scales"] = _pool(pages, tpp, c["Hkv"], c["D"], c["format"], g)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(B, S, c["Hq"], device=DEV)
    return s


# ------------------------------------------------------------ plain forms --

def _rotate(x, cos, sin, r, style):
    """x' = x * cos + rotate(x) * sin on the first r dims of [T, H, D]; cos, sin [T, r/2]."""
    cos, sin = cos[:, None], sin[:, None]
    head, tail = x[..., :r], x[..., r:]
    if style == NEOX:
        a, b = head[..., :r // 2], head[..., r // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, tail], -1)


def _plain_mrope(s):
    c, r = s["case"], s["case"]["r"]
    axis = s["freq_axis"].to(DEV, non_blocking=True).long()
    rows = s["positions"][axis].t()                      # [T, r/2]: the row of each frequency
    f = torch.arange(r // 2, device=DEV)
    cos, sin = s["cos_sin"][rows, f], s["cos_sin"][rows, f + r // 2]
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, r, c["style"]))
    k = _rotate(s["k"].float(), cos, sin, r, c["style"]).half()
    s["key_cache"].view(-1, c["Hkv"], c["D"])[s["slots"]] = k
    s["value_cache"].view(-1, c["Hkv"], c["D"])[s["slots"]] = s["v"]
    return {"q": s["q_out"], "k": s["key_cache"], "v": s["value_cache"]}


def _quantise(x, fmt):
    """Codes of [T, H, D] and one scale per token and head (64 bits until the codes:
    a value next to a border between two codes decides by its last bits)."""
    big = E4M3_MAX if fmt == "e4m3" else INT8_MAX
    amax = x.abs().amax(-1)
    codes = x * torch.where(amax > 0, big / amax, 0.0)[..., None]
    codes = codes.float().to(torch.float8_e4m3fn) if fmt == "e4m3" else codes.round().to(torch.int8)
    return codes, (amax / big).float()


def _plain_quant(s):
    c, r = s["case"], s["case"]["r"]
    row = s["cos_sin"][s["positions"]].double()
    cos, sin = row[:, :r // 2], row[:, r // 2:]
    s["q_out"].copy_(_rotate(s["q"].double(), cos, sin, r, c["style"]))
    slots = s["slots"]
    block, at = slots // c["bs"], slots % c["bs"]
    k, ks = _quantise(_rotate(s["k"].double(), cos, sin, r, c["style"]), c["format"])
    v, vs = _quantise(s["v"].double(), c["format"])
    flat = s["cache"].view(torch.uint8).view(2, -1, c["Hkv"], c["D"])
    flat[0, slots], flat[1, slots] = k.view(torch.uint8), v.view(torch.uint8)
    s["scales"][0, block, :, at], s["scales"][1, block, :, at] = ks, vs
    return {"q": s["q_out"], "kv": s["cache"], "scales": s["scales"]}


def _pages(cache, scales, ids):
    """Rows of the pages `ids` (flat ids of the [2, pages] pool) in 32 bits, [..., tpp, Hkv, D]."""
    x = cache.flatten(0, 1)[ids].float() if cache.dtype != torch.float8_e4m3fn else \
        cache.view(torch.uint8).flatten(0, 1)[ids].view(torch.float8_e4m3fn).float()
    return x if scales is None else x * scales.flatten(0, 1)[ids].transpose(-1, -2)[..., None]


def _plain_rows(s, plane, out):
    pos, seq = s["row_positions"].long(), s["row_sequences"].long()
    tpp = s["cache"].shape[2]
    lp, at = pos.clamp(min=0) // tpp, pos.clamp(min=0) % tpp
    ids = s["page_table"][seq.clamp(min=0), plane, lp].long()
    x = s["cache"].view(torch.uint8).flatten(0, 1)[ids, at].view(s["cache"].dtype).float()
    if s["scales"] is not None:
        x = x * s["scales"].flatten(0, 1)[ids, :, at][..., None]
    out.copy_(torch.where(((pos >= 0) & (seq >= 0))[:, None, None], x.half(), out))


def _plain_read(s):
    _plain_rows(s, 0, s["k_out"])
    _plain_rows(s, 1, s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_attention(s):
    c = s["case"]
    B, S, Hq, Hkv, D, P, tpp = (c[n] for n in ("B", "S", "Hq", "Hkv", "D", "prefix", "tpp"))
    G, first, cols = Hq // Hkv, P // tpp, s["page_table"].shape[2]
    q = s["q"].float().view(B, S, Hkv, G, D) / math.sqrt(D)
    last = s["kv_lens"].long()[:, None] - S + torch.arange(S, device=DEV)          # [B, S]
    # the shared prefix, once for all rows of the batch
    kv = _pages(s["cache"], s["scales"], s["prefix_table"].long()).flatten(1, 2)[:, :P]
    qp = q.permute(2, 0, 1, 3, 4).reshape(Hkv, B * S * G, D)
    sp = (qp @ kv[0].permute(1, 2, 0)).view(Hkv, B, S, G, P)
    sp = sp.masked_fill(torch.arange(P, device=DEV) > last[None, :, :, None, None], -math.inf)
    # each sequence's own tokens, padded to the longest
    ids = s["page_table"][:, :, first:].long()
    own_kv = _pages(s["cache"], s["scales"], ids.clamp(min=0)).flatten(2, 3)         # [B, 2, L, Hkv, D]
    t = first * tpp + torch.arange((cols - first) * tpp, device=DEV)
    hide = (t[None, None] > last[..., None]) | (t < P)                              # [B, S, L]
    qs = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, S * G, D)
    so = (qs @ own_kv[:, 0].permute(0, 2, 3, 1)).view(B, Hkv, S, G, -1)
    so = so.masked_fill(hide[:, None, :, None], -math.inf)
    # one softmax over both parts
    m = torch.maximum(sp.amax(-1).permute(1, 0, 2, 3), so.amax(-1))                  # [B, Hkv, S, G]
    m0 = torch.where(torch.isfinite(m), m, 0.0)
    pp = torch.exp(sp - m0.permute(1, 0, 2, 3)[..., None])
    po = torch.exp(so - m0[..., None])
    l = pp.sum(-1).permute(1, 0, 2, 3) + po.sum(-1)
    o = (pp.view(Hkv, B * S * G, P) @ kv[1].permute(1, 0, 2)).view(Hkv, B, S, G, D).permute(1, 0, 2, 3, 4)
    vals = torch.where(hide.all(1)[:, :, None, None], 0.0, own_kv[:, 1])
    o = o + (po.view(B, Hkv, S * G, -1) @ vals.permute(0, 2, 1, 3)).view(B, Hkv, S, G, D)
    o = torch.where(l[..., None] > 0, o / l[..., None], 0.0)
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(B, S, Hq, D))
    s["lse"].copy_((m0 + torch.log(l)).permute(0, 2, 1, 3).reshape(B, S, Hq))
    return {"out": s["out"], "lse": s["lse"]}


# -------------------------------------------------------------- own calls --

def _own(s):
    import rope_kv_cache_gb300 as rk
    c = s["case"]
    if c["op"] == "mrope":
        rk.rope_write_kv_mrope(s["cos_sin"], s["positions"], s["freq_axis"], s["q"], s["k"], s["v"],
                               s["slots"], s["key_cache"], s["value_cache"], s["q_out"],
                               style=c["style"])
        return {"q": s["q_out"], "k": s["key_cache"], "v": s["value_cache"]}
    if c["op"] in ("quant", "chunk"):
        cache, scales = s["cache"], s["scales"]
        rk.rope_write_kv_slot_mapping_quant(s["cos_sin"], s["positions"], s["q"], s["k"], s["v"],
                                            s["slots"], cache[0], cache[1], scales[0], scales[1],
                                            s["q_out"], style=c["style"])
        if c["op"] == "quant":
            return {"q": s["q_out"], "kv": cache, "scales": scales}
    if c["op"] in ("read", "chunk"):
        rk.paged_kv_read(s["cache"], s["page_table"], s["row_positions"], s["row_sequences"],
                         s["k_out"], s["v_out"], kv_scales=s["scales"])
        if c["op"] == "chunk":
            return {"q": s["q_out"], "scales": s["scales"], "k": s["k_out"], "v": s["v_out"]}
        return {"k": s["k_out"], "v": s["v_out"]}
    rk.paged_attention_shared_prefix(s["q"], s["cache"], s["prefix_table"], c["prefix"],
                                     s["page_table"], s["kv_lens"], s["out"], lse=s["lse"],
                                     kv_scales=s["scales"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "mrope":
        return _plain_mrope(state)
    if op == "quant":
        return _plain_quant(state)
    if op == "read":
        return _plain_read(state)
    if op == "chunk":
        w = _plain_quant(state)
        return {"q": w["q"], "scales": w["scales"], **_plain_read(state)}
    return _plain_attention(state)


# -------------------------------------------------- the definition, 64 bits --

def _turn(x, z, r, style):
    """Rotation of [T, H, D] as a product of complex numbers: pair i by z[:, i]."""
    x = x.to(torch.float64).clone()
    i = torch.arange(r // 2, device=x.device)
    re, im = (i, i + r // 2) if style == NEOX else (2 * i, 2 * i + 1)
    w = torch.complex(x[..., re], x[..., im]) * z[:, None]
    x[..., re], x[..., im] = w.real, w.imag
    return x


def _exact_write(s):
    c, h = s["case"], s["case"]["r"] // 2
    z = torch.complex(s["cos_sin"][:, :h].double(), s["cos_sin"][:, h:].double())
    if c["op"] == "mrope":
        pos = torch.empty(c["T"], h, dtype=torch.long, device=DEV)
        for f, a in enumerate(s["freq_axis"].tolist()):
            pos[:, f] = s["positions"][a]
        z = torch.gather(z, 0, pos)
    else:
        z = z[s["positions"]]
    return (_turn(s["q"], z, c["r"], c["style"]), _turn(s["k"], z, c["r"], c["style"]),
            s["v"].double())


def _exact_attention(s):
    c = s["case"]
    B, S, Hq, Hkv, P, tpp = (c[n] for n in ("B", "S", "Hq", "Hkv", "prefix", "tpp"))

    def rows(table, plane, lo, hi):
        p = torch.arange(lo, hi, device=DEV)
        page = table[plane][p // tpp].long() - plane * s["cache"].shape[1]
        x = s["cache"][plane].view(torch.uint8)[page, p % tpp].view(s["cache"].dtype).double()
        return x if s["scales"] is None else x * s["scales"][plane][page, :, p % tpp].double()[..., None]
    pk, pv = (rows(s["prefix_table"], plane, 0, P) for plane in (0, 1))
    out = torch.zeros(B, S, Hq, c["D"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(B, S, Hq, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["kv_lens"].tolist()):
        k = torch.cat([pk, rows(s["page_table"][b], 0, P, n)]).repeat_interleave(Hq // Hkv, 1)
        v = torch.cat([pv, rows(s["page_table"][b], 1, P, n)]).repeat_interleave(Hq // Hkv, 1)
        for j in range(S):
            seen = n - S + j + 1
            score = torch.einsum("hd,thd->ht", s["q"][b, j].double(), k[:seen]) / c["D"] ** 0.5
            lse[b, j] = torch.logsumexp(score, 1)
            out[b, j] = torch.einsum("ht,thd->hd", torch.softmax(score, 1), v[:seen])
    return {"out": out, "lse": lse}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "attention":
        # about two fused products of 64 bits per value read: a few seconds at most
        return _exact_attention(s)
    if c["op"] == "read":
        k, v = torch.zeros_like(s["k_out"], dtype=torch.float64), torch.zeros_like(s["v_out"], dtype=torch.float64)
        n = torch.nonzero(s["row_positions"] >= 0)[:, 0]
        p, b = s["row_positions"][n].long(), s["row_sequences"][n].long()
        for plane, out in ((0, k), (1, v)):
            page = s["page_table"][b, plane, p // c["tpp"]].long() - plane * s["cache"].shape[1]
            x = s["cache"][plane].view(torch.uint8)[page, p % c["tpp"]].view(s["cache"].dtype).double()
            if s["scales"] is not None:
                x = x * s["scales"][plane][page, :, p % c["tpp"]].double()[..., None]
            out[n] = x
        return {"k": k, "v": v}
    q, k, v = _exact_write(s)
    if c["op"] == "mrope":
        kc, vc = s["key_cache"].double(), s["value_cache"].double()
        kc.flatten(0, 1)[s["slots"]], vc.flatten(0, 1)[s["slots"]] = k, v
        return {"q": q, "k": kc, "v": vc}
    big = E4M3_MAX if c["format"] == "e4m3" else INT8_MAX
    scales = s["scales"].double()
    block, at = s["slots"] // c["bs"], s["slots"] % c["bs"]
    unit = [x.abs().max(-1).values / big for x in (k, v)]
    for plane in (0, 1):
        scales[plane, block, :, at] = unit[plane]
    if c["op"] == "quant":
        # the values before they are rounded to E4M3: what every rounding is half a step from
        kv = torch.zeros(s["cache"].shape, dtype=torch.float64, device=DEV)
        for plane, x in ((0, k), (1, v)):
            kv[plane].flatten(0, 1)[s["slots"]] = x / unit[plane][..., None]
        return {"q": q, "kv": kv, "scales": scales}
    code = s["cache"].double()
    for plane, x in ((0, k), (1, v)):
        code[plane].flatten(0, 1)[s["slots"]] = torch.round(x / unit[plane][..., None])
    p = torch.arange(c["context"] + c["T"], device=DEV)
    page = s["page_table"][0, 0][p // c["bs"]].long()
    back = [code[plane][page, p % c["bs"]] * scales[plane][page, :, p % c["bs"]][..., None]
            for plane in (0, 1)]
    return {"q": q, "scales": scales, "k": back[0], "v": back[1]}
