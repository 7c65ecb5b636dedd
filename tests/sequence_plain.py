"""Plain 64-bit implementations of the operators on whole sequences (torch, no code
shared with the kernels), and the error bounds that GPU results are held to.

Half a rounding step relative to the value: FP16 2^-11, FP32 2^-24.
"""
import math

import torch


def attend(q, k, v, sees, scale=None):
    """Rows q [n, Hq, D] against keys k, v [t, Hkv, D], row i seeing key j where sees[i, j]; all in
    64 bits: (out [n, Hq, D], lse [n, Hq], tol_out, tol_lse).

    Bounds, with s the scores in natural units, w = softmax, N keys, c = scale:
      score: D products of FP16 values are exact, their FP32 sum (tensor cores may truncate:
        2^-23 a step) is off by ds <= D 2^-23 sum|q k| |c|, and three roundings of the scale product;
      weight: e^ds - 1, ex2 2^-22, one FP16 rounding 2^-11; below FP16's normal range 2^-25 absolute,
        relative to the largest weight (>= 1);
      sums: N 2^-23 relative for O and for l; joining parts: a few 2^-23;
      result: one FP16 rounding (below its normal range 2^-25 absolute).
    A value of V that is not finite makes the elements of out that see it not finite."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    c = D ** -0.5 if scale is None else scale
    q, k, v = q.double(), k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    hide = ~sees[None]
    zero = torch.zeros((), dtype=torch.float64, device=q.device)
    sc = (torch.einsum("nhd,thd->hnt", q, k) * c).masked_fill(hide, -math.inf)
    mag = (torch.einsum("nhd,thd->hnt", q.abs(), k.abs()) * abs(c)).masked_fill(hide, 0)
    any_ = sees.any(1)[None, :, None]
    if k.shape[0] == 0:
        return (zero.expand(n, Hq, D), torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device),
                zero.expand(n, Hq, D), zero.expand(n, Hq))
    m = torch.where(any_, sc.amax(-1, keepdim=True), zero)
    e = torch.where(hide, zero, torch.exp(sc - m))
    L = e.sum(-1, keepdim=True)
    w = torch.where(any_, e / L, zero)
    fine = torch.where(v.isfinite(), v, zero)
    out = torch.einsum("hnt,thd->nhd", w, fine)
    bad = torch.where(v.isfinite(), zero, v)
    if (~v.isfinite()).any():
        for t in torch.nonzero((~v.isfinite()).flatten(1).any(1))[:, 0].tolist():
            out = out + torch.where(sees[:, t, None, None], bad[t], zero)
    lse = torch.where(any_, m + torch.log(L), -math.inf)[..., 0].t()
    N = sees.sum(1)[None, :, None].double()
    ds = (D + 4) * 2.0 ** -23 * mag.amax(-1, keepdim=True) + 4 * 2.0 ** -24 * sc.masked_fill(hide, 0).abs().amax(-1, keepdim=True)
    rel = 2 * torch.expm1(ds) + 2.0 ** -11 + (2 * N + 40) * 2.0 ** -23                     # [Hq, n, 1]
    wv = torch.einsum("hnt,thd->nhd", w, fine.abs())
    small = 2.0 ** -24 * fine.abs().amax((0, 2))[:, None, None] * N / L.clamp(min=1e-300)    # [Hq, n, 1]
    tol_o = rel.permute(1, 0, 2) * wv + 2.0 ** -11 * out.abs() + 2.0 ** -24 + torch.where(any_, small, zero).permute(1, 0, 2)
    tol_l = (ds + (N + 40) * 2.0 ** -23)[..., 0].t() + 2.0 ** -22 * torch.where(lse.isfinite(), lse.abs(), zero)
    return out, lse, tol_o, tol_l


def check(got, want, tol, what):
    got = got.double()
    fine = want.isfinite()
    assert torch.equal(got.isfinite(), fine), f"{what}: other elements are finite: {int((got.isfinite() != fine).sum())}"
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: other elements are NaN"
    assert torch.equal(got[~fine].nan_to_num(0.5), want[~fine].nan_to_num(0.5)), f"{what}: other infinities"
    err, tol = (got - want)[fine].abs(), tol.expand(want.shape)[fine]
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol)[bad].max())} x the bound"


def causal(nq, nk, device="cpu"):
    i, t = torch.arange(nq, device=device)[:, None], torch.arange(nk, device=device)[None]
    return t <= nk - nq + i


def tree_sees(mask, S):
    """[S, S] of one sequence's mask words [S, W]."""
    j = torch.arange(S, device=mask.device)
    return (mask.long()[:, j // 32] >> (j % 32) & 1) == 1


# ------------------------------------------------------------------ pages --

def accept(rows, lens, S, accepted, accepted_lens, cap):
    """rows(b, p): the row (any tensor) of position p, or None; moved in the order of j. Returns
    {(b, p): row} of what is written, and the new lengths."""
    new, out = {}, list(lens)
    for b, n in enumerate(lens):
        count = max(0, min(accepted_lens[b], min(S, len(accepted[b]))))
        for j in range(count):
            a = accepted[b][j]
            src, dst = n - S + a, n - S + j
            if a < j or a >= S or not 0 <= src < cap or not 0 <= dst < cap:
                continue
            x = rows(b, src)
            if x is not None and rows(b, dst) is not None:
                new[b, dst] = x
        if n >= S:
            out[b] = n - S + count
    return new, out


def fork(table, lens, refs, parents, children, tpp):
    """In place on lists: table [B][2][M], lens [B], refs [P]. Returns the copies [(src page, dst page, tokens)]."""
    B, M, P = len(lens), len(table[0][0]) if table else 0, len(refs)
    ok = [0 <= p < B and 0 <= c < B for p, c in zip(parents, children)]
    named = [c for c, o in zip(children, ok) if o]
    heads = {p for p, o in zip(parents, ok) if o}
    todo = [i for i, o in enumerate(ok) if o and named.count(children[i]) == 1 and children[i] not in heads
            and lens[children[i]] <= 0]
    free = [p for p in range(P) if refs[p] <= 0]
    copies = []
    for i in todo:
        p, c = parents[i], children[i]
        n = min(max(lens[p], 0), M * tpp)
        whole, rest = divmod(n, tpp)
        row = [x if 0 <= x < P else -1 for x in table[p][0][:whole]]
        for x in row:
            if x >= 0:
                refs[x] += 1
        if rest:
            tail = table[p][0][whole]
            if 0 <= tail < P and free:
                page = free.pop(0)
                copies.append((tail, page, rest))
                refs[page] = 1
                row.append(page)
            else:
                n = whole * tpp
        row += [-1] * (M - len(row))
        table[c][0], table[c][1] = row, [x + P if x >= 0 else -1 for x in row]
        lens[c] = n
    return copies


def free(table, lens, refs, sequences, keep, tpp):
    B, M, P = len(lens), len(table[0][0]) if table else 0, len(refs)
    for i, s in enumerate(sequences):
        if not 0 <= s < B:
            continue
        k = max(0, keep[i]) if keep is not None else 0
        for col in range(-(-k // tpp), M):
            x = table[s][0][col]
            if 0 <= x < P:
                refs[x] -= 1
            table[s][0][col] = table[s][1][col] = -1
        lens[s] = min(lens[s], k)
