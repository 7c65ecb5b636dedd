"""Plain 64-bit implementations and seeded inputs of the serving operators
(numpy, no code shared with the kernels), and the error bounds the GPU results
are held to.

Half a rounding step relative to the value: FP16 2^-11, FP32 2^-24, E4M3 2^-4.
"""
import numpy as np

NEOX, GPTJ = 0, 1
F16, E4M3, INT8 = "f16", "e4m3", "int8"
MAXCODE = {E4M3: 448.0, INT8: 127.0}


def e4m3_table():
    """Value of each of the 256 E4M3 codes, from the format's definition."""
    out = np.empty(256)
    for b in range(256):
        s, e, m = -1.0 if b & 0x80 else 1.0, (b >> 3) & 15, b & 7
        out[b] = s * (m * 2.0 ** -9 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
        if b & 0x7F == 0x7F:
            out[b] = np.nan
    return out


E4M3_VALUES = e4m3_table()


def decode(codes, fmt):
    return E4M3_VALUES[codes.view(np.uint8)] if fmt == E4M3 else codes.astype(np.float64)


def rotate(x, cos, sin, r, style):
    """[T, H, D] float64 rotated on its first r dims; cos, sin [T, r/2]. Also the sum of
    magnitudes |x cos| + |partner sin| of every element (|x| past r)."""
    y, mag = x.copy(), np.abs(x)
    i = np.arange(r // 2)
    a, b = (i, i + r // 2) if style == NEOX else (2 * i, 2 * i + 1)
    c, s = cos[:, None, :], sin[:, None, :]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
    mag[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, mag


def check_f16(got, want, mag, what):
    """FP16 results of a two-term FP32 sum: half an FP16 step of the value (or of the
    subnormal step 2^-24), and three FP32 roundings of terms of size `mag`."""
    tol = 2.0 ** -11 * np.abs(want) + 3 * 2.0 ** -24 * mag * 1.01 + 2.0 ** -25
    err = np.abs(got.astype(np.float64) - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err / tol)[bad].max())} x the bound"


def table(rows, r, theta=1e4):
    ang = np.arange(rows)[:, None] * theta ** (-2.0 * np.arange(r // 2) / r)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


# --------------------------------------------------------------- attention --

class AttentionCase:
    """A paged pool in which only the slots that some sequence owns hold finite
    values: everything else (codes and scales) is NaN."""

    def __init__(self, seed, B, S, Hq, Hkv, D, tpp, prefix, own, fmt, q_scale=1.0, v_scale=1.0,
                 unmapped=0.0, spread=0.0):
        rng = np.random.Generator(np.random.PCG64(seed))
        own = list(own)
        assert len(own) == B
        self.B, self.S, self.Hq, self.Hkv, self.D, self.tpp = B, S, Hq, Hkv, D, tpp
        self.P, self.fmt = prefix, fmt
        # own[b] = tokens behind the prefix (with the S new ones); None = inactive (length 0)
        self.kv_lens = np.array([0 if n is None else prefix + n for n in own], np.int32)
        top = max([prefix + (n or 0) for n in own] + [1])
        cols = -(-top // tpp)
        first, shared = prefix // tpp, -(-prefix // tpp)
        need = [0 if n is None else -(-(prefix + n) // tpp) - first for n in own]
        pages = shared + sum(need) + 2
        kid, vid = rng.permutation(pages), rng.permutation(pages) + pages
        self.pages = pages
        self.prefix_table = np.stack([kid[:shared], vid[:shared]]).astype(np.int32)
        self.page_table = np.full((B, 2, cols), -1, np.int32)
        at = shared
        for b in range(B):
            self.page_table[b, 0, first:first + need[b]] = kid[at:at + need[b]]
            self.page_table[b, 1, first:first + need[b]] = vid[at:at + need[b]]
            at += need[b]
        if unmapped:
            for t in (self.prefix_table, self.page_table):
                drop = rng.random(t.shape) < unmapped
                t[drop & (t >= 0)] = rng.choice([-1, -7, 2 * pages + 5])
        self.q = (rng.standard_normal((B, S, Hq, D)) * q_scale).astype(np.float16)
        shape = (2, pages, tpp, Hkv, D)
        x = rng.standard_normal(shape)
        x[1] *= v_scale
        if spread:  # heads of very different sizes
            x *= 2.0 ** rng.uniform(-spread, spread, shape[:4])[..., None]
        if fmt == F16:
            self.pool, self.scales = x.astype(np.float16), None
        else:
            scale = np.abs(x).max(-1) / MAXCODE[fmt]
            self.scales = scale.astype(np.float32).transpose(0, 1, 3, 2).copy()
            u = x / scale[..., None]
            if fmt == INT8:
                self.pool = np.rint(u).astype(np.int8)
            else:
                order = np.argsort(np.where(np.isnan(E4M3_VALUES), 1e9, E4M3_VALUES))[:254]
                v = E4M3_VALUES[order]
                i = np.clip(np.searchsorted(v, u), 1, 253)
                near = np.where(np.abs(v[i] - u) < np.abs(v[i - 1] - u), i, i - 1)
                self.pool = order[near].astype(np.uint8)
        self._poison()

    def _poison(self):
        used = np.zeros((2, self.pages, self.tpp), bool)

        def mark(tab, lo, hi):
            for p in range(lo, hi):
                for plane in (0, 1):
                    i = tab[plane, p // self.tpp] - plane * self.pages
                    if 0 <= i < self.pages:
                        used[plane, i, p % self.tpp] = True
        mark(self.prefix_table, 0, self.P)
        for b in range(self.B):
            mark(self.page_table[b], self.P, self.kv_lens[b])
        if self.fmt == F16:
            self.pool[~used] = np.nan
        else:
            self.pool[~used] = 0x7F if self.fmt == E4M3 else 77
            s = self.scales.transpose(0, 1, 3, 2).copy()
            s[~used] = np.nan
            self.scales = s.transpose(0, 1, 3, 2).copy()

    def values(self):
        x = decode(self.pool, self.fmt)
        return x if self.scales is None else x * self.scales.astype(np.float64).transpose(0, 1, 3, 2)[..., None]

    def solve(self, sm_scale=None, batch=None):
        """(out, lse, tol_out, tol_lse) in 64 bits, of the sequences in `batch` (default: all).

        Bounds, with s the scores in natural units, w = softmax, N positions:
          score: D products of FP16 values are exact, their FP32 sum (tensor cores may
            truncate: 2^-23 a step) is off by ds <= D 2^-23 sum|q k| c, c = sm_scale, and
            three roundings of the scale product (one more from the code's scale);
          weight: e^ds - 1, ex2 2^-22, one FP16 rounding 2^-11 and the FP32 product with
            the V scale; below FP16's normal range 2^-25 absolute, relative to the largest
            weight (>= 1, V scales at most doubled by their power of two);
          sums: N 2^-23 relative for O and for l; joining parts: a few 2^-23;
          result: one FP16 rounding."""
        c = sm_scale if sm_scale is not None else self.D ** -0.5
        kv = self.values()
        out = np.zeros((self.B, self.S, self.Hq, self.D))
        lse = np.full((self.B, self.S, self.Hq), -np.inf)
        tol_o, tol_l = np.zeros_like(out), np.zeros_like(lse)
        G = self.Hq // self.Hkv

        def rows(tab, lo, hi):
            ks, vs = [], []
            for p in range(lo, hi):
                if p // self.tpp >= tab.shape[1]:
                    break
                i, j = tab[0, p // self.tpp], tab[1, p // self.tpp] - self.pages
                if 0 <= i < self.pages and 0 <= j < self.pages:
                    ks.append((p, kv[0, i, p % self.tpp]))
                    vs.append(kv[1, j, p % self.tpp])
            return ks, vs
        pre = rows(self.prefix_table, 0, self.P)
        for b in range(self.B) if batch is None else batch:
            mine = rows(self.page_table[b], self.P, int(self.kv_lens[b]))
            ks, vs = pre[0] + mine[0], pre[1] + mine[1]
            if not ks:
                continue
            pos = np.array([p for p, _ in ks])
            K, V = np.stack([k for _, k in ks]), np.stack(vs)       # [N, Hkv, D]
            for s in range(self.S):
                last = int(self.kv_lens[b]) - self.S + s
                see = pos <= last
                if last < self.P or not see.any():
                    continue
                k = np.repeat(K[see], G, 1)
                v = np.repeat(V[see], G, 1)
                q = self.q[b, s].astype(np.float64)
                sc = np.einsum("hd,nhd->hn", q, k) * c
                mag = np.einsum("hd,nhd->hn", np.abs(q), np.abs(k)) * abs(c)
                m = sc.max(1, keepdims=True)
                e = np.exp(sc - m)
                L = e.sum(1, keepdims=True)
                w = e / L
                out[b, s] = np.einsum("hn,nhd->hd", w, v)
                lse[b, s] = (m + np.log(L))[:, 0]
                N = see.sum()
                ds = (self.D + 4) * 2.0 ** -23 * mag.max(1) + 4 * 2.0 ** -24 * np.abs(sc).max(1)
                wv = np.einsum("hn,nhd->hd", w, np.abs(v))
                rel = 2 * np.expm1(ds) + 2.0 ** -11 + (2 * N + 40) * 2.0 ** -23
                tol_o[b, s] = rel[:, None] * wv + 2.0 ** -11 * np.abs(out[b, s]) + 2.0 ** -24 \
                    + 2.0 ** -24 * np.abs(v).max((0, 2))[:, None] * N / L
                tol_l[b, s] = ds + (N + 40) * 2.0 ** -23 + 2.0 ** -22 * np.abs(lse[b, s])
        return out, lse, tol_o, tol_l
