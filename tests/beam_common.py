"""Float64 definitions and input builders of the beam-search serving operators'
tests (appending to paged caches, caches in 8 bits, beam selection, reordering)."""
import math

import numpy as np
import torch

from operator_common import AttnCase

D = 64
E32 = 2.0 ** -24


# ------------------------------------------------------------------ e4m3 with powers of two
def e4m3_value(codes):
    """float64 values of e4m3 codes (uint8 array)."""
    c = np.asarray(codes).astype(np.int64)
    e, m = c >> 3 & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def e4m3_round(x):
    """Nearest e4m3 value (ties to even) of float64 numbers up to 448; what is not finite becomes NaN."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        step = 2.0 ** (np.maximum(np.frexp(np.abs(x))[1] - 1, -6) - 3)
        return np.where(np.isfinite(x), np.round(x / step) * step, np.nan)


def needed_exponent(m):
    """Exponent of the smallest power of two s >= 2^-127 with m <= 448 s."""
    e = -127
    while m > 448.0 * 2.0 ** e:
        e += 1
    return e


def turned(x, pos, inv_freq, dims, adjacent):
    """Rows [n, heads, 64] (float64) turned by pos [n]."""
    y = np.array(x, dtype=np.float64)
    if inv_freq is None:
        return y
    a = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(inv_freq)[None]
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    i = np.arange(dims // 2)
    p, q = (2 * i, 2 * i + 1) if adjacent else (i, i + dims // 2)
    u, v = y[..., p].copy(), y[..., q].copy()
    y[..., p], y[..., q] = u * c - v * s, u * s + v * c
    return y


class Pool:
    """A cache's tensors on the GPU, random contents, and the same as float64 numpy arrays for the rules below.

    layout: "head" [pages, heads, tokens, 64], "token" [pages, tokens, heads, 64] or "pair" (keys and values of a page
    beside each other)."""

    def __init__(self, slots, width, hkv, page, dtype, block=0, layout="head", seed=0, spare=2, dev="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.slots, self.width, self.hkv, self.page, self.dtype, self.block, self.dev = slots, width, hkv, page, dtype, block, dev
        pages = slots * width + spare
        q8 = dtype is torch.float8_e4m3fn
        if q8:
            codes = torch.randint(0, 256, (2, pages, hkv, page, D), generator=g, dtype=torch.uint8)
            codes = torch.where((codes & 0x7F) == 0x7F, codes - 1, codes)
            raw = codes.view(torch.float8_e4m3fn)
        else:
            raw = torch.randn(2, pages, hkv, page, D, generator=g).to(dtype)

        def up(x):
            x = x.view(torch.uint8) if q8 else x
            if layout == "token":
                x = x.permute(0, 2, 1, 3).contiguous().to(dev).permute(0, 2, 1, 3)
            elif layout == "pair":
                box = torch.empty(pages, 2, hkv, page, D, dtype=x.dtype, device=dev)
                box[:, 0] = x.to(dev)
                x = box[:, 0]
            else:
                x = x.contiguous().to(dev)
            return x.view(dtype)
        self.k, self.v = up(raw[0]), up(raw[1])
        self.table = torch.randperm(pages, generator=g)[: slots * width].reshape(slots, width).to(torch.int32).to(dev)
        self.scales = None
        if q8:
            self.scales = torch.randint(118, 128, (2, pages, hkv, page // block), generator=g, dtype=torch.uint8).to(dev)

    def cache(self, R):
        if self.scales is None:
            return R.PagedCache(self.k, self.v, self.table)
        return R.PagedCache(self.k, self.v, self.table, k_scale=self.scales[0], v_scale=self.scales[1])

    def read(self):
        """(contents [2, pages, heads, tokens, 64] as stored, float64; scale exponents or None; table)."""
        if self.scales is None:
            x = torch.stack([self.k, self.v]).double().cpu().numpy()
            return x, None, self.table.cpu().numpy().copy()
        x = torch.stack([self.k.view(torch.uint8), self.v.view(torch.uint8)]).cpu().numpy()
        return e4m3_value(x), self.scales.cpu().numpy().astype(np.int64) - 127, self.table.cpu().numpy().copy()

    def bits(self):
        ks = [t.contiguous().view(torch.uint8).cpu().clone() for t in (self.k, self.v)]
        return ks + ([] if self.scales is None else [self.scales.cpu().clone()]) + [self.table.cpu().clone()]


def append_rule(before, table, page, block, k, v, kv_len, cu, max_q, ids, inv_freq, dims, adjacent, pos, q=None):
    """What an append leaves: (contents, exponents, allowed error of each content, queries, rows with queries).
    k, v, q: float64 [rows, heads, 64]."""
    x, ex = before
    x, ex = x.copy(), None if ex is None else ex.copy()
    tol = np.zeros_like(x)
    n_pages = x.shape[1]
    q_out = None if q is None else q.copy()
    seen = np.zeros(len(k), dtype=bool)
    for i in range(len(cu) - 1):
        slot = i if ids is None else ids[i]
        if not 0 <= slot < len(table):
            continue
        c = min(max(cu[i + 1] - cu[i], 0), max_q)
        start = kv_len[slot] - c
        rows = [r for r in range(c) if start + r >= 0]
        if not rows:
            continue
        at = np.array([cu[i] + r for r in rows])
        places = np.array([start + r for r in rows])
        m = places if pos is None else pos[at]
        kk = turned(k[at], m, inv_freq, dims, adjacent)
        size = np.abs(k[at]).max(-1, keepdims=True)
        if q is not None:
            q_out[at] = turned(q[at], m, inv_freq, dims, adjacent)
        seen[at] = True

        def page_of(t):
            e = t // page
            g = int(table[slot, e]) if e < table.shape[1] else -1
            return g if 0 <= g < n_pages else -1
        for w, new in ((0, kk), (1, v[at])):
            # a turned element: two products, a sum, a cosine and a sine good to 2^-22
            err = size * 2.0 ** -21 if w == 0 and inv_freq is not None else np.zeros_like(size)
            err = np.broadcast_to(err, new.shape)
            if not block:
                for j, t in enumerate(places):
                    g = page_of(t)
                    if g >= 0:
                        x[w, g, :, t % page], tol[w, g, :, t % page] = new[j], err[j]
                continue
            for b in sorted({int(t) // block for t in places}):
                g = page_of(b * block)
                if g < 0:
                    continue
                js = [j for j, t in enumerate(places) if t // block == b]
                t0 = b * block % page
                for h in range(x.shape[2]):
                    rowsx = new[js, h]
                    fin = np.abs(rowsx[np.isfinite(rowsx)])
                    e = needed_exponent(fin.max() if fin.size else 0.0)
                    if b * block < places[0]:
                        was = ex[w, g, h, t0 // block]
                        e = max(e, was)
                        old = x[w, g, h, t0: t0 + places[0] - b * block]
                        if e > was:
                            old[:] = e4m3_round(old * 2.0 ** int(was - e))
                    ex[w, g, h, t0 // block] = e
                    for j in js:
                        x[w, g, h, places[j] % page] = e4m3_round(new[j, h] * 2.0 ** -int(e))
                        tol[w, g, h, places[j] % page] = err[j, h] * 2.0 ** -int(e)
    return x, ex, tol, q_out, seen


def check_appended(name, got, want, tol, quantized):
    """Contents against the rule: exact where nothing was turned; a turned element may round to the other side of a
    border that it is within its error of."""
    same_nan = np.isnan(got) == np.isnan(want)
    assert same_nan.all(), f"{name}: NaN in other places ({int((~same_nan).sum())})"
    g, w = np.nan_to_num(got), np.nan_to_num(want)
    off = np.abs(g - w)
    exact = tol == 0
    assert not off[exact].any(), f"{name}: {int((off[exact] > 0).sum())} elements that no rounding explains"
    if quantized:
        step = 2.0 ** (np.maximum(np.frexp(np.maximum(np.abs(g), np.abs(w)))[1] - 1, -6) - 3)
        moved = off > 0
        assert (off <= step * 1.0001)[moved].all(), f"{name}: more than one step off"
        # a border lies within the error with a chance of twice the error over the step
        expected = (2 * tol / step)[~exact].sum()
        assert moved.sum() <= 4 * expected + 4, f"{name}: {int(moved.sum())} elements at another step, {expected:.2g} expected"


# ------------------------------------------------------------------ attention over a cache in 8 bits
class Q8Case(AttnCase):
    """The bf16 case with its live contents rounded to e4m3 with a scale per block, and the cache in 8 bits that
    stands for the same values; codes that are not live are NaN and scales of blocks without live positions 255."""

    def __init__(self, *a, block=16, spread=3, tails=0, seed=0, **kw):
        super().__init__(*a, dtype=torch.bfloat16, seed=seed, **kw)
        g = torch.Generator().manual_seed(seed + 1)
        self.block = block
        pages, hkv, page = self.k.shape[:3]
        self.codes, self.scales = [], torch.full((2, pages, hkv, page // block), 255, dtype=torch.uint8)
        for w, x in enumerate((self.k, self.v)):
            y = x.float().cpu().reshape(pages, hkv, page // block, block, D)
            y = y * torch.exp2(torch.randint(-spread, spread + 1, y.shape[:3], generator=g).float())[..., None, None]
            if tails:                      # every exponent and the numbers below the normal ones occur
                y = y * torch.exp2(-torch.randint(0, tails + 1, y.shape, generator=g).float())
            live = ~torch.isnan(y[..., 0])
            m = torch.nan_to_num(y).abs().amax((3, 4))
            e = torch.tensor([needed_exponent(float(t)) for t in m.reshape(-1)]).reshape(m.shape)
            q = torch.from_numpy(e4m3_round((y * torch.exp2(-e.float())[..., None, None]).double().numpy()))
            self.scales[w][live.any(3)] = (e + 127).to(torch.uint8)[live.any(3)]
            code = q.float().to(torch.float8_e4m3fn)
            code = torch.where(live[..., None], code.view(torch.uint8), torch.full_like(code.view(torch.uint8), 0x7F))
            self.codes.append(code.reshape(pages, hkv, page, D))
            value = (q * torch.exp2(e.double())[..., None, None]).reshape(x.shape)
            x.copy_(torch.where(torch.isnan(x.double().cpu()), x.double().cpu(), value).to(torch.bfloat16))
        strided = self.k.stride(2) != D

        def up(c):
            c = c.permute(0, 2, 1, 3).contiguous().to(self.k.device).permute(0, 2, 1, 3) if strided else c.to(self.k.device)
            return c.view(torch.float8_e4m3fn)
        self.k8, self.v8 = up(self.codes[0]), up(self.codes[1])
        self.scales = self.scales.to(self.k.device)

    def cache(self, R):
        return R.PagedCache(self.k8, self.v8, self.table, k_scale=self.scales[0], v_scale=self.scales[1])


# ------------------------------------------------------------------ beam selection
def beam_rule(logits, score, eos, tokens=None, length=None, n_done=None, room=0):
    """One step for float32 arrays: dict of outputs, scores in float64; done: per request a list of
    (score, transcript)."""
    n, B, V = logits.shape
    cap = None if tokens is None else tokens.shape[2]
    out = dict(parent=np.tile(np.arange(B), (n, 1)), token=np.full((n, B), -1), score=np.full((n, B), -np.inf),
               tokens=[], done=[[] for _ in range(n)], idle=np.zeros(n, dtype=bool))
    for i in range(n):
        L = 0 if length is None else length[i]
        if (n_done is not None and n_done[i] >= room) or (cap is not None and L >= cap):
            out["score"][i] = score[i]
            out["idle"][i] = True
            out["tokens"].append(None if tokens is None else [list(tokens[i, b, :L]) for b in range(B)])
            continue
        cand = []
        for b in range(B):
            z = logits[i, b].astype(np.float64)
            if not np.isfinite(score[i, b]) or np.isnan(z).any() or (z == np.inf).any() or not (z > -np.inf).any():
                continue
            m = z.max()
            c = float(score[i, b]) + (z - m - math.log(np.exp(z - m).sum()))
            best = np.lexsort((np.arange(V), -z))[: 2 * B]
            cand += [(-c[v], b, int(v)) for v in best if z[v] > -np.inf]
        live = 0
        had = 0 if n_done is None else int(n_done[i])
        for c, b, v in sorted(cand):
            if v == eos:
                if n_done is not None and had + len(out["done"][i]) < room:
                    out["done"][i].append((-c, None if tokens is None else list(tokens[i, b, :L])))
                continue
            out["parent"][i, live], out["token"][i, live], out["score"][i, live] = b, v, -c
            live += 1
            if live == B:
                break
        out["tokens"].append(None if tokens is None else
                             [list(tokens[i, out["parent"][i, b], :L]) + [out["token"][i, b]] for b in range(B)])
    return out
