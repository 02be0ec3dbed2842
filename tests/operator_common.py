"""Float64 definitions and input builders of the decode-serving operators'
tests (attention over a paged cache, eviction, logits rules)."""
import math

import numpy as np
import torch

D = 64
E32 = 2.0 ** -24                     # half a step of fp32, relative
EB = 2.0 ** -8                       # half a step of bf16, relative


class AttnCase:
    """A pool whose every element outside the slots' live positions is NaN, with random pages, and random chunks."""

    def __init__(self, chunks, lens, hq=4, hkv=2, page=64, dtype=torch.bfloat16, causal=True, layout="head", seed=0,
                 scale=0.125, req_ids=None, slots=None, spare_rows=3, dev="cuda", amp=1.5):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.chunks, self.lens, self.hq, self.hkv, self.page, self.dtype = list(chunks), list(lens), hq, hkv, page, dtype
        self.causal, self.scale, self.G = causal, scale, hq // hkv
        n = len(self.chunks)
        self.ids = list(range(n)) if req_ids is None else list(req_ids)
        self.slots = slots or n
        slot_len = [0] * self.slots
        for i, s in enumerate(self.ids):
            if 0 <= s < self.slots:
                slot_len[s] = self.lens[i]
        self.slot_len = slot_len
        width = max(1, max(-(-x // page) for x in slot_len))
        total = self.slots * width + 2
        perm = torch.randperm(total, generator=g)[: self.slots * width].reshape(self.slots, width).to(torch.int32)
        shape = (total, hkv, page, D) if layout == "head" else (total, page, hkv, D)
        k, v = (torch.full(shape, math.nan, dtype=dtype) for _ in range(2))
        if layout != "head":
            k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
        for s in range(self.slots):
            for p in range(-(-slot_len[s] // page)):
                m = min(page, slot_len[s] - p * page)
                for x in (k, v):
                    x[perm[s, p], :, :m] = torch.randn(hkv, m, D, generator=g).to(dtype)
        strided = layout != "head"
        def up(x):
            return x.permute(0, 2, 1, 3).contiguous().to(dev).permute(0, 2, 1, 3) if strided else x.to(dev)
        self.k, self.v, self.table = up(k), up(v), perm.to(dev)
        rows = sum(self.chunks)
        self.rows = rows
        self.q_all = (torch.randn(rows + spare_rows, hq, D, generator=g) * amp).to(dtype).to(dev)
        self.q = self.q_all[: rows + spare_rows]
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(self.chunks)]).astype(np.int32), device=dev)
        self.kv_len = torch.tensor(slot_len, dtype=torch.int32, device=dev)
        self.req = None if req_ids is None else torch.tensor(self.ids, dtype=torch.int32, device=dev)
        self.max_q, self.max_kv = max(1, max(self.chunks, default=1)), max(1, max(slot_len))
        self.mass0 = torch.rand(self.slots, hkv, self.max_kv + 5, generator=g).to(dev)

    def reference(self, bad_pages=()):
        """(out, lse, mass, allowed errors of each) in float64: outputs of the first `rows` rows."""
        bf = self.dtype is torch.bfloat16
        out = torch.zeros(self.rows, self.hq, D, dtype=torch.float64)
        lse = torch.full((self.rows, self.hq), -math.inf, dtype=torch.float64)
        mass = self.mass0.double().cpu().clone()
        t_out, t_lse, t_mass = torch.zeros_like(out), torch.zeros_like(lse), mass.abs() * E32
        row = 0
        for i, c in enumerate(self.chunks):
            s = self.ids[i]
            L = self.slot_len[s] if 0 <= s < self.slots else 0
            ok = torch.ones(max(L, 1), dtype=torch.bool)[:L]
            if L:
                pg = self.table[s, : -(-L // self.page)].cpu().long().clamp(0, self.k.shape[0] - 1)
                k = self.k.cpu()[pg].transpose(1, 2).reshape(-1, self.hkv, D)[:L].double()
                v = self.v.cpu()[pg].transpose(1, 2).reshape(-1, self.hkv, D)[:L].double()
                for b in bad_pages:
                    ok[b * self.page: (b + 1) * self.page] = False
            for t in range(c):
                lim = min(L, max(0, L - c + t + 1)) if self.causal else L
                see = ok[:lim]
                if not bool(see.any()):
                    row += 1
                    continue
                for u in range(self.hq):
                    h = u // self.G
                    q = self.q[row, u].cpu().double()
                    kk, vv = k[:lim, h][see], v[:lim, h][see]
                    z = kk @ q * self.scale
                    w = torch.exp(z - torch.logsumexp(z, 0))
                    out[row, u], lse[row, u] = w @ vv, torch.logsumexp(z, 0)
                    mass[s, h, :lim][see] += w
                    # a score: 64 products and sums, the scaling and the exponent's argument in fp32; the exponential
                    # itself is good to 2^-21; a running sum of m terms to m steps
                    ds = 70 * E32 * abs(self.scale) * float((kk.abs() @ q.abs()).max()) + 6 * E32 * float(z.abs().max()) + 2.0 ** -20
                    m = len(z)
                    mean = w @ vv.abs()
                    t_out[row, u] = (2 * ds + m * E32 + (EB if bf else 0)) * mean + ((EB if bf else E32) * out[row, u].abs()) + 1e-30
                    t_lse[row, u] = ds + m * E32 + 4 * E32 * lse[row, u].abs() + 4 * E32
                    t_mass[s, h, :lim][see] += w * (2 * ds + 2 * m * E32 + 4 * E32 * lse[row, u].abs()) + 1e-30
                row += 1
        heads = c_rows = sum(self.chunks) * self.G
        t_mass += c_rows * E32 * mass.abs()
        del heads
        return (out, lse, mass), (t_out * 1.01, t_lse, t_mass)


def close(name, got, want, tol):
    got, want = got.double().cpu(), want.cpu()
    same_inf = torch.isinf(want)
    assert torch.equal(got[same_inf], want[same_inf]), name
    err = (got - want).abs()[~same_inf]
    lim = tol.cpu()[~same_inf]
    assert bool(torch.isfinite(got[~same_inf]).all()), f"{name}: not finite"
    bad = err > lim
    assert not bool(bad.any()), f"{name}: {float((err / lim.clamp(min=1e-300)).max()):.3g} times the allowed error, {int(bad.sum())} places"


def evict_rule(mass, L, keep, sink, recent):
    """Kept positions, ascending, of one slot and head."""
    k = min(L, keep)
    key = []
    for j in range(L):
        m = float(mass[j])
        m = 0.0 if (math.isnan(m) or m < 0) else m
        key.append((0 if (j < sink or j >= L - recent) else 1, -m, j))
    return sorted(j for _, _, j in sorted(key)[:k])


def rules_rule(z, history, hist_len, block, block_len, window, rep, pres, freq, bias, masks, mask_row):
    """New logits step by step in numpy float32; the target and the log probability in float64."""
    n, H, V = z.shape
    f = np.float32
    out, target, lp = z.copy(), np.full((n, H), -1, np.int32), np.zeros((n, H))
    for i in range(n):
        for j in range(H if block_len is None else min(H, block_len[i])):
            seen = ([] if history is None else [int(t) for t in history[i][: max(0, min(hist_len[i], len(history[i])))]])
            if block is not None:
                seen += [int(t) for t in block[i][1: j + 1]]
            if window > 0:
                seen = seen[-window:]
            y = z[i, j].astype(f).copy()
            counts = {}
            for t in seen:
                if 0 <= t < V:
                    counts[t] = counts.get(t, 0) + 1
            th = f(1) if rep is None else f(rep[i])
            al, fr = (f(0) if a is None else f(a[i]) for a in (pres, freq))
            with np.errstate(all="ignore"):
                for t, c in counts.items():
                    x = f(y[t] / th) if y[t] > 0 else f(y[t] * th)
                    y[t] = f(x - f(f(fr * f(c)) + al))
                used = set()
                if bias is not None:
                    ids, vals, lens = bias
                    for e in range(max(0, min(lens[i], ids.shape[1]))):
                        b = int(ids[i, e])
                        if 0 <= b < V and b not in used:
                            used.add(b)
                            y[b] = f(y[b] + f(vals[i, e]))
                if masks is not None and 0 <= mask_row[i, j] < len(masks):
                    w = masks[mask_row[i, j]].astype(np.uint32)
                    bits = (w[:, None] >> np.arange(32, dtype=np.uint32)) & 1
                    y[bits.reshape(-1)[:V] == 0] = -np.inf
                out[i, j] = y
                c = np.where(np.isnan(y), -np.inf, y).astype(np.float64)
                best = int(np.argmax(c))
                if c[best] == -np.inf:
                    lp[i, j] = -np.inf
                else:
                    target[i, j] = best
                    y64 = y.astype(np.float64)
                    e = np.where(y64 == c[best], 1.0, np.exp(y64 - c[best]))
                    lp[i, j] = -np.log(e.sum())
    return out, target, lp
