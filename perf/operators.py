"""Cases of the decode-serving operators: attention of a chunk of new tokens
over a paged key/value cache (with its log-sum-exp and the accumulated
attention weight of every cached position), eviction from that cache by the
accumulated weight, and the penalties, biases and grammar masks of the logits.

``run`` computes an operator either in its plain form (elementary torch
operations in fp32) or, with ``own`` set, through the framework's entry
points.  ``exact`` gives the definition in float64.
"""
import math

import torch

own = False

D = 64                  # head width of the framework's caches
FLT_MAX = 3.4028234663852886e38
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one beam step of one request: self-attention of one new token over a full 448-position decoder cache
        dict(name="attend-1", op="attend", n=1, c=1, kv=448, hq=20, hkv=20, page=64, dtype="bf16", causal=True,
             mass=False, ragged=False),
        # batch-96 block verification: 9 rows per request against up to 1500 acoustic frames, weights accumulated
        dict(name="attend-verify-b96", op="attend", n=96, c=9, kv=1500, hq=20, hkv=20, page=64, dtype="bf16",
             causal=False, mass=True, ragged=True),
        # single-token serving of long transcripts with shared key/value heads
        dict(name="attend-long-gqa", op="attend", n=16, c=1, kv=65536, hq=32, hkv=8, page=64, dtype="bf16",
             causal=True, mass=False, ragged=True),
        # a prompt chunk appended to cached context, with the weights an eviction needs
        dict(name="attend-prefill", op="attend", n=4, c=2048, kv=8192, hq=20, hkv=20, page=16, dtype="bf16",
             causal=True, mass=True, ragged=True),
        # the fp32 model (tiny widths): a 16-row block over its decoder cache
        dict(name="attend-f32", op="attend", n=8, c=16, kv=448, hq=6, hkv=6, page=64, dtype="f32", causal=True,
             mass=True, ragged=True),
        # one request's 1500 acoustic frames (one slab) cut to half
        dict(name="evict-1", op="evict", n=1, kv=1500, hkv=20, page=1500, dtype="bf16", keep=750, sink=0, recent=0,
             ragged=False),
        # a batch of 96 requests: up to 1500 frames cut to 512
        dict(name="evict-b96", op="evict", n=96, kv=1500, hkv=20, page=64, dtype="bf16", keep=512, sink=4,
             recent=32, ragged=True),
        # long transcripts cut to a quarter, first and last positions kept
        dict(name="evict-long", op="evict", n=8, kv=65536, hkv=8, page=64, dtype="bf16", keep=16384, sink=4,
             recent=1024, ragged=True),
        # the fp32 model's decoder cache, small pages
        dict(name="evict-f32", op="evict", n=7, kv=448, hkv=6, page=16, dtype="f32", keep=200, sink=1, recent=50,
             ragged=True),
        # one token of one request: everything a decoding step applies
        dict(name="rules-1", op="rules", n=1, h=1, vocab=51866, hist=224, window=0, bias=16, masks=4),
        # the fallback decoder: penalties alone on odd-sized rows
        dict(name="rules-b16", op="rules", n=16, h=9, vocab=51865, hist=448, window=0, bias=0, masks=0),
        # batch-96 block verification: a grammar state per row, recent tokens penalised
        dict(name="rules-b96", op="rules", n=96, h=9, vocab=51866, hist=448, window=64, bias=64, masks=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "evict", "rules"])
    if op == "attend":
        f32 = rng.random() < 0.25
        hkv = rng.choice([1, 2, 5, 6, 8, 20])
        hq = hkv * rng.choice([1, 1, 2, 4])
        n, c = _log(rng, 1, 96), _log(rng, 1, 2048)
        kv = max(c, _log(rng, 16, 65536))
        # no more work than the largest listed cases: score elements, and bytes of cache
        while n * hq * c * kv > (2 ** 27 if f32 else 2 ** 30) or n * hkv * kv > 2 ** 22:
            if n > 1:
                n = n // 2
            elif c > 1:
                c = c // 2
            else:
                kv = kv // 2
        return dict(op=op, n=n, c=c, kv=max(kv, c), hq=hq, hkv=hkv, page=rng.choice([16, 32, 64, 128, 100]),
                    dtype="f32" if f32 else "bf16", causal=rng.random() < 0.7, mass=rng.random() < 0.5,
                    ragged=rng.random() < 0.8)
    if op == "evict":
        hkv = rng.choice([1, 2, 6, 8, 20])
        n, kv = _log(rng, 1, 96), _log(rng, 32, 65536)
        while n * hkv * kv > 2 ** 22:
            n, kv = max(1, n // 2), (kv if n > 1 else kv // 2)
        keep = max(1, int(kv * rng.uniform(0.1, 0.9)))
        return dict(op=op, n=n, kv=kv, hkv=hkv, page=rng.choice([16, 32, 64, 128, 100]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), keep=keep, sink=rng.randint(0, min(4, keep)),
                    recent=int((keep - min(4, keep)) * rng.uniform(0, 0.5)), ragged=rng.random() < 0.8)
    return dict(op=op, n=_log(rng, 1, 96), h=rng.randint(1, 9), vocab=_log(rng, 1000, 65536), hist=_log(rng, 8, 448),
                window=rng.choice([0, 0, 16, 100]), bias=rng.choice([0, 1, 33, 64]), masks=rng.choice([0, 1, 7, 64]))


def _spread(n, lo, hi):
    """n lengths over lo..hi, the first the largest: a function of the sizes alone."""
    return [hi if i == 0 else lo + int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _chunks(case):
    n, c = case["n"], case["c"]
    return _spread(n, max(1, c // 2), c) if case["ragged"] else [c] * n


def _kv_lens(case):
    n, kv = case["n"], case["kv"]
    if not case["ragged"]:
        return [kv] * n
    lens = _spread(n, max(1, kv // 4), kv)
    return [max(a, b) for a, b in zip(lens, _chunks(case))] if case["op"] == "attend" else lens


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _pages(lens, page, g, start=0):
    """A page table whose requests own disjoint pages of a shuffled pool."""
    per = [-(-x // page) for x in lens]
    width, total = max(per), sum(per)
    perm = (torch.randperm(total, generator=g, device=DEV) + start).to(torch.int32)
    slot = torch.zeros(len(lens), width, dtype=torch.int64, device=DEV)
    count = torch.as_tensor(per, device=DEV)
    first = torch.cumsum(count, 0) - count
    slot = (first[:, None] + torch.arange(width, device=DEV)[None]).clamp_(max=total - 1)
    table = torch.where(torch.arange(width, device=DEV)[None] < count[:, None], perm[slot], torch.full_like(perm[slot], start))
    return table.contiguous(), total


def _i32(v):
    return torch.as_tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case, op=case["op"])
    if case["op"] == "rules":
        n, h, V = case["n"], case["h"], case["vocab"]
        s["logits"] = torch.randn(n, h, V, generator=g, device=DEV) * 3.0
        s["out"] = torch.zeros(n, h, V, device=DEV)
        # transcripts repeat a few frequent tokens
        s["history"] = (torch.rand(n, case["hist"], generator=g, device=DEV) ** 3 * V).to(torch.int32).clamp_(max=V - 1)
        s["hist_len"] = _i32(_spread(n, case["hist"] // 2, case["hist"]))
        s["block"] = (torch.rand(n, h, generator=g, device=DEV) ** 3 * V).to(torch.int32).clamp_(max=V - 1)
        s["block_len"] = _i32(_spread(n, max(1, h // 2), h))
        s["repetition"] = 1.0 + 0.3 * torch.rand(n, generator=g, device=DEV)
        s["presence"] = 0.5 * torch.rand(n, generator=g, device=DEV)
        s["frequency"] = 0.3 * torch.rand(n, generator=g, device=DEV)
        s["bias_ids"] = s["bias_vals"] = s["bias_len"] = s["masks"] = s["mask_row"] = None
        if case["bias"]:
            s["bias_ids"] = torch.randint(0, V, (n, case["bias"]), generator=g, device=DEV, dtype=torch.int32)
            s["bias_vals"] = 4.0 * torch.randn(n, case["bias"], generator=g, device=DEV)
            s["bias_len"] = _i32(_spread(n, case["bias"] // 2, case["bias"]))
        if case["masks"]:
            words = -(-V // 32)
            bits = torch.randint(-2 ** 31, 2 ** 31, (2, case["masks"], words), generator=g, device=DEV, dtype=torch.int64)
            s["masks"] = (bits[0] & bits[1]).to(torch.int32)
            s["mask_row"] = torch.randint(-1, case["masks"], (n, h), generator=g, device=DEV, dtype=torch.int32)
        s["target"] = torch.full((n, h), -1, dtype=torch.int32, device=DEV)
        s["logprob"] = torch.zeros(n, h, device=DEV)
        if own:
            from speculative_whisper_asr_gb300 import runtime as R
            s["rules"] = R.LogitsRules(repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                                       window=case["window"], bias_ids=s["bias_ids"], bias_vals=s["bias_vals"],
                                       bias_len=s["bias_len"], masks=s["masks"])
        return s

    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    n, hkv, page = case["n"], case["hkv"], case["page"]
    lens = _kv_lens(case)
    s["kv_len"] = _i32(lens)
    s["table"], total = _pages(lens, page, g)
    if case["op"] == "attend":
        c = _chunks(case)
        s["pool"] = torch.randn(total, 2, hkv, page, D, generator=g, device=DEV, dtype=dt)
        s["cu_q"] = _i32([0] + [sum(c[: i + 1]) for i in range(n)])
        s["q"] = torch.randn(sum(c), case["hq"], D, generator=g, device=DEV, dtype=dt) * 1.5
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(sum(c), case["hq"], device=DEV)
        s["mass"] = torch.rand(n, hkv, case["kv"], generator=g, device=DEV) if case["mass"] else None
    else:
        new = [min(x, case["keep"]) for x in lens]
        s["table_out"], more = _pages(new, page, g, start=total)
        s["pool"] = torch.randn(total + more, 2, hkv, page, D, generator=g, device=DEV, dtype=dt)
        s["pool"][total:] = 0
        s["dst"] = total
        # accumulated weights: a few positions hold most, some were never looked at
        w = torch.exp(2.0 * torch.randn(n, hkv, case["kv"], generator=g, device=DEV))
        s["mass"] = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.1, torch.zeros_like(w), w)
        s["pos"] = torch.arange(case["kv"], device=DEV, dtype=torch.int32).expand(n, hkv, case["kv"]).contiguous()
        s["mass_out"] = torch.zeros(n, hkv, case["keep"], device=DEV)
        s["pos_out"] = torch.zeros(n, hkv, case["keep"], dtype=torch.int32, device=DEV)
        s["kv_len_out"] = torch.zeros(n, dtype=torch.int32, device=DEV)
    if own:
        from speculative_whisper_asr_gb300 import runtime as R
        s["cache"] = R.PagedCache(s["pool"][:, 0], s["pool"][:, 1], s["table"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if s["op"] == "attend":
        return _attend_own(s) if own else _attend(s)
    if s["op"] == "evict":
        return _evict_own(s) if own else _evict(s)
    return _rules_own(s) if own else _rules(s)


def _attend_own(s):
    case = s["case"]
    s["cache"].attend(s["q"], s["kv_len"], s["cu_q"], max_q=case["c"], max_kv=case["kv"], causal=case["causal"],
                      out=s["out"], lse=s["lse"], mass=s["mass"])
    return [s["out"], s["lse"], s["mass"]]


def _evict_own(s):
    case = s["case"]
    s["cache"].evict(s["kv_len"], s["mass"], keep=case["keep"], max_kv=case["kv"], sink=case["sink"],
                     recent=case["recent"], page_table_out=s["table_out"], kv_len_out=s["kv_len_out"],
                     mass_out=s["mass_out"], pos=s["pos"], pos_out=s["pos_out"])
    return [s["pool"][s["dst"]:], s["mass_out"], s["pos_out"], s["kv_len_out"]]


def _rules_own(s):
    s["rules"].apply(s["logits"], history=s["history"], hist_len=s["hist_len"], block=s["block"],
                     block_len=s["block_len"], mask_row=s["mask_row"], out=s["out"], target=s["target"],
                     logprob=s["logprob"])
    return [s["out"], s["target"], s["logprob"]]


def _dense(pool, table, kv):
    """[n, Hkv, kv, D] fp32 keys or values of the requests' pages."""
    x = pool[table.long()]                                    # [n, P, Hkv, page, D]
    n, P, H, page, _ = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, H, P * page, D)[:, :, :kv].float()


def _attend(s):
    case = s["case"]
    n, c, kv, hq, hkv = case["n"], case["c"], case["kv"], case["hq"], case["hkv"]
    G = hq // hkv
    start, count = s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    r = torch.arange(c, device=DEV)
    live = r[None] < count[:, None]                           # [n, c]
    rows = (start[:, None] + r[None]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().reshape(n, c, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(n, hkv, c * G, D)
    k, v = _dense(s["pool"][:, 0], s["table"], kv), _dense(s["pool"][:, 1], s["table"], kv)
    z = torch.matmul(q, k.transpose(2, 3)).mul_(0.125)        # [n, hkv, c * G, kv]
    t, L = torch.arange(kv, device=DEV), s["kv_len"].long()
    see = (t[None, None] < L[:, None, None]) & live[:, :, None]
    if case["causal"]:
        see = see & (t[None, None] <= (L - count)[:, None, None] + r[None, :, None])
    see = see[:, None, :, None].expand(n, 1, c, G, kv).reshape(n, 1, c * G, kv)
    z.masked_fill_(~see, -math.inf)
    m = z.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = z.sub_(m).exp_()
    l = p.sum(3, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0, torch.ones_like(l), l)
    o = o.reshape(n, hkv, c, G, D).permute(0, 2, 1, 3, 4).reshape(n, c, hq, D)
    lse = (m + torch.log(l)).reshape(n, hkv, c, G).permute(0, 2, 1, 3).reshape(n, c, hq)
    s["out"][rows[live]] = o[live].to(s["out"].dtype)
    s["lse"][rows[live]] = lse[live]
    if s["mass"] is not None:
        s["mass"] += p.div_(torch.where(l == 0, torch.ones_like(l), l)).sum(2)
    return [s["out"], s["lse"], s["mass"]]


def _evict(s):
    case = s["case"]
    n, hkv, kv, keep, page = case["n"], case["hkv"], case["kv"], case["keep"], case["page"]
    L = s["kv_len"].long()
    t = torch.arange(kv, device=DEV)
    inside = t[None] < L[:, None]
    held = inside & ((t[None] < case["sink"]) | (t[None] >= L[:, None] - case["recent"]))
    key = torch.nan_to_num(s["mass"], nan=0.0, posinf=FLT_MAX).clamp(min=0.0)
    key = torch.where(held[:, None], torch.full_like(key, math.inf), key)
    key = torch.where(inside[:, None], key, torch.full_like(key, -1.0))
    best = torch.sort(key, dim=2, descending=True, stable=True).indices[:, :, :keep]
    if best.shape[2] < keep:
        best = torch.nn.functional.pad(best, (0, keep - best.shape[2]), value=kv)
    new = torch.clamp(L, max=keep)
    j = torch.arange(keep, device=DEV)
    best = torch.where(j[None, None] < new[:, None, None], best, torch.full_like(best, kv))
    src = torch.sort(best, dim=2).values                      # ascending positions, then the unused places
    fill = (j[None] < new[:, None])[:, None].expand(n, hkv, keep)
    i, h, jj = torch.nonzero(fill, as_tuple=True)
    p = src[i, h, jj]
    from_page, to_page = s["table"].long()[i, p // page], s["table_out"].long()[i, jj // page]
    s["pool"][to_page, :, h, jj % page] = s["pool"][from_page, :, h, p % page]
    s["mass_out"][i, h, jj] = s["mass"][i, h, p]
    s["pos_out"][i, h, jj] = s["pos"][i, h, p]
    s["kv_len_out"].copy_(new)
    return [s["pool"][s["dst"]:], s["mass_out"], s["pos_out"], s["kv_len_out"]]


def _rules(s):
    case = s["case"]
    n, H, V, Sh, W = case["n"], case["h"], case["vocab"], case["hist"], case["window"]
    j, hl = torch.arange(H, device=DEV), s["hist_len"].long()
    total = hl[:, None] + j[None]                             # tokens before row j: the transcript, then proposals 1..j
    ph = torch.arange(Sh, device=DEV)
    pb = hl[:, None] + torch.arange(H - 1, device=DEV)[None]
    place = torch.cat([ph[None].expand(n, Sh), pb], 1)        # [n, Sh + H - 1] places in the token sequence
    tok = torch.cat([s["history"], s["block"][:, 1:]], 1).long()
    real = torch.cat([ph[None] < hl[:, None], torch.ones_like(pb, dtype=torch.bool)], 1)
    use = real[:, None] & (place[:, None] < total[:, :, None])
    if W:
        use = use & (place[:, None] >= total[:, :, None] - W)
    use = use & ((tok >= 0) & (tok < V))[:, None]
    idx = torch.where(use, tok[:, None].expand_as(use), torch.full_like(use, V, dtype=torch.long))
    count = torch.zeros(n, H, V + 1, device=DEV).scatter_add_(2, idx, use.float())[:, :, :V]
    theta, al, fr = (s[k][:, None, None] for k in ("repetition", "presence", "frequency"))
    y = s["logits"]
    hit = count > 0
    y = torch.where(hit, torch.where(y > 0, y / theta, y * theta) - (fr * count + al), y)
    if s["bias_ids"] is not None:
        nb = case["bias"]
        e = torch.arange(nb, device=DEV)
        ids = s["bias_ids"].long()
        ids = torch.where((e[None] < s["bias_len"][:, None]) & (ids >= 0) & (ids < V), ids, torch.full_like(ids, V))
        first = torch.full((n, V + 1), nb, dtype=torch.long, device=DEV)
        first = first.scatter_reduce(1, ids, e[None].expand(n, nb), "amin")[:, :V]
        add = torch.gather(s["bias_vals"], 1, first.clamp(max=nb - 1))
        y = torch.where((first < nb)[:, None], y + add[:, None], y)
    if s["masks"] is not None:
        v = torch.arange(V, device=DEV)
        row = s["mask_row"].long()
        on = (row >= 0) & (row < s["masks"].shape[0])
        word = s["masks"][:, v >> 5]                          # [masks, V]
        allow = ((word >> (v & 31)[None].to(torch.int32)) & 1).bool()
        y = torch.where(on[:, :, None] & ~allow[row.clamp(0, allow.shape[0] - 1)], torch.full_like(y, -math.inf), y)
    live = j[None] < s["block_len"].long()[:, None]
    best, at = y.max(2)
    at = torch.argmax(y, 2)
    lp = -torch.log(torch.where(y == best[:, :, None], torch.ones_like(y), torch.exp(y - best[:, :, None])).sum(2))
    none = best == -math.inf
    lp = torch.where(none, best, lp)
    at = torch.where(none, torch.full_like(at, -1), at)
    s["out"].copy_(torch.where(live[:, :, None], y, s["out"]))
    s["target"].copy_(torch.where(live, at, torch.full_like(at, -1)))
    s["logprob"].copy_(torch.where(live, lp, torch.zeros_like(lp)))
    return [s["out"], s["target"], s["logprob"]]


# ------------------------------------------------------------------ the work that cannot be done without
def work(case):
    if case["op"] == "rules":
        rows = sum(_spread(case["n"], max(1, case["h"] // 2), case["h"]))
        V = case["vocab"]
        b = rows * V * 8 + rows * 8 + case["n"] * (4 * case["hist"] + 8 * case["bias"] + 12)
        b += min(case["masks"], rows) * (-(-V // 32)) * 4
        return dict(bytes=b, flops=3 * rows * V)
    es = 2 if case["dtype"] == "bf16" else 4
    lens = _kv_lens(case)
    if case["op"] == "evict":
        new = sum(min(x, case["keep"]) for x in lens)
        # every weight is read; each kept position's key, value, weight and position is read and written
        b = case["hkv"] * (4 * sum(lens) + new * (2 * 2 * D * es + 2 * 4 + 4))
        return dict(bytes=b, flops=case["hkv"] * sum(lens))
    c = _chunks(case)
    pairs = sum(a * L - (a * (a - 1) // 2 if case["causal"] else 0) for a, L in zip(c, lens))
    b = 2 * sum(lens) * case["hkv"] * D * es + 2 * sum(c) * case["hq"] * D * es + sum(c) * case["hq"] * 4
    if case["mass"]:
        b += 8 * sum(lens) * case["hkv"]
    return dict(bytes=b, flops=4 * D * pairs * case["hq"])


# ------------------------------------------------------------------ the definition in float64
def exact(case, seed):
    s = prepare(dict(case), seed)
    if case["op"] == "attend":
        return _exact_attend(s, case)
    if case["op"] == "evict":
        return _exact_evict(s, case)
    return _exact_rules(s, case)


def _exact_attend(s, case):
    G, page = case["hq"] // case["hkv"], case["page"]
    out, lse = s["out"].double(), s["lse"].double()
    mass = None if s["mass"] is None else s["mass"].double()
    cu, lens = s["cu_q"].tolist(), s["kv_len"].tolist()
    for i, L in enumerate(lens):
        a, e = cu[i], cu[i + 1]
        pages = s["table"][i, : -(-L // page)].long()
        kv = s["pool"][pages].double()                        # [P, 2, Hkv, page, D]
        last = L - (e - a) + torch.arange(e - a, device=DEV) if case["causal"] else torch.full((e - a,), L - 1, device=DEV)
        for h in range(case["hkv"]):
            k, v = (kv[:, w, h].reshape(-1, D)[:L] for w in (0, 1))
            for u in range(h * G, (h + 1) * G):
                z = (s["q"][a:e, u].double() @ k.T) / 8.0
                z[torch.arange(L, device=DEV)[None] > last[:, None]] = -math.inf
                norm = torch.logsumexp(z, 1)
                w = torch.exp(z - norm[:, None])
                out[a:e, u], lse[a:e, u] = w @ v, norm
                if mass is not None:
                    mass[i, h, :L] += w.sum(0)
    return [out, lse, mass]


def _exact_evict(s, case):
    page, keep = case["page"], case["keep"]
    pool, mass = s["pool"].double(), s["mass"].cpu().double()
    w_out, p_out = s["mass_out"].double(), s["pos_out"]
    for i, L in enumerate(s["kv_len"].tolist()):
        if L * case["hkv"] * case["n"] > 5e6:
            return None
        k = min(L, keep)
        for h in range(case["hkv"]):
            w = mass[i, h, :L].clone()
            w[: case["sink"]] = math.inf
            w[L - min(L, case["recent"]):] = math.inf
            chosen = torch.argsort(-w, stable=True)[:k].sort().values.to(DEV)
            dst = torch.arange(k, device=DEV)
            a, b = s["table"][i].long(), s["table_out"][i].long()
            pool[b[dst // page], :, h, dst % page] = pool[a[chosen // page], :, h, chosen % page]
            w_out[i, h, :k] = s["mass"][i, h, chosen].double()
            p_out[i, h, :k] = chosen.to(torch.int32)
        s["kv_len_out"][i] = k
    return [pool[s["dst"]:], w_out, p_out, s["kv_len_out"]]


def _exact_rules(s, case):
    V, W = case["vocab"], case["window"]
    out, lp = s["out"].double(), s["logprob"].double()
    for i in range(case["n"]):
        hist = s["history"][i, : int(s["hist_len"][i])].tolist()
        block = s["block"][i].tolist()
        th, al, fr = (float(s[k][i]) for k in ("repetition", "presence", "frequency"))
        for j in range(int(s["block_len"][i])):
            seen = hist + block[1: j + 1]
            seen = seen[-W:] if W else seen
            y = s["logits"][i, j].double()
            if seen:
                ids, c = torch.unique(torch.as_tensor(seen, device=DEV), return_counts=True)
                z = y[ids]
                y[ids] = torch.where(z > 0, z / th, z * th) - fr * c.double() - al
            if s["bias_ids"] is not None:
                used = {}
                for b, val in list(zip(s["bias_ids"][i].tolist(), s["bias_vals"][i].double().tolist()))[: int(s["bias_len"][i])]:
                    used.setdefault(b, val)
                if used:
                    y[torch.as_tensor(list(used), device=DEV)] += torch.as_tensor(list(used.values()), device=DEV, dtype=torch.float64)
            m = -1 if s["mask_row"] is None else int(s["mask_row"][i, j])
            if m >= 0:
                word = s["masks"][m].long() & 0xFFFFFFFF
                bits = (word[:, None] >> torch.arange(32, device=DEV)[None]) & 1
                y[bits.reshape(-1)[:V] == 0] = -math.inf
            out[i, j] = y
            lp[i, j] = y.max() - torch.logsumexp(y, 0)
    return [out, None, lp]
