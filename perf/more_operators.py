"""Cases of the beam-search serving operators: appending keys and values to a
paged cache with the position rotation applied on the way (bf16, fp32, or 8
bits with a scale for each block of tokens and head), attention over a cache
held in 8 bits, the selection of a beam-search step over beams and vocabulary,
and the reordering of paged caches by the beams' parents.

A cache in 8 bits holds e4m3 values; block b of a page and head has one scale
2^(s - 127) for its keys and one for its values.  Appended rows x of a block
take the smallest power of two with max |x| <= 448 * scale, or keep the
block's scale where earlier tokens of the block need a larger one; where the
scale grows, the block's earlier tokens are rounded to it.

``run`` computes an operator either in its plain form (elementary torch
operations) or, with ``own`` set, through the framework's entry points.
``exact`` gives the definition in float64.
"""
import math

import torch

own = False

D = 64                  # head width of the framework's caches
DEV = "cuda"
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one beam step of one request on the model's own cache type: its token's keys, values and queries
        dict(name="append-1", op="append", n=1, c=1, kv=448, hq=20, hkv=20, page=64, block=0, dtype="bf16",
             rotate="adjacent", dims=64, shift=0, ragged=False),
        # batch-96 nine-row blocks onto 8-bit decoder caches: blocks of 16 tokens, most of them begun before the call
        dict(name="append-b96-8bit", op="append", n=96, c=9, kv=448, hq=20, hkv=20, page=64, block=16, dtype="e4m3",
             rotate="adjacent", dims=64, shift=0, ragged=True),
        # prompt chunks with shared key/value heads, far along a transcript whose cache was cut (positions run ahead)
        dict(name="append-chunk-8bit", op="append", n=4, c=2048, kv=8192, hq=32, hkv=8, page=64, block=64, dtype="e4m3",
             rotate="halves", dims=64, shift=1000003, ragged=True),
        # the fp32 model: 16-row blocks, half of each head rotated
        dict(name="append-f32", op="append", n=8, c=16, kv=448, hq=6, hkv=6, page=16, block=0, dtype="f32",
             rotate="adjacent", dims=32, shift=0, ragged=True),
        # one token of one request over its 8-bit decoder cache
        dict(name="attend8-1", op="attend", n=1, c=1, kv=448, hq=20, hkv=20, page=64, block=64, causal=True, ragged=False),
        # batch-96 block verification: 9 rows per request against up to 1500 acoustic frames in 8 bits
        dict(name="attend8-verify-b96", op="attend", n=96, c=9, kv=1500, hq=20, hkv=20, page=64, block=32, causal=False,
             ragged=True),
        # single-token serving of long transcripts with shared key/value heads
        dict(name="attend8-long-gqa", op="attend", n=16, c=1, kv=65536, hq=32, hkv=8, page=64, block=64, causal=True,
             ragged=True),
        # a prompt chunk appended to cached context, small pages
        dict(name="attend8-chunk", op="attend", n=4, c=2048, kv=8192, hq=20, hkv=20, page=16, block=16, causal=True,
             ragged=True),
        # one request's beam step: five beams, the fallback decoder's width
        dict(name="beam-1", op="beam", n=1, beams=5, vocab=51866, length=224, done=5),
        # a batch of 96 requests
        dict(name="beam-b96", op="beam", n=96, beams=5, vocab=51866, length=224, done=5),
        # one request's five caches
        dict(name="reorder-1", op="reorder", n=1, beams=5, kv=430, hkv=20, page=64, block=0, dtype="bf16", ragged=False),
        # 96 requests, the caches of four layers side by side as heads, in 8 bits
        dict(name="reorder-b96-8bit", op="reorder", n=96, beams=5, kv=448, hkv=80, page=64, block=16, dtype="e4m3",
             ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _paging(rng):
    page = rng.choice([16, 32, 64, 128, 48])
    return page, rng.choice([b for b in (8, 16, 32, 64, 128, 48) if page % b == 0])


def draw(rng):
    op = rng.choice(["append", "attend", "beam", "reorder"])
    page, block = _paging(rng)
    if op == "append":
        dtype = rng.choice(["bf16", "e4m3", "e4m3", "f32"])
        hkv = rng.choice([1, 2, 5, 6, 8, 20])
        hq = hkv * rng.choice([1, 1, 2, 4])
        n, c = _log(rng, 1, 96), _log(rng, 1, 2048)
        kv = max(c, _log(rng, 16, 8192))
        while n * c * (hq + 2 * hkv) > 4 * 2048 * 48 or n * hkv * kv > 2 ** 20:
            if n > 1:
                n = n // 2
            elif c > 1:
                c = c // 2
            else:
                kv = kv // 2
        return dict(op=op, n=n, c=c, kv=max(kv, c), hq=hq, hkv=hkv, page=page, block=block if dtype == "e4m3" else 0,
                    dtype=dtype, rotate=rng.choice(["adjacent", "halves", "none"]), dims=rng.choice([64, 64, 32, 16]),
                    shift=rng.choice([0, 0, 70000, 5000011]), ragged=rng.random() < 0.8)
    if op == "attend":
        hkv = rng.choice([1, 2, 5, 6, 8, 20])
        hq = hkv * rng.choice([1, 1, 2, 4])
        n, c = _log(rng, 1, 96), _log(rng, 1, 2048)
        kv = max(c, _log(rng, 16, 65536))
        while n * hq * c * kv > 2 ** 30 or n * hkv * kv > 2 ** 22:
            if n > 1:
                n = n // 2
            elif c > 1:
                c = c // 2
            else:
                kv = kv // 2
        return dict(op=op, n=n, c=c, kv=max(kv, c), hq=hq, hkv=hkv, page=page, block=block, causal=rng.random() < 0.7,
                    ragged=rng.random() < 0.8)
    if op == "beam":
        n, beams, vocab = _log(rng, 1, 96), rng.randint(1, 12), _log(rng, 500, 65536)
        while n * beams * vocab > 96 * 5 * 51866:
            n = n // 2
        return dict(op=op, n=n, beams=beams, vocab=vocab, length=_log(rng, 1, 440), done=rng.randint(1, 8))
    hkv, n, beams, kv = _log(rng, 1, 80), _log(rng, 1, 96), rng.randint(2, 12), _log(rng, 4, 2048)
    while n * beams * hkv * (kv + page) > 96 * 5 * 80 * 448:
        if n > 1:
            n = n // 2
        elif kv > 4:
            kv = kv // 2
        else:
            hkv = max(1, hkv // 2)
    dtype = rng.choice(["bf16", "f32", "e4m3"])
    if dtype != "e4m3":
        hkv = max(1, hkv // 4)
    return dict(op=op, n=n, beams=beams, kv=kv, hkv=hkv, page=page, block=block if dtype == "e4m3" else 0, dtype=dtype,
                ragged=rng.random() < 0.8)


def _spread(n, lo, hi):
    """n lengths over lo..hi, the first the largest: a function of the sizes alone."""
    return [hi if i == 0 else lo + int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _chunks(case):
    n, c = case["n"], case["c"]
    return _spread(n, max(1, c // 2), c) if case["ragged"] else [c] * n


def _kv_lens(case):
    n, kv = case["n"], case["kv"]
    lens = _spread(n, max(1, kv // 4), kv) if case["ragged"] else [kv] * n
    return [max(a, b) for a, b in zip(lens, _chunks(case))] if "c" in case else lens


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(v):
    return torch.as_tensor(v, dtype=torch.int32, device=DEV)


def _pages(lens, page, g):
    """A page table whose slots own disjoint pages of a shuffled pool."""
    per = [-(-x // page) for x in lens]
    width, total = max(per), sum(per)
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    count = torch.as_tensor(per, device=DEV)
    first = torch.cumsum(count, 0) - count
    at = torch.arange(width, device=DEV)[None]
    slot = (first[:, None] + at).clamp_(max=total - 1)
    table = torch.where(at < count[:, None], perm[slot], torch.zeros_like(perm[slot]))
    return table.contiguous(), total


def _needed(m):
    """Exponent of the smallest power of two s with m <= 448 s, in -127 .. 127 (fp32 or float64 maxima)."""
    f, e = torch.frexp(m)                                      # m = f 2^e, f in [1/2, 1); 448 = 0.875 * 2^9
    return torch.where(m > 0, e - 9 + (f > 0.875).to(e.dtype), torch.full_like(e, -127)).clamp(-127, 127)


def _two(e, dtype=torch.float32):
    """2^e for whole e in -254 .. 254, from its bits, in two factors (2^-127 is below fp32's normal numbers)."""
    h = torch.div(e, 2, rounding_mode="floor").to(torch.int32)
    return ((h + 127) << 23).view(torch.float32).to(dtype) * ((e.to(torch.int32) - h + 127) << 23).view(torch.float32).to(dtype)


def _quantized(x, block):
    """e4m3 values and scale bytes of x [..., page, 64] whose blocks are all full."""
    b = x.unflatten(-2, (-1, block))
    e = _needed(b.abs().amax((-2, -1)))
    return (b * _two(-e)[..., None, None]).flatten(-3, -2).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _pool(case, total, g, few=64):
    """A pool [pages, K|V, heads, page, 64]: key channels differ in size, and so do the tokens of one page from another's."""
    hkv, page = case["hkv"], case["page"]
    channel = torch.exp2(torch.randn(2, hkv, 1, D, generator=g, device=DEV))
    channel[1] = 1.0
    dt = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}[case["dtype"]]
    pool = torch.empty(total, 2, hkv, page, D, dtype=dt, device=DEV)
    scales = torch.empty(total, 2, hkv, page // case["block"], dtype=torch.uint8, device=DEV) if case["block"] else None
    for a in range(0, total, max(1, total // few)):
        e = min(total, a + max(1, total // few))
        x = torch.randn(e - a, 2, hkv, page, D, generator=g, device=DEV)
        x *= channel * torch.exp2(torch.randint(-2, 2, (e - a, 2, hkv, 1, 1), generator=g, device=DEV).float())
        if scales is None:
            pool[a:e] = x.to(dt)
        else:
            pool[a:e], scales[a:e] = _quantized(x, case["block"])
    return pool, scales


def prepare(case, seed):
    g = _gen(seed)
    case = dict(case)
    s = dict(case=case, op=case["op"])
    if case["op"] == "beam":
        return _prepare_beam(s, case, g)
    if case["op"] == "attend":
        case["dtype"] = "e4m3"
    beams = case.get("beams", 1)
    lens = _kv_lens(case)
    s["table"], total = _pages([x for x in lens for _ in range(beams)], case["page"], g)
    s["kv_len"] = _i32([x for x in lens for _ in range(beams)])
    s["pool"], s["scales"] = _pool(case, total, g)
    if case["op"] == "reorder":
        # the best beam tends to have several successors
        s["parent"] = (torch.rand(case["n"], beams, generator=g, device=DEV) ** 1.5 * beams).to(torch.int32)
    else:
        c, hq, hkv = _chunks(case), case["hq"], case["hkv"]
        rows = sum(c)
        s["cu_q"] = _i32([0] + [sum(c[: i + 1]) for i in range(case["n"])])
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        if case["op"] == "attend":
            s["q"] = (torch.randn(rows, hq, D, generator=g, device=DEV) * 0.5).to(dt)
            s["out"] = torch.zeros_like(s["q"])
            s["lse"] = torch.zeros(rows, hq, device=DEV)
        else:
            # the rows of one projection: queries, keys and values side by side
            s["qkv"] = (torch.randn(rows, hq + 2 * hkv, D, generator=g, device=DEV)
                        * torch.exp2(torch.randint(-2, 2, (rows, 1, 1), generator=g, device=DEV).float())).to(dt)
            s["q"], s["k"], s["v"] = s["qkv"].split([hq, hkv, hkv], 1)
            s["q_out"] = torch.zeros(rows, hq, D, dtype=dt, device=DEV)
            s["inv"] = 10000.0 ** (-torch.arange(0, case["dims"], 2, dtype=torch.float64, device=DEV) / case["dims"])
            s["pos"] = None
            if case["shift"]:
                t = torch.arange(rows, device=DEV)
                i = torch.searchsorted(s["cu_q"].long(), t, right=True) - 1
                ahead = torch.randint(0, case["shift"], (case["n"],), generator=g, device=DEV)
                L, cu = s["kv_len"].long(), s["cu_q"].long()
                s["pos"] = (L[i] - (cu[i + 1] - t) + ahead[i]).to(torch.int32)
    if own:
        from speculative_whisper_asr_gb300 import runtime as R
        sc = (None, None) if s["scales"] is None else (s["scales"][:, 0], s["scales"][:, 1])
        s["cache"] = R.PagedCache(s["pool"][:, 0], s["pool"][:, 1], s["table"], k_scale=sc[0], v_scale=sc[1])
        if case["op"] == "append":
            s["rotation"] = None if case["rotate"] == "none" else R.Rotation(
                dims=case["dims"], base=10000.0, adjacent=case["rotate"] == "adjacent")
    return s


def _prepare_beam(s, case, g):
    n, B, V, L, F = case["n"], case["beams"], case["vocab"], case["length"], case["done"]
    # a decoder's logits: a few tokens far above the rest, the end of transcript among them now and then, and tokens
    # that the rules have taken out
    z = torch.randn(n, B, V, generator=g, device=DEV) * 2.0
    hot = torch.randint(0, V, (n, B, 8), generator=g, device=DEV)
    z.scatter_add_(2, hot, 8.0 + 4.0 * torch.rand(n, B, 8, generator=g, device=DEV))
    s["eos"] = V // 2
    z[:, :, s["eos"]] += 12.0 * torch.rand(n, B, generator=g, device=DEV)
    z[:, :, V - V // 30:] = -math.inf
    s["logits"] = z
    s["score"] = -(30.0 * torch.rand(n, 1, generator=g, device=DEV) + torch.cumsum(torch.rand(n, B, generator=g, device=DEV), 1))
    s["tokens"] = torch.randint(0, V, (n, B, 448), generator=g, device=DEV, dtype=torch.int32)
    s["length"] = _i32(_spread(n, max(1, L // 2), L))
    s["n_done"] = torch.randint(0, F, (n,), generator=g, device=DEV, dtype=torch.int32)
    s["parent"], s["token"] = (torch.zeros(n, B, dtype=torch.int32, device=DEV) for _ in range(2))
    s["score_out"], s["tokens_out"] = torch.zeros_like(s["score"]), torch.zeros_like(s["tokens"])
    s["length_out"], s["n_done_out"] = torch.zeros_like(s["length"]), torch.zeros_like(s["n_done"])
    s["done_score"] = torch.zeros(n, F, device=DEV)
    s["done_length"] = torch.zeros(n, F, dtype=torch.int32, device=DEV)
    s["done_tokens"] = torch.zeros(n, F, 448, dtype=torch.int32, device=DEV)
    if own:
        from speculative_whisper_asr_gb300 import runtime as R
        s["beam"] = R.BeamSearch(eos_id=s["eos"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"append": _append_own if own else _append, "attend": _attend_own if own else _attend,
            "beam": _beam_own if own else _beam, "reorder": _reorder_own if own else _reorder}[s["op"]](s)


def _cache_outputs(s):
    """The pool and, as the values they stand for, its scales."""
    return [s["pool"], None if s["scales"] is None else s["scales"].view(torch.float8_e8m0fnu)]


def _append_own(s):
    s["cache"].append(s["k"], s["v"], s["kv_len"], s["cu_q"], max_q=s["case"]["c"], rotation=s["rotation"], pos=s["pos"],
                      q=s["q"], q_out=s["q_out"])
    return _cache_outputs(s) + [s["q_out"]]


def _attend_own(s):
    case = s["case"]
    s["cache"].attend(s["q"], s["kv_len"], s["cu_q"], max_q=case["c"], max_kv=case["kv"], causal=case["causal"],
                      out=s["out"], lse=s["lse"])
    return [s["out"], s["lse"]]


def _beam_own(s):
    s["beam"].select(s["logits"], s["score"], s["parent"], s["token"], score_out=s["score_out"], tokens=s["tokens"],
                     length=s["length"], tokens_out=s["tokens_out"], length_out=s["length_out"], n_done=s["n_done"],
                     n_done_out=s["n_done_out"], done_score=s["done_score"], done_length=s["done_length"],
                     done_tokens=s["done_tokens"])
    return _beam_outputs(s)


def _beam_outputs(s):
    return [s[k] for k in ("parent", "token", "score_out", "tokens_out", "length_out", "n_done_out", "done_score",
                           "done_length", "done_tokens")]


def _reorder_own(s):
    s["cache"].reorder(s["parent"], s["kv_len"])
    return _cache_outputs(s) + [s["table"]]


def _rotated(x, pos, inv, kind):
    """x [rows, heads, 64] turned by pos [rows] * inv [dims / 2]: angles in float64, the rest in fp32."""
    if kind == "none":
        return x.float()
    a = pos.double()[:, None] * inv[None]
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    h = inv.shape[0]
    y = x.float()
    r = y[..., : 2 * h]
    if kind == "adjacent":
        p, q = r[..., 0::2], r[..., 1::2]
        t = torch.stack([p * cos - q * sin, p * sin + q * cos], -1).flatten(-2)
    else:
        p, q = r[..., :h], r[..., h:]
        t = torch.cat([p * cos - q * sin, p * sin + q * cos], -1)
    return torch.cat([t, y[..., 2 * h:]], -1)


def _append(s):
    case = s["case"]
    page, block = case["page"], case["block"]
    cu, L, table = s["cu_q"].long(), s["kv_len"].long(), s["table"].long()
    rows = s["q"].shape[0]
    t = torch.arange(rows, device=DEV)
    i = torch.searchsorted(cu, t, right=True) - 1
    place = L[i] - (cu[i + 1] - t)                             # position in the cache
    pos = place if s["pos"] is None else s["pos"].long()
    s["q_out"].copy_(_rotated(s["q"], pos, s["inv"], case["rotate"]))
    new = torch.stack([_rotated(s["k"], pos, s["inv"], case["rotate"]), s["v"].float()], 1)    # [rows, 2, heads, 64]
    to = table[i, place // page]
    if not block:
        s["pool"][to, :, :, place % page] = new.to(s["pool"].dtype)
        return _cache_outputs(s) + [s["q_out"]]
    # every block that a request's rows touch, dense: [n, blocks, 2, heads, block, 64]
    n, c = case["n"], case["c"]
    start = L - (cu[1:] - cu[:-1])
    nb = (c + block - 2) // block + 1
    b = (start // block)[:, None] + torch.arange(nb, device=DEV)[None]
    used = b * block < L[:, None]
    bc = torch.where(used, b, (start // block)[:, None])
    pg, sub = table.gather(1, bc * block // page), bc % (page // block)
    codes = s["pool"].view(torch.uint8).unflatten(3, (-1, block))
    old = codes.permute(0, 3, 1, 2, 4, 5)[pg, sub].view(torch.float8_e4m3fn).float()
    e_old = s["scales"].permute(0, 3, 1, 2)[pg, sub].int() - 127
    fresh = torch.zeros_like(old)
    j = place // block - (start // block)[i]
    fresh[i, j, :, :, place % block] = new
    p = b[:, :, None] * block + torch.arange(block, device=DEV)
    is_new = ((p >= start[:, None, None]) & (p < L[:, None, None]))[:, :, None, None, :, None]
    is_old = (p < start[:, None, None])[:, :, None, None, :, None]
    e_need = _needed(fresh.abs().amax((-2, -1)))
    first = (b * block >= start[:, None])[:, :, None, None]    # the block begins with this call
    e = torch.where(first, e_need, torch.maximum(e_old, e_need))
    moved = (old * _two(e_old - e)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    put = (fresh * _two(-e)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    val = torch.where(is_new, put, torch.where(is_old & ~first[..., None, None], moved, codes.permute(0, 3, 1, 2, 4, 5)[pg, sub]))
    a, k = torch.nonzero(used, as_tuple=True)
    codes.permute(0, 3, 1, 2, 4, 5)[pg[a, k], sub[a, k]] = val[a, k]
    s["scales"].permute(0, 3, 1, 2)[pg[a, k], sub[a, k]] = (e[a, k] + 127).to(torch.uint8)
    return _cache_outputs(s) + [s["q_out"]]


def _dense(s, w, kv, dtype=torch.float32):
    """[n, Hkv, kv, D] keys (w = 0) or values (1) of the requests' pages."""
    t = s["table"].long()
    x = s["pool"].view(torch.uint8)[:, w][t].view(torch.float8_e4m3fn).to(dtype)
    n, P, H, page, _ = x.shape
    f = _two(s["scales"][:, w][t].int() - 127, dtype)          # [n, P, H, blocks]
    x = (x.unflatten(3, (f.shape[3], -1)) * f[..., None, None]).flatten(3, 4)
    return x.permute(0, 2, 1, 3, 4).reshape(n, H, P * page, D)[:, :, :kv]


def _attend(s):
    case = s["case"]
    n, c, hq, hkv = case["n"], case["c"], case["hq"], case["hkv"]
    kv = case["kv"]
    G = hq // hkv
    start, count = s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    r = torch.arange(c, device=DEV)
    live = r[None] < count[:, None]                           # [n, c]
    rows = (start[:, None] + r[None]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().reshape(n, c, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(n, hkv, c * G, D)
    z = torch.matmul(q, _dense(s, 0, kv).transpose(2, 3)).mul_(0.125)        # [n, hkv, c * G, kv]
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
    o = torch.matmul(p, _dense(s, 1, kv)) / torch.where(l == 0, torch.ones_like(l), l)
    o = o.reshape(n, hkv, c, G, D).permute(0, 2, 1, 3, 4).reshape(n, c, hq, D)
    lse = (m + torch.log(l)).reshape(n, hkv, c, G).permute(0, 2, 1, 3).reshape(n, c, hq)
    s["out"][rows[live]] = o[live].to(s["out"].dtype)
    s["lse"][rows[live]] = lse[live]
    return [s["out"], s["lse"]]


def _beam(s):
    case = s["case"]
    n, B, V, F, eos = case["n"], case["beams"], case["vocab"], case["done"], s["eos"]
    z = s["logits"].double()
    c = s["score"].double()[:, :, None] + (z - torch.logsumexp(z, 2, keepdim=True))
    c = torch.where(torch.isfinite(c), c, torch.full_like(c, -math.inf)).flatten(1)
    K = min(2 * B, B * V)
    best, at = (x[:, :K] for x in torch.sort(c, dim=1, descending=True, stable=True))
    beam, tok = at // V, at % V
    real = best > -math.inf
    is_end = real & (tok == eos)
    lives = real & ~is_end
    rank = torch.cumsum(lives, 1) - 1                          # among the candidates that go on
    goes = lives & (rank < B)
    before = torch.cumsum(lives, 1) - lives.long()             # of those, before this candidate
    ends = is_end & (before < B)
    busy = (s["n_done"] < F) & (s["length"] < s["tokens"].shape[2])
    place = s["n_done"].long()[:, None] + torch.cumsum(ends, 1) - 1
    ends = ends & (place < F) & busy[:, None]
    own_b = torch.arange(B, device=DEV)[None].expand(n, B)
    parent, token = own_b.clone(), torch.full((n, B), -1, dtype=torch.long, device=DEV)
    score = torch.full((n, B), -math.inf, dtype=torch.float64, device=DEV)
    i, k = torch.nonzero(goes, as_tuple=True)
    parent[i, rank[i, k]], token[i, rank[i, k]], score[i, rank[i, k]] = beam[i, k], tok[i, k], best[i, k]
    parent = torch.where(busy[:, None], parent, own_b)
    token = torch.where(busy[:, None], token, torch.full_like(token, -1))
    L = s["length"].long()
    s["score_out"].copy_(torch.where(busy[:, None], score, s["score"].double()))
    col = torch.arange(s["tokens"].shape[2], device=DEV)
    kept = s["tokens"].gather(1, parent[:, :, None].expand(-1, -1, s["tokens"].shape[2]))
    kept = torch.where(busy[:, None, None] & (col[None, None] == L[:, None, None]), token[:, :, None].to(torch.int32), kept)
    wide = L + busy.long()
    s["tokens_out"].copy_(torch.where(col[None, None] < wide[:, None, None], kept, s["tokens_out"]))
    s["parent"].copy_(parent)
    s["token"].copy_(token)
    s["length_out"].copy_(wide)
    i, k = torch.nonzero(ends, as_tuple=True)
    f = place[i, k]
    s["done_score"][i, f] = best[i, k].float()
    s["done_length"][i, f] = s["length"][i]
    s["done_tokens"][i, f] = torch.where(col[None] < L[i][:, None], s["tokens"][i, beam[i, k]], s["done_tokens"][i, f])
    s["n_done_out"].copy_(s["n_done"] + ends.sum(1))
    return _beam_outputs(s)


def _reorder(s):
    case = s["case"]
    n, B, page = case["n"], case["beams"], case["page"]
    t = s["table"].long().reshape(n, B, -1)
    L = s["kv_len"].long().reshape(n, B)[:, 0]
    full, rest = L // page, L % page
    par = s["parent"].long()
    src = t.gather(2, full.clamp(max=t.shape[2] - 1)[:, None, None].expand(n, B, 1))[:, :, 0]
    i, b, j = torch.nonzero((torch.arange(page, device=DEV)[None, None] < rest[:, None, None]).expand(n, B, page), as_tuple=True)
    pool = s["pool"].view(torch.uint8) if s["scales"] is not None else s["pool"]
    pool[src[i, b], :, :, j] = pool[src[i, par[i, b]], :, :, j]
    if s["scales"] is not None:
        used = torch.arange(page // case["block"], device=DEV)[None, None] * case["block"] < rest[:, None, None]
        i, b, j = torch.nonzero(used.expand(n, B, -1), as_tuple=True)
        s["scales"][src[i, b], :, :, j] = s["scales"][src[i, par[i, b]], :, :, j]
    moved = t.gather(1, par[:, :, None].expand_as(t))
    keep = torch.arange(t.shape[2], device=DEV)[None, None] >= full[:, None, None]
    s["table"].copy_(torch.where(keep, t, moved).reshape(n * B, -1))
    return _cache_outputs(s) + [s["table"]]


# ------------------------------------------------------------------ the work that cannot be done without
def work(case):
    if case["op"] == "beam":
        n, B, V = case["n"], case["beams"], case["vocab"]
        L = sum(_spread(n, max(1, case["length"] // 2), case["length"]))
        # every logit once; transcripts, scores and choices in and out
        return dict(bytes=n * B * V * 4 + 8 * B * L + 20 * n * B, flops=3 * n * B * V)
    es = {"bf16": 2, "f32": 4, "e4m3": 1}[case.get("dtype", "e4m3")]
    lens = _kv_lens(case)
    hkv, block = case["hkv"], case["block"]
    if case["op"] == "reorder":
        B, page = case["beams"], case["page"]
        part = sum(x % page for x in lens)
        scales = sum(-(-(x % page) // block) for x in lens) if block else 0
        # a partly filled page and a table row of each beam, in and out
        return dict(bytes=2 * B * (2 * hkv * (part * D * es + scales) + 4 * sum(x // page for x in lens)), flops=0)
    c, hq = _chunks(case), case["hq"]
    rows = sum(c)
    if case["op"] == "append":
        rs = 4 if case["dtype"] == "f32" else 2
        touched = sum((x - 1) // block - (x - a) // block + 1 for x, a in zip(lens, c)) if block else 0
        return dict(bytes=rows * D * (2 * hkv * (rs + es) + 2 * hq * rs) + 4 * touched * hkv, flops=3 * rows * D * (hq + hkv))
    pairs = sum(a * x - (a * (a - 1) // 2 if case["causal"] else 0) for a, x in zip(c, lens))
    scales = sum(-(-x // block) for x in lens)
    return dict(bytes=2 * hkv * (sum(lens) * D + scales) + rows * hq * (4 * D + 4), flops=4 * D * pairs * hq)


# ------------------------------------------------------------------ the definition in float64
def exact(case, seed):
    s = prepare(dict(case), seed)
    return {"append": _exact_append, "attend": _exact_attend, "beam": _exact_beam, "reorder": _exact_reorder}[s["op"]](s)


def _turned(x, pos, s):
    """Rows x [rows, heads, 64] as complex numbers times e^(i angle)."""
    case = s["case"]
    y = x.double().clone()
    if case["rotate"] == "none":
        return y
    h = case["dims"] // 2
    w = torch.polar(torch.ones(len(pos), h, dtype=torch.float64, device=DEV), pos.double()[:, None] * s["inv"])[:, None]
    pairs = y[..., : 2 * h].unflatten(-1, (h, 2) if case["rotate"] == "adjacent" else (2, h))
    if case["rotate"] == "halves":
        pairs = pairs.transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
    y[..., : 2 * h] = (z if case["rotate"] == "adjacent" else z.transpose(-1, -2)).flatten(-2)
    return y


def _e4m3(x):
    """x (float64, at most 448 in size) at the nearest e4m3 value, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _powers():
    return torch.tensor([2.0 ** k for k in range(-127, 128)], dtype=torch.float64, device=DEV)


def _exact_append(s):
    case = s["case"]
    power = _powers()
    page, block = case["page"], case["block"]
    cu, lens = s["cu_q"].tolist(), s["kv_len"].tolist()
    pool = s["pool"].double()
    scale = None if not block else power[s["scales"].long()]
    q_out = s["q_out"].double()
    for i, L in enumerate(lens):
        a, e = cu[i], cu[i + 1]
        first = L - (e - a)
        at = torch.arange(first, L, device=DEV)
        pos = at if s["pos"] is None else s["pos"][a:e]
        q_out[a:e] = _turned(s["q"][a:e], pos, s)
        new = torch.stack([_turned(s["k"][a:e], pos, s), s["v"][a:e].double()], 1)
        tab = s["table"][i].long()
        if not block:
            pool[tab[at // page], :, :, at % page] = new
            continue
        for b in range(first // block, (L - 1) // block + 1):
            lo, hi = max(first, b * block), min(L, (b + 1) * block)
            pg, t0 = int(tab[b * block // page]), b * block % page
            x = new[lo - first: hi - first]                    # [rows, 2, heads, 64]
            m = x.abs().amax((0, 3))
            need = power[(m[..., None] > E4M3_MAX * power).sum(-1).clamp(max=254)]
            was = scale[pg, :, :, t0 // block].clone()
            f = need if lo == b * block else torch.maximum(was, need)
            if lo > b * block:
                older = pool[pg, :, :, t0: lo - b * block + t0]
                older.copy_(_e4m3(older * (was / f)[..., None, None]))
            scale[pg, :, :, t0 // block] = f
            pool[pg, :, :, lo - b * block + t0: hi - b * block + t0] = _e4m3(x.permute(1, 2, 0, 3) / f[..., None, None])
    return [pool, scale, q_out]


def _exact_attend(s):
    case = s["case"]
    G, page, block = case["hq"] // case["hkv"], case["page"], case["block"]
    out, lse, power = s["out"].double(), s["lse"].double(), _powers()
    cu, lens = s["cu_q"].tolist(), s["kv_len"].tolist()
    for i, L in enumerate(lens):
        a, e = cu[i], cu[i + 1]
        pages = s["table"][i, : -(-L // page)].long()
        codes = s["pool"].view(torch.uint8)[pages].view(torch.float8_e4m3fn)       # [P, 2, Hkv, page, D]
        size = power[s["scales"][pages].long()].repeat_interleave(block, 3)
        last = L - (e - a) + torch.arange(e - a, device=DEV) if case["causal"] else torch.full((e - a,), L - 1, device=DEV)
        for h in range(case["hkv"]):
            k, v = ((codes[:, w, h].double() * size[:, w, h, :, None]).reshape(-1, D)[:L] for w in (0, 1))
            for u in range(h * G, (h + 1) * G):
                z = (s["q"][a:e, u].double() @ k.T) / 8.0
                z[torch.arange(L, device=DEV)[None] > last[:, None]] = -math.inf
                norm = torch.logsumexp(z, 1)
                out[a:e, u], lse[a:e, u] = torch.exp(z - norm[:, None]) @ v, norm
    return [out, lse]


def _exact_beam(s):
    case = s["case"]
    B, V, F, T = case["beams"], case["vocab"], case["done"], s["tokens"].shape[2]
    score, done = s["score_out"].double(), s["done_score"].double()
    for i in range(case["n"]):
        L, used = int(s["length"][i]), int(s["n_done"][i])
        s["length_out"][i], s["n_done_out"][i] = L, used
        if used >= F or L >= T:
            score[i] = s["score"][i].double()
            s["parent"][i], s["token"][i] = torch.arange(B, device=DEV), -1
            s["tokens_out"][i, :, :L] = s["tokens"][i, :, :L]
            continue
        near = []                                              # (-score, beam, token) of each beam's best
        for b in range(B):
            z = s["logits"][i, b].double()
            lp = z - z.max() - torch.log(torch.exp(z - z.max()).sum())
            order = torch.argsort(-lp, stable=True)[: 2 * B]
            near += [(-(float(s["score"][i, b]) + float(x)), b, int(v)) for v, x in zip(order.tolist(), lp[order].tolist())
                     if x > -math.inf]
        live = 0
        for c, b, v in sorted(near):
            if v == s["eos"]:
                if used < F:
                    done[i, used], s["done_length"][i, used] = -c, L
                    s["done_tokens"][i, used, :L] = s["tokens"][i, b, :L]
                    used += 1
                continue
            s["parent"][i, live], s["token"][i, live], score[i, live] = b, v, -c
            s["tokens_out"][i, live, :L] = s["tokens"][i, b, :L]
            s["tokens_out"][i, live, L] = v
            live += 1
            if live == B:
                break
        for b in range(live, B):
            s["parent"][i, b], s["token"][i, b], score[i, b] = b, -1, -math.inf
            s["tokens_out"][i, b, :L] = s["tokens"][i, b, :L]
            s["tokens_out"][i, b, L] = -1
        s["length_out"][i], s["n_done_out"][i] = L + 1, used
    return [None, None, score, None, None, None, done, None, None]


def _exact_reorder(s):
    case = s["case"]
    B, page, block = case["beams"], case["page"], case["block"]
    scale = None if not block else _powers()[s["scales"].long()]
    pool = s["pool"].double()
    for i in range(case["n"]):
        L = int(s["kv_len"][i * B])
        full, rest = L // page, L % page
        par = s["parent"][i].long()
        old = s["table"][i * B: (i + 1) * B].long()
        if rest:
            at = old[:, full]
            pool[at, :, :, :rest] = pool[at[par], :, :, :rest]
            if block:
                scale[at, :, :, : -(-rest // block)] = scale[at[par], :, :, : -(-rest // block)]
    return [pool, scale, None]
