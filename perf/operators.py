"""Cases of the decode's score modifiers, of the decode that accumulates
attention weights, and of the eviction that goes by them.

Four operators over the compressed paged cache (slot bytes as in include/tq.h):

  decode   one query token per sequence; its scores are capped by a tanh, get
           a bias linear in the distance, and are masked by a window, a prefix
           and the current document's start
  weights  the same, and the softmax weight of every visible token, summed over
           the query heads of its kv head, is added to a running sum per
           (sequence, kv head, token)
  select   which tokens each kv head keeps: the first ones, the newest ones and
           those with the largest running sums; ascending token indices
  compact  the kept slots (and their running sums) move to the front of the
           sequence, in place

`run` computes them in plain torch operations, or, with `own` set, by the
library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
#          fp8 keys, key bits, value bits
PRESETS = {"k8v4": (0, True, 8, 4), "4bit": (1, False, 4, 4), "k3v4": (2, False, 3, 4),
           "3bit": (3, False, 3, 3), "2bit": (4, False, 2, 2)}
SOA_BIT = 0x100


# ------------------------------------------------------------------ cases
def _decode(name, op, preset, B, Hq, Hk, ctx, bs, dtype, **kw):
    c = dict(name=name, op=op, preset=preset, B=B, Hq=Hq, Hk=Hk, ctx=ctx, bs=bs, dtype=dtype, ragged=False,
             soa=False, softcap=0.0, alibi=False, window=0, prefix=0, docs=False)
    c.update(kw)
    return c


def _evict(name, op, preset, B, Hk, ctx, bs, budget, **kw):
    c = dict(name=name, op=op, preset=preset, B=B, Hk=Hk, ctx=ctx, bs=bs, budget=budget, ragged=False,
             soa=False, prefix=4, recent=32)
    c.update(kw)
    return c


def listed():
    return [
        # one request, a short context: the call's latency
        _decode("decode_one_cap", "decode", "4bit", 1, 8, 2, 500, 16, "f16", softcap=50.0),
        # a serving batch of an 8-kv-head model with distance biases
        _decode("decode_batch_alibi", "decode", "k8v4", 32, 32, 8, 8192, 16, "bf16", alibi=True),
        # long prompts, a layer that sees a window and the first tokens only; ragged, groups of 8
        _decode("decode_window_prefix", "decode", "k3v4", 64, 64, 8, 32768, 64, "f16", ragged=True, softcap=30.0,
                window=4096, prefix=64),
        # few very long sequences of several packed documents, SoA blocks
        _decode("decode_long_docs", "decode", "3bit", 4, 32, 8, 131072, 128, "bf16", ragged=True, soa=True,
                softcap=50.0, docs=True),
        # one request whose cache is watched for eviction
        _decode("weights_one", "weights", "k3v4", 1, 32, 8, 2047, 16, "f16"),
        # a ragged serving batch with capped scores
        _decode("weights_batch_cap", "weights", "k8v4", 16, 32, 8, 16384, 32, "bf16", ragged=True, softcap=50.0),
        # long contexts, groups of 8, distance biases
        _decode("weights_long", "weights", "4bit", 8, 64, 8, 65536, 64, "f16", alibi=True),
        # a few short sequences, odd sizes
        _evict("select_short", "select", "k3v4", 3, 5, 1237, 16, 311),
        # a batch of ragged prompts
        _evict("select_batch", "select", "k3v4", 64, 8, 32768, 64, 8192, ragged=True, recent=256),
        # very long contexts, few rows
        _evict("select_long", "select", "3bit", 4, 8, 262144, 128, 32768, recent=1024),
        # a short sequence's cache cut to a third
        _evict("compact_short", "compact", "2bit", 2, 8, 1500, 16, 500),
        # a ragged serving batch cut to a quarter
        _evict("compact_batch", "compact", "k3v4", 32, 8, 16384, 64, 4096, ragged=True, recent=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "weights", "weights", "select", "compact"])
    preset = rng.choice(sorted(PRESETS))
    Hk = rng.choice([1, 2, 3, 4, 5, 8, 8, 8])
    B = _log(rng, 1, 64)
    bs = rng.choice([16, 32, 64, 128])
    ragged = rng.random() < 0.6
    soa = rng.random() < 0.3
    # at most 2^18 tokens of 8 heads in all
    most = max(64, (1 << 18) * 8 // (B * max(Hk, 4)))
    ctx = _log(rng, 33, min(most, 131072))
    if op in ("decode", "weights"):
        c = _decode("", op, preset, B, Hk * rng.choice([1, 2, 4, 5, 8, 12, 16]), Hk, ctx, bs,
                    rng.choice(["f16", "bf16"]), ragged=ragged, soa=soa,
                    softcap=rng.choice([0.0, 20.0, 30.0, 50.0]), alibi=rng.random() < 0.4,
                    docs=rng.random() < 0.25)
        if rng.random() < 0.4:
            c["window"] = _log(rng, 1, ctx)
            c["prefix"] = rng.choice([0, 1, 4, 64])
    else:
        budget = _log(rng, max(2, ctx // 16), max(3, ctx))
        c = _evict("", op, preset, B, Hk, ctx, bs, budget, ragged=ragged, soa=soa,
                   prefix=min(rng.choice([0, 1, 4, 16]), budget // 2),
                   recent=min(rng.choice([0, 1, 32, 256]), budget // 2))
    del c["name"]
    return c


def _lens(c):
    """Sequence lengths: all ctx, or from half of it up, the last of four or more a padding row of no tokens."""
    if not c["ragged"]:
        return [c["ctx"]] * c["B"]
    r = random.Random(c["ctx"] * 131 + c["B"])
    n = [r.randint((c["ctx"] + 1) // 2, c["ctx"]) for _ in range(c["B"])]
    n[0] = c["ctx"]
    if c["B"] >= 4:
        n[-1] = 0
    return n


def _starts(c):
    """First token of each sequence's current document."""
    return [(n * (37 * b % 61)) // 80 if c["docs"] else 0 for b, n in enumerate(_lens(c))]


def _slot(c):
    _, fp8, kb, vb = PRESETS[c["preset"]]
    kd, vd = (D if fp8 else D * kb // 8), D * vb // 8
    return dict(fp8=fp8, kb=kb, vb=vb, kd=kd, vd=vd, mb=4 if fp8 else 6, slot=kd + vd + (4 if fp8 else 6))


def _visible(c):
    """Visible tokens of every sequence, in all."""
    total = 0
    for n, lo in zip(_lens(c), _starts(c)):
        first = lo if c["window"] <= 0 else max(lo, n - c["window"])
        total += max(0, n - first) + min(max(0, first - lo), c["prefix"])
    return total


def work(case):
    c, s = case, _slot(case)
    if c["op"] in ("decode", "weights"):
        n = _visible(c)
        rows = c["B"] * c["Hq"]
        b = n * c["Hk"] * s["slot"] + rows * (4 * D + 4)
        b += 8 * n * c["Hk"] if c["op"] == "weights" else 0
        return {"bytes": b, "flops": 4.0 * D * n * (c["Hq"])}
    n = sum(_lens(c))
    kept = sum(min(m, c["budget"]) for m in _lens(c))
    if c["op"] == "select":
        return {"bytes": 4 * c["Hk"] * (n + kept), "flops": n * c["Hk"]}
    # slots that stay where they are: those of the first tokens and of sequences within the budget
    moved = sum(c["budget"] - c["prefix"] for m in _lens(c) if m > c["budget"])
    tail = sum(m - c["budget"] for m in _lens(c) if m > c["budget"])
    return {"bytes": c["Hk"] * (moved * (2 * s["slot"] + 12) + 4 * tail), "flops": 0}


# ------------------------------------------------------------------ inputs
def _centroids(bits):
    """Lloyd-Max levels of N(0, 1/D), and their midpoints."""
    n = 1 << bits
    c = np.linspace(-2.5, 2.5, n)
    pdf = lambda x: np.exp(-x * x / 2) / math.sqrt(2 * math.pi)  # noqa: E731
    cdf = lambda x: 0.5 * (1 + np.array([math.erf(v / math.sqrt(2)) for v in x]))  # noqa: E731
    for _ in range(300):
        e = np.concatenate([[-12.0], (c[1:] + c[:-1]) / 2, [12.0]])
        c = (pdf(e[:-1]) - pdf(e[1:])) / (cdf(e[1:]) - cdf(e[:-1]))
    c = (c / math.sqrt(D)).astype(np.float32)
    return c, ((c[1:] + c[:-1]) / 2).astype(np.float32)


def _pack(codes, bits):
    """(..., 128) codes to the LSB-first byte stream."""
    if bits == 3:
        g = codes.view(*codes.shape[:-1], D // 8, 8).int()
        w = sum(g[..., i] << (3 * i) for i in range(8))
        return torch.stack([(w >> (8 * i)) & 255 for i in range(3)], -1).to(torch.uint8).flatten(-2)
    per = 8 // bits
    g = codes.view(*codes.shape[:-1], D // per, per).int()
    return sum(g[..., i] << (bits * i) for i in range(per)).to(torch.uint8)


def _half_bytes(x):
    return x.to(torch.float16).unsqueeze(-1).view(torch.uint8)


def _cache(c, gen, nb, cent, mid):
    """Blocks of quantised normal keys (norms around sqrt(128)) and values."""
    s, Hk, bs = _slot(c), c["Hk"], c["bs"]
    cache = torch.empty((nb, bs, Hk, s["slot"]), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 19) // (bs * Hk))
    for b0 in range(0, nb, step):
        shape = (min(step, nb - b0), bs, Hk, D)
        k = torch.randn(shape, generator=gen, device="cuda")
        v = torch.randn(shape, generator=gen, device="cuda")
        lo, hi = v.amin(-1), v.amax(-1)
        levels = (1 << s["vb"]) - 1
        sc, ze = ((hi - lo) / levels).half(), lo.half()
        vc = ((v - ze.float()[..., None]) / sc.float()[..., None]).round().clamp(0, levels)
        meta = [_half_bytes(sc), _half_bytes(ze)]
        if s["fp8"]:
            kd = k.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            n = k.norm(dim=-1, keepdim=True)
            code = torch.bucketize(k / n, mid)
            kd = _pack(code, s["kb"])
            meta = [_half_bytes(n[..., 0] / cent[code].norm(dim=-1))] + meta
        vd = _pack(vc.int(), s["vb"])
        to = cache[b0:b0 + shape[0]]
        if c["soa"]:
            n = shape[0]
            to.view(n, -1).copy_(torch.cat([torch.cat([kd, vd], -1).reshape(n, -1),
                                            torch.cat(meta, -1).reshape(n, -1)], 1))
        elif s["fp8"]:
            to.copy_(torch.cat([kd, vd] + meta, -1))
        else:
            to.copy_(torch.cat([kd, meta[0], vd] + meta[1:], -1))
    return cache


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens = _lens(c)
    st = dict(c=c, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), max_len=c["ctx"])
    B, Hk = c["B"], c["Hk"]
    if c["op"] != "select":
        need = [-(-n // c["bs"]) for n in lens]
        nb = sum(need) + 2
        fp8, kb = _slot(c)["fp8"], _slot(c)["kb"]
        st["cent"] = st["mid"] = None
        if not fp8:
            st["cent"], st["mid"] = (torch.from_numpy(x).cuda() for x in _centroids(kb))
        st["cache"] = _cache(c, gen, nb, st["cent"], st["mid"])
        perm = torch.randperm(nb - 1, generator=gen, device="cuda").int()
        # table entries past a sequence's pages name the last block, which no sequence owns
        table = torch.full((B, max(need) + 1), nb - 1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        st["table"] = table
    # running sums of attention weight: heavy-tailed, the newest tokens' still zero
    width = -(-c["ctx"] // 32) * 32
    if c["op"] != "decode":
        acc = torch.rand((B, Hk, width), generator=gen, device="cuda").clamp_min_(1e-6).log_().neg_().pow_(3)
        acc[torch.rand(acc.shape, generator=gen, device="cuda") < 0.05] = 0.0
        if c["op"] == "weights":
            acc *= 16.0 * (c["Hq"] // Hk) / c["ctx"]     # about a hundred steps' worth
        st["acc"] = acc
    if c["op"] in ("decode", "weights"):
        dt = torch.float16 if c["dtype"] == "f16" else torch.bfloat16
        st["q"] = (torch.randn((B, c["Hq"], D), generator=gen, device="cuda") * 1.5).to(dt)
        st["signs"] = (torch.randint(0, 2, (D,), generator=gen, device="cuda") * 2 - 1).to(torch.int8)
        st["slopes"] = None
        if c["alibi"]:
            i = torch.arange(1, c["Hq"] + 1, device="cuda")
            st["slopes"] = torch.exp2(-8.0 * i / c["Hq"]).float()
        st["starts"] = torch.tensor(_starts(c), dtype=torch.int32, device="cuda") if c["docs"] else None
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((B, c["Hq"]), device="cuda")
    elif c["op"] == "select":
        st["keep"] = torch.empty((B, Hk, c["budget"]), dtype=torch.int32, device="cuda")
        st["new_lens"] = torch.empty((B,), dtype=torch.int32, device="cuda")
    else:
        # any ascending choice of tokens is a selection; here: the first ones, the newest, and random others
        t = torch.arange(width, device="cuda")
        L = st["seq_lens"].view(B, 1, 1)
        r = torch.rand((B, Hk, width), generator=gen, device="cuda")
        r = torch.where((t < c["prefix"]) | (t >= L - c["recent"]), 2.0, r)
        r = torch.where(t < L, r, -1.0)
        top = r.topk(min(c["budget"], width), dim=-1).indices
        n = torch.minimum(L, torch.tensor(c["budget"], device="cuda"))
        top = torch.where(torch.arange(top.shape[-1], device="cuda") < n, top, 1 << 30).sort(-1).values
        top = torch.where(top == 1 << 30, -1, top)
        st["keep"] = torch.full((B, Hk, c["budget"]), -1, dtype=torch.int32, device="cuda")
        st["keep"][..., :top.shape[-1]] = top.int()
    return st


# ------------------------------------------------------------------ the plain forms
def _fields(st):
    """Key data, value data, norm, scale and zero bytes as (block, offset, head, byte) views of the cache."""
    c, s = st["c"], _slot(st["c"])
    cache, Hk, bs = st["cache"], c["Hk"], c["bs"]
    if c["soa"]:
        db, mb, nb = s["kd"] + s["vd"], s["mb"], cache.shape[0]
        blk = bs * Hk * s["slot"]
        data = cache.as_strided((nb, bs, Hk, db), (blk, Hk * db, db, 1))
        meta = cache.as_strided((nb, bs, Hk, mb), (blk, Hk * mb, mb, 1), bs * Hk * db)
        kd, vd = data[..., :s["kd"]], data[..., s["kd"]:]
    else:
        kd = cache[..., :s["kd"]]
        v0 = s["kd"] + (0 if s["fp8"] else 2)
        vd = cache[..., v0:v0 + s["vd"]]
        meta = torch.cat([cache[..., s["kd"]:v0], cache[..., v0 + s["vd"]:]], -1)
    return kd, vd, meta


def _codes(b, bits):
    """Byte stream (..., n) to (..., 128) int32 codes."""
    b = b.int()
    if bits == 3:
        g = b.unflatten(-1, (D // 8, 3))
        w = g[..., 0] | g[..., 1] << 8 | g[..., 2] << 16
        return ((w[..., None] >> (3 * torch.arange(8, device=b.device, dtype=torch.int32))) & 7).flatten(-2)
    sh = bits * torch.arange(8 // bits, device=b.device, dtype=torch.int32)
    return ((b[..., None] >> sh) & ((1 << bits) - 1)).flatten(-2)


def _halves(b):
    return b.contiguous().view(torch.float16).float()


def _hadamard(dtype):
    i = torch.arange(D, device="cuda")
    x = i[:, None] & i[None, :]
    bits = sum((x >> k) & 1 for k in range(7))
    return (1.0 - 2.0 * (bits & 1)).to(dtype) / math.sqrt(D)


def _plain_decode(st):
    c, s = st["c"], _slot(st["c"])
    B, Hq, Hk, bs = c["B"], c["Hq"], c["Hk"], c["bs"]
    G = Hq // Hk
    L = st["seq_lens"].long().view(B, 1)
    lo = torch.zeros_like(L) if st["starts"] is None else st["starts"].long().view(B, 1)
    first = torch.maximum(lo, L - c["window"]) if c["window"] > 0 else lo
    # visible tokens of each row, in order: the prefix, then the window
    n1 = torch.minimum((first - lo).clamp_min(0), torch.tensor(c["prefix"], device="cuda"))
    W = c["ctx"] if c["window"] <= 0 else min(c["ctx"], c["window"] + c["prefix"])
    j = torch.arange(W, device="cuda")
    t = torch.where(j < n1, lo + j, first + j - n1)
    ok = t < L
    t = t.clamp_max(c["ctx"] - 1).clamp_min(0)
    page = torch.gather(st["table"].long(), 1, t // bs)
    kd, vd, meta = _fields(st)
    m = _halves(meta[page, t % bs])
    if s["fp8"]:
        k = kd[page, t % bs].contiguous().view(torch.float8_e4m3fn).float()
        q = st["q"].float()
    else:
        k = st["cent"][_codes(kd[page, t % bs], s["kb"])] * m[..., :1]
        q = (st["q"].float() * st["signs"].float()) @ _hadamard(torch.float32)
    x = torch.einsum("bhgd,bthd->bhgt", q.view(B, Hk, G, D), k) / math.sqrt(D)
    del k
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    if st["slopes"] is not None:
        x = x - st["slopes"].view(1, Hk, G, 1) * (L - 1 - t).float().view(B, 1, 1, W)
    x = torch.where(ok.view(B, 1, 1, W), x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    v = _codes(vd[page, t % bs], s["vb"]).float() * m[..., -2:-1] + m[..., -1:]
    o = torch.einsum("bhgt,bthd->bhgd", p, v) / torch.where(total > 0, total, 1.0)
    del v
    st["out"].copy_(o.view(B, Hq, D))
    lse = (top + torch.log(total))[..., 0]
    st["lse"].copy_(lse.view(B, Hq))
    if c["op"] == "decode":
        return {"out": st["out"], "lse": st["lse"]}
    w = torch.where(total > 0, p / total, 0.0).sum(2)
    st["acc"].scatter_add_(2, t.view(B, 1, W).expand(B, Hk, W), torch.where(ok.view(B, 1, W), w, 0.0))
    return {"out": st["out"], "lse": st["lse"], "acc": st["acc"]}


def _plain_select(st):
    c = st["c"]
    B, budget = c["B"], c["budget"]
    L = st["seq_lens"].view(B, 1, 1)
    width = st["acc"].shape[-1]
    t = torch.arange(width, device="cuda")
    x = torch.where((t < c["prefix"]) | (t >= L - c["recent"]), math.inf, st["acc"])
    x = torch.where(t < L, x, -math.inf)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :budget]
    n = L.clamp_max(budget)
    order = torch.where(torch.arange(order.shape[-1], device="cuda") < n, order, 1 << 30).sort(-1).values
    st["keep"].fill_(-1)
    st["keep"][..., :order.shape[-1]] = torch.where(order == 1 << 30, -1, order).int()
    st["new_lens"].copy_(n.view(B))
    return {"keep": st["keep"], "new_lens": st["new_lens"]}


def _plain_compact(st):
    c, s = st["c"], _slot(st["c"])
    B, Hk, bs, n = c["B"], c["Hk"], c["bs"], min(c["budget"], c["ctx"])
    keep = st["keep"][..., :n].long()
    L = st["seq_lens"].view(B, 1, 1)
    b, h, i = ((keep >= 0) & (keep != torch.arange(n, device="cuda"))).nonzero(as_tuple=True)
    src, table = keep[b, h, i], st["table"].long()
    sp, so, dp, do = table[b, src // bs], src % bs, table[b, i // bs], i % bs
    if c["soa"]:
        db, mb, nb = s["kd"] + s["vd"], s["mb"], st["cache"].shape[0]
        blk = bs * Hk * s["slot"]
        parts = [st["cache"].as_strided((nb, bs, Hk, db), (blk, Hk * db, db, 1)),
                 st["cache"].as_strided((nb, bs, Hk, mb), (blk, Hk * mb, mb, 1), bs * Hk * db)]
    else:
        parts = [st["cache"]]
    for x in parts:
        x[dp, do, h] = x[sp, so, h]
    acc = st["acc"]
    t = torch.arange(acc.shape[-1], device="cuda")
    moved = torch.gather(acc, 2, keep.clamp_min(0))
    acc[..., :n] = torch.where(keep >= 0, moved, acc[..., :n])
    acc.masked_fill_((t >= L.clamp_max(c["budget"])) & (t < L), 0.0)
    return {"cache": st["cache"], "acc": acc}


# ------------------------------------------------------------------ the library's calls
def _own(st):
    import quantized_kv_cache_04_gb300 as tq
    c = st["c"]
    preset = PRESETS[c["preset"]][0] | (SOA_BIT if c["soa"] else 0)
    if c["op"] == "select":
        tq.evict_select(st["acc"], st["seq_lens"], st["max_len"], c["budget"], st["keep"], st["new_lens"],
                        prefix=c["prefix"], recent=c["recent"])
        return {"keep": st["keep"], "new_lens": st["new_lens"]}
    if c["op"] == "compact":
        tq.evict_compact(preset, st["keep"], st["seq_lens"], st["cache"], st["table"], c["Hk"], c["bs"],
                         acc=st["acc"])
        return {"cache": st["cache"], "acc": st["acc"]}
    mods = dict(softcap=c["softcap"], alibi_slopes=st["slopes"], window=c["window"], prefix=c["prefix"],
                doc_start=st["starts"])
    if "ws" not in st:
        # one workspace for every layer, as a program keeps it
        n = tq.scored_workspace_bytes(preset, c["B"], c["Hq"], c["Hk"], st["max_len"], window=c["window"],
                                      prefix=c["prefix"], weights=c["op"] == "weights")
        st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    args = (preset, st["q"], st["cache"], st["table"], st["seq_lens"], st["max_len"], c["Hk"], c["bs"], st["signs"],
            st["cent"], st["out"], st["lse"], st["ws"])
    if c["op"] == "decode":
        tq.decode_attention_scored(*args, **mods)
        return {"out": st["out"], "lse": st["lse"]}
    tq.decode_attention_weights(*args, st["acc"], **mods)
    return {"out": st["out"], "lse": st["lse"], "acc": st["acc"]}


def run(state):
    if own:
        return _own(state)
    op = state["c"]["op"]
    if op == "select":
        return _plain_select(state)
    return _plain_compact(state) if op == "compact" else _plain_decode(state)


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_rows(st, b, slots):
    """Keys and values of `slots` of the cache in 64 bits, decoded code by code: (n, Hk, 128) each."""
    c, s = st["c"], _slot(st["c"])
    bs, Hk, n = c["bs"], c["Hk"], slots.numel()
    flat = st["cache"].reshape(-1)
    blk, off = slots // bs, slots % bs
    rec = off[:, None] * Hk + torch.arange(Hk, device="cuda")
    base = (blk * (bs * Hk * s["slot"]))[:, None]
    if c["soa"]:
        data = base + rec * (s["kd"] + s["vd"])
        meta = base + bs * Hk * (s["kd"] + s["vd"]) + rec * s["mb"]
        value, field = data + s["kd"], [meta + 2 * i for i in range(s["mb"] // 2)]
    else:
        data = base + rec * s["slot"]
        value = data + s["kd"] + (0 if s["fp8"] else 2)
        field = ([] if s["fp8"] else [data + s["kd"]]) + [value + s["vd"], value + s["vd"] + 2]

    def half(at):
        return torch.stack([flat[at], flat[at + 1]], -1).view(torch.float16)[..., 0].double()

    def code(at, bits):
        bit = torch.arange(D, device="cuda") * bits
        here = (at[..., None] + bit // 8)
        low = flat[here].long()
        high = flat[torch.where(bit % 8 + bits > 8, here + 1, here)].long()
        return ((low | high << 8) >> (bit % 8)) & ((1 << bits) - 1)

    v = code(value, s["vb"]).double() * half(field[-2])[..., None] + half(field[-1])[..., None]
    if s["fp8"]:
        k = flat[data[..., None] + torch.arange(D, device="cuda")].view(torch.float8_e4m3fn).double()
    else:
        k = st["cent"].double()[code(data, s["kb"])] * half(field[0])[..., None]
    return k, v


def exact(case, seed):
    c = dict(case)
    if c["op"] == "select":
        return None                      # whole numbers
    st = prepare(case, seed)
    B, Hk = c["B"], c["Hk"]
    if c["op"] == "compact":
        acc = st["acc"].double()
        new = acc.clone()
        for b, n in enumerate(_lens(c)):
            m = min(n, c["budget"])
            new[b, :, m:n] = 0.0
            for h in range(Hk):
                new[b, h, :m] = acc[b, h, st["keep"][b, h, :m].long()]
        return {"cache": None, "acc": new}
    Hq, G = c["Hq"], c["Hq"] // Hk
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    acc = st["acc"].double() if c["op"] == "weights" else None
    q = st["q"].double()
    if not _slot(c)["fp8"]:
        had = torch.ones((1, 1), dtype=torch.float64, device="cuda")
        for _ in range(7):
            had = torch.cat([torch.cat([had, had], 1), torch.cat([had, -had], 1)], 0)
        q = torch.matmul(q * st["signs"].double(), had) / math.sqrt(D)
    for b, (n, lo) in enumerate(zip(_lens(c), _starts(c))):
        t = torch.arange(n, device="cuda")
        see = t >= lo
        if c["window"] > 0:
            see &= (t >= n - c["window"]) | (t < lo + c["prefix"])
        t = t[see]
        if not t.numel():
            continue
        parts = []
        # the keys' pass and the values' pass over pieces of the sequence
        pieces = t.split(1 << 14)
        slots = [st["table"][b, p // c["bs"]].long() * c["bs"] + p % c["bs"] for p in pieces]
        rows = [_exact_rows(st, b, s) for s in slots]
        for p, (k, _) in zip(pieces, rows):
            x = torch.matmul(q[b].view(Hk, G, D), k.permute(1, 2, 0)) * D ** -0.5
            if c["softcap"]:
                x = torch.tanh(x / c["softcap"]) * c["softcap"]
            if c["alibi"]:
                x = x + st["slopes"].double().view(Hk, G, 1) * (p - (n - 1)).double()
            parts.append(x)
        x = torch.cat(parts, -1)
        z = torch.logsumexp(x, -1, keepdim=True)
        w = torch.exp(x - z)
        v = torch.cat([r[1] for r in rows], 0)
        out[b] = torch.matmul(w, v.transpose(0, 1)).reshape(Hq, D)
        lse[b] = z.reshape(Hq)
        if acc is not None:
            acc[b][:, t] += w.sum(1)
        del rows, parts, v
    return {"out": out, "lse": lse} if acc is None else {"out": out, "lse": lse, "acc": acc}
