"""Plain 64-bit forms of the scored decode, of the weights it accumulates and
of the eviction, and small helpers to call the library."""
import math

import numpy as np
import torch

import quantized_kv_cache_04_gb300 as tq

D = 128
# lse: the project's bar for the decode (natural log units)
LSE_ABS = 1e-4


def sequence_kv(orc, preset, cache, bt_row, n, bs, signs, c32):
    """K and V of tokens 0..n-1 of one sequence, float64 (n, Hk, D), from an AoS cache."""
    Hk = cache.shape[2]
    k, v = np.zeros((n, Hk, D)), np.zeros((n, Hk, D))
    for t in range(n):
        page, off = bt_row[t // bs], t % bs
        for h in range(Hk):
            k[t, h], v[t, h] = orc.dequant_slot(preset, cache[page, off, h], signs, c32)
    return k, v


def visible(n, window=0, prefix=0, lo=0):
    """Visible tokens of a sequence of n, as a mask."""
    t = np.arange(n)
    lo = max(lo, 0)
    ok = t >= lo
    if window > 0:
        ok &= (t >= n - window) | (t < lo + prefix)
    return ok


def attend(q, k, v, n, softcap=0.0, slopes=None, window=0, prefix=0, lo=0, scale=D ** -0.5):
    """One sequence: q (Hq, D) float64.  Returns out (Hq, D), lse (Hq,), weights per kv head (Hk, n)."""
    Hq, Hk = q.shape[0], k.shape[1]
    G = Hq // Hk
    out, lse, w = np.zeros((Hq, D)), np.full(Hq, -math.inf), np.zeros((Hk, n))
    ok = visible(n, window, prefix, lo)
    if not ok.any():
        return out, lse, w
    t = np.nonzero(ok)[0]
    for hq in range(Hq):
        h = hq // G
        x = k[t, h] @ q[hq] * scale
        if softcap:
            x = softcap * np.tanh(x / softcap)
        if slopes is not None:
            x = x - float(slopes[hq]) * (n - 1 - t)
        m = x.max()
        e = np.exp(x - m)
        lse[hq] = m + math.log(e.sum())
        p = e / e.sum()
        out[hq] = p @ v[t, h]
        w[h, t] += p
    return out, lse, w


def device_problem(pb, preset, seq_lens, cache=None):
    dev = torch.device("cuda")
    L = tq.tq_get_layout(preset & 0xFF)
    return dict(cache=torch.from_numpy(pb["cache"] if cache is None else cache).to(dev),
                bt=torch.from_numpy(pb["bt"]).to(dev),
                sl=torch.from_numpy(np.asarray(seq_lens, np.int32)).to(dev),
                signs=torch.from_numpy(pb["signs"]).to(dev),
                cent=None if L["key_fp8"] else torch.from_numpy(pb["c32"]).to(dev))


def call(preset, q, d, Hk, bs, max_len, acc=None, num_splits=0, out_dtype=torch.float32, want_lse=True, ws=None,
         stream=None, **mods):
    """decode_attention_scored, or with acc decode_attention_weights; returns (out, lse) on the GPU."""
    B, Hq, _ = q.shape
    dev = d["cache"].device
    out = torch.full((B, Hq, D), 7.0, dtype=out_dtype, device=dev)
    lse = torch.full((B, Hq), 7.0, device=dev) if want_lse else None
    if ws is None:
        # whatever an earlier use left: NaN in every word
        ws = torch.full((tq.scored_workspace_bytes(preset, B, Hq, Hk, max_len, mods.get("window", 0),
                                                   mods.get("prefix", 0), acc is not None, num_splits),), 255,
                        dtype=torch.uint8, device=dev)
    args = (preset, q, d["cache"], d["bt"], d["sl"], max_len, Hk, bs, d["signs"], d["cent"], out, lse, ws)
    if acc is None:
        tq.decode_attention_scored(*args, num_splits=num_splits, stream=stream, **mods)
    else:
        tq.decode_attention_weights(*args, acc, num_splits=num_splits, stream=stream, **mods)
    return out, lse


def select_ref(acc, seq_lens, budget, prefix, recent):
    """keep (B, Hk, budget) and new_lens of float32 sums acc (B, Hk, T)."""
    B, Hk, _ = acc.shape
    keep = np.full((B, Hk, budget), -1, np.int32)
    new = np.minimum(np.maximum(np.asarray(seq_lens), 0), budget).astype(np.int32)
    for b in range(B):
        n = max(int(seq_lens[b]), 0)
        for h in range(Hk):
            if n <= budget:
                keep[b, h, :n] = np.arange(n)
                continue
            x = acc[b, h, :n].astype(np.float64)
            t = np.arange(n)
            always = (t < prefix) | (t >= n - recent)
            rank = np.where(np.isnan(x), 1, 0) + np.where(always, 2, 0)      # NaN above numbers, always-kept above all
            x = np.where(rank > 0, 0.0, x) + 0.0
            order = np.lexsort((t, -x, -rank))
            keep[b, h] = np.sort(order[:budget])
    return keep, new


def compact_ref(cache, bt, keep, seq_lens, bs, acc=None):
    """AoS cache (blocks, bs, Hk, slot) and sums after the move, as new arrays."""
    cache, old = cache.copy(), cache
    acc, old_acc = (None, None) if acc is None else (acc.copy(), acc)
    B, Hk, budget = keep.shape
    for b in range(B):
        n = int(seq_lens[b])
        if n <= budget:
            continue
        for h in range(Hk):
            for i in range(budget):
                t = keep[b, h, i]
                if t < 0 or t >= n:
                    continue
                cache[bt[b, i // bs], i % bs, h] = old[bt[b, t // bs], t % bs, h]
                if acc is not None:
                    acc[b, h, i] = old_acc[b, h, t]
        if acc is not None:
            acc[b, :, budget:n] = 0.0
    return cache, acc
