"""Decode with score modifiers, and the attention weights it accumulates,
against plain attention in 64 bits over the oracle's dequantised cache.

Tolerances.  The output and lse bars are the decode's (2e-3, 1e-4).  A weight
exp(x - lse) inherits the error of x and of lse, each within the lse bar, so
it is within 2 * 1e-4 of itself; the running sum adds one rounding of half a
step (2^-24) of the sum per query head and one for the addition."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_04_gb300 as tq
from _helpers import aos_to_soa, check_decode, expected_kernel_kind, paged_problem, to_f32
from _scored import LSE_ABS, attend, call, device_problem, sequence_kv, visible

pytestmark = pytest.mark.gpu
PRESETS = [0, 1, 2, 3, 4]


def _slopes(Hq):
    return (2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)).astype(np.float32)


# (G, Hk, bs, seq_lens, splits)
SHAPES = {
    "g4": (4, 8, 16, [300, 0, 33, 1], 0),
    "g8": (8, 2, 64, [257, 129, 64], 3),
    "g16": (16, 4, 32, [190, 31], 2),
    "g5": (5, 4, 128, [140, 96], 0),
    "g1": (1, 8, 32, [222, 17], 5),
    # rows of 2 mod 4 bytes (Lloyd-Max presets), SoA metadata of 6 and 18 bytes a token
    "odd3": (3, 3, 16, [211, 45, 0], 4),
    "odd1": (4, 1, 32, [130, 64], 2),
    "odd5": (8, 5, 16, [100, 37], 2),
    # rows above what the tensor-core kernels take (CUDA cores, but for 2-bit slots and FP8 keys)
    "wide": (2, 16, 16, [75, 40], 2),
    "wide17": (9, 17, 32, [50, 33], 2),
}
MODS = {
    "cap": dict(softcap=5.0),
    "alibi": dict(alibi=True),
    "window": dict(window=40),
    "window1": dict(window=1),
    "window_prefix": dict(window=33, prefix=5),
    "prefix_meets_window": dict(window=100, prefix=90, softcap=30.0),
    "docs": dict(docs=True, softcap=20.0),
    "all": dict(softcap=8.0, alibi=True, window=50, prefix=7, docs=True),
    "none": dict(),
}


def _mods(m, Hq, seq_lens):
    """(reference keywords per sequence, device keywords)."""
    dev, ref = {}, [dict() for _ in seq_lens]
    for k in ("softcap", "window", "prefix"):
        if k in m:
            dev[k] = m[k]
            for r in ref:
                r[k] = m[k]
    if m.get("alibi"):
        s = _slopes(Hq)
        dev["alibi_slopes"] = torch.from_numpy(s).cuda()
        for r in ref:
            r["slopes"] = s
    if m.get("docs"):
        # in the middle of a tile, at its edge, past the end, negative
        lo = [(3 * n // 5, 32, n + 5, -3)[b % 4] for b, n in enumerate(seq_lens)]
        dev["doc_start"] = torch.tensor(lo, dtype=torch.int32, device="cuda")
        for r, x in zip(ref, lo):
            r["lo"] = x
    return ref, dev


def _reference(orc, preset, pb, q, seq_lens, bs, ref):
    B, Hq, _ = q.shape
    Hk = pb["cache"].shape[2]
    qf = to_f32(q).astype(np.float64)
    out, lse, ws = np.zeros((B, Hq, 128)), np.zeros((B, Hq)), []
    for b, n in enumerate(seq_lens):
        k, v = sequence_kv(orc, preset, pb["cache"], pb["bt"][b], n, bs, pb["signs"], pb["c32"])
        out[b], lse[b], w = attend(qf[b], k, v, n, **ref[b])
        ws.append(w)
    return out, lse, ws


def _check_acc(acc, acc0, ws, seq_lens, G):
    for b, n in enumerate(seq_lens):
        got, was, w = acc[b].astype(np.float64), acc0[b].astype(np.float64), ws[b]
        exact = was[:, :n] + w
        bound = 2 * LSE_ABS * w + (G + 1) * 2.0 ** -24 * np.abs(exact) + 1e-30
        assert np.all(np.abs(got[:, :n] - exact) <= bound), b
        hidden = w == 0
        assert np.array_equal(got[:, :n][hidden], was[:, :n][hidden])
        assert np.array_equal(acc[b][:, n:], acc0[b][:, n:])       # behind the sequence


@pytest.mark.parametrize("mods", sorted(MODS))
@pytest.mark.parametrize("shape", sorted(SHAPES))
@pytest.mark.parametrize("preset", PRESETS)
def test_scored_and_weights(orc, preset, shape, mods):
    G, Hk, bs, seq_lens, S = SHAPES[shape]
    Hq, B = G * Hk, len(seq_lens)
    assert tq.tq_decode_kernel_kind(preset, 128, Hq, Hk) == expected_kernel_kind(preset, G, Hk)
    rng = np.random.default_rng(31 * preset + 7 * sorted(SHAPES).index(shape) + 1000 * sorted(MODS).index(mods))
    dt = torch.bfloat16 if (preset + len(mods)) % 2 else torch.float16
    pb = paged_problem(orc, preset, seq_lens, Hk, bs, rng, dtype="float16" if dt == torch.float16 else "bfloat16")
    q = torch.from_numpy(rng.normal(size=(B, Hq, 128)) * 2.0).to(dt)
    ref, dev = _mods(MODS[mods], Hq, seq_lens)
    o, l, ws = _reference(orc, preset, pb, q, seq_lens, bs, ref)
    d, qd = device_problem(pb, preset, seq_lens), q.cuda()
    max_len = max(seq_lens)
    go, gl = call(preset, qd, d, Hk, bs, max_len, num_splits=S, **dev)
    check_decode(go.cpu().numpy(), gl.cpu().numpy(), o, l, "scored")
    acc0 = rng.exponential(size=(B, Hk, max_len + 13)).astype(np.float32)
    acc = torch.from_numpy(acc0).cuda()
    go, gl = call(preset, qd, d, Hk, bs, max_len, acc=acc, num_splits=S, **dev)
    check_decode(go.cpu().numpy(), gl.cpu().numpy(), o, l, "weights")
    _check_acc(acc.cpu().numpy(), acc0, ws, seq_lens, G)
    # the same from an SoA cache
    soa = device_problem(pb, preset, seq_lens, aos_to_soa(orc, preset, pb["cache"]))
    acc2 = torch.from_numpy(acc0).cuda()
    go, gl = call(preset | tq.TQ_LAYOUT_SOA, qd, soa, Hk, bs, max_len, acc=acc2, num_splits=S, **dev)
    check_decode(go.cpu().numpy(), gl.cpu().numpy(), o, l, "weights, SoA")
    _check_acc(acc2.cpu().numpy(), acc0, ws, seq_lens, G)


def _simple(orc, preset=2, G=4, Hk=8, bs=16, seq_lens=(200, 77), seed=5, dtype=torch.float16, qscale=2.0):
    rng = np.random.default_rng(seed)
    pb = paged_problem(orc, preset, list(seq_lens), Hk, bs, rng)
    q = torch.from_numpy(rng.normal(size=(len(seq_lens), G * Hk, 128)) * qscale).to(dtype)
    return pb, q, device_problem(pb, preset, list(seq_lens))


@pytest.mark.parametrize("preset", PRESETS)
def test_no_modifier_is_the_plain_decode(orc, preset):
    pb, q, d = _simple(orc, preset)
    S = 2
    a, la = call(preset, q.cuda(), d, 8, 16, 200, num_splits=S)
    b, lb = torch.empty_like(a), torch.empty_like(la)
    ws = torch.empty(tq.tq_decode_workspace_bytes(2, 32, S), dtype=torch.uint8, device="cuda")
    tq.decode_attention(preset, q.cuda(), d["cache"], d["bt"], d["sl"], 200, 8, 16, d["signs"], d["cent"], b, lb, ws,
                        num_splits=S)
    assert torch.equal(a, b) and torch.equal(la, lb)
    # a window of the whole sequence hides nothing
    c, lc = call(preset, q.cuda(), d, 8, 16, 200, num_splits=S, window=200)
    assert (a - c).abs().max() <= 2e-5 and (la - lc).abs().max() <= LSE_ABS


@pytest.mark.parametrize("preset,Hk,soa", [(2, 3, False), (4, 1, False), (3, 5, True), (0, 3, True)])
def test_no_modifier_where_the_plain_decode_is_on_cuda_cores(orc, preset, Hk, soa):
    seq_lens = [200, 77, 0]
    assert tq.tq_decode_kernel_kind(preset | (tq.TQ_LAYOUT_SOA if soa else 0), 128, 4 * Hk, Hk) == 0
    pb, q, d = _simple(orc, preset, 4, Hk, 16, seq_lens)
    if soa:
        d = device_problem(pb, preset, seq_lens, aos_to_soa(orc, preset, pb["cache"]))
        preset |= tq.TQ_LAYOUT_SOA
    out, lse = call(preset, q.cuda(), d, Hk, 16, 200)
    want, wl = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(tq.tq_decode_workspace_bytes(3, 4 * Hk, 2), dtype=torch.uint8, device="cuda")
    tq.decode_attention(preset, q.cuda(), d["cache"], d["bt"], d["sl"], 200, Hk, 16, d["signs"], d["cent"], want, wl, ws,
                        num_splits=2)
    assert (out - want).abs().max() <= 2e-5
    assert torch.equal(lse.isneginf(), wl.isneginf()) and (lse - wl).nan_to_num(0.0).abs().max() <= LSE_ABS


@pytest.mark.parametrize("preset,Hk", [(0, 8), (2, 8), (2, 3), (4, 1)])
@pytest.mark.parametrize("bs", [16, 64])
def test_pages_of_hidden_tokens_are_never_looked_up(orc, preset, Hk, bs):
    seq_lens = [500, 333]
    pb, q, d = _simple(orc, preset, 4, Hk, bs, seq_lens)
    mods = dict(window=70, prefix=9)
    clean = call(preset, q.cuda(), d, Hk, bs, 500, num_splits=3, **mods)
    stale = pb["bt"].copy()
    for b, n in enumerate(seq_lens):
        ok = visible(n, 70, 9)
        for p in range(-(-n // bs)):
            if not ok[p * bs:min(n, p * bs + bs)].any():
                stale[b, p] = (-1, pb["cache"].shape[0], 2 ** 31 - 1)[p % 3]
    assert (stale != pb["bt"]).any()
    d2 = dict(d, bt=torch.from_numpy(stale).cuda())
    got = call(preset, q.cuda(), d2, Hk, bs, 500, num_splits=3, **mods)
    assert torch.equal(clean[0], got[0]) and torch.equal(clean[1], got[1])
    acc = [torch.zeros((2, Hk, 500), device="cuda") for _ in range(2)]
    call(preset, q.cuda(), d, Hk, bs, 500, acc=acc[0], num_splits=3, **mods)
    call(preset, q.cuda(), d2, Hk, bs, 500, acc=acc[1], num_splits=3, **mods)
    assert torch.equal(acc[0], acc[1])


@pytest.mark.parametrize("preset,Hk", [(0, 8), (2, 8), (2, 3)])
def test_visible_page_outside_the_cache(orc, preset, Hk):
    """The entry points into the same allocation: a view of a larger buffer is the cache."""
    seq_lens = [300, 200, 90]
    pb, q, d = _simple(orc, preset, 4, Hk, 16, seq_lens)
    nb = pb["cache"].shape[0]
    big = torch.zeros((nb + 4,) + pb["cache"].shape[1:], dtype=torch.uint8, device="cuda")
    big[:nb] = d["cache"]
    d = dict(d, cache=big[:nb])
    acc0 = torch.zeros((3, Hk, 300), device="cuda")
    clean_acc = acc0.clone()
    clean = call(preset, q.cuda(), d, Hk, 16, 300, acc=clean_acc, num_splits=2, window=64, prefix=8)
    bad = pb["bt"].copy()
    bad[1, (200 - 10) // 16] = nb + 1
    got_acc = acc0.clone()
    got = call(preset, q.cuda(), dict(d, bt=torch.from_numpy(bad).cuda()), Hk, 16, 300, acc=got_acc, num_splits=2,
               window=64, prefix=8)
    for b in (0, 2):
        assert torch.equal(clean[0][b], got[0][b]) and torch.equal(clean[1][b], got[1][b])
        assert torch.equal(clean_acc[b], got_acc[b])
    assert got[0][1].isnan().all() and got[1][1].isnan().all()
    see = torch.from_numpy(visible(200, 64, 8)).cuda()
    assert got_acc[1][:, :200][:, see].isnan().all()
    assert (got_acc[1][:, :200][:, ~see] == 0).all() and (got_acc[1][:, 200:] == 0).all()


@pytest.mark.parametrize("preset,Hk", [(3, 8), (3, 3)])
def test_longer_than_max_seq_len(orc, preset, Hk):
    pb, q, d = _simple(orc, preset, 4, Hk, 16, [200, 77])
    acc = torch.ones((2, Hk, 100), device="cuda")
    out, lse = call(preset, q.cuda(), d, Hk, 16, 100, acc=acc, num_splits=2)
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert (acc[0] == 1).all()
    want, wl = call(preset, q.cuda(), d, Hk, 16, 200, num_splits=2)
    assert (out[1] - want[1]).abs().max() <= 2e-5 and (lse[1] - wl[1]).abs().max() <= LSE_ABS
    assert (acc[1, :, 77:] == 1).all() and (acc[1, :, :77] > 1).any()


@pytest.mark.parametrize("preset,Hk", [(1, 8), (4, 3)])
def test_sums_of_other_orders_and_types(orc, preset, Hk):
    """Strided and head-major sums, no lse, 16-bit outputs, one query of a shared table row per batch row."""
    pb, q, d = _simple(orc, preset, 4, Hk, 16, [200, 200])
    d["bt"] = d["bt"][:1].expand(2, -1)                     # stride 0
    d["sl"] = torch.tensor([200, 150], dtype=torch.int32, device="cuda")
    base = torch.zeros((2, Hk, 200), device="cuda")
    o, l = call(preset, q.cuda(), d, Hk, 16, 200, acc=base, softcap=9.0)
    G = 4
    assert (base.double().sum(-1) - G).abs().max() <= G * 2 * LSE_ABS
    wide = torch.zeros((2, Hk + 2, 333), device="cuda")
    call(preset, q.cuda(), d, Hk, 16, 200, acc=wide[:, 1:Hk + 1, 5:300], softcap=9.0, want_lse=False)
    assert torch.equal(wide[:, 1:Hk + 1, 5:205], base)
    wide[:, 1:Hk + 1, 5:205] = 0
    assert (wide == 0).all()
    hm = torch.zeros((Hk, 2, 200), device="cuda")
    o16, _ = call(preset, q.cuda(), d, Hk, 16, 200, acc=hm.transpose(0, 1), softcap=9.0, out_dtype=torch.float16)
    assert torch.equal(hm.transpose(0, 1), base)
    assert ((o16.float() - o).abs() <= o.abs() * 2.0 ** -11 + 2e-5).all()


@pytest.mark.parametrize("softcap", [0.0, 1e-3, 50.0])
def test_extreme_scores(orc, softcap):
    """Scores of thousands: a cap bounds them, without one the softmax is one token's."""
    for preset in PRESETS:
        pb, q, d = _simple(orc, preset, 8, 2, 16, [150], qscale=300.0)
        o, l, ws = _reference(orc, preset, pb, q, [150], 16, [dict(softcap=softcap)])
        acc = torch.zeros((1, 2, 150), device="cuda")
        out, lse = call(preset, q.cuda(), d, 2, 16, 150, acc=acc, softcap=softcap)
        # scores of size s carry an error of 2^-20 s (fp32 sums of 128 products of split operands)
        s = 300.0 * 12 * 12 / 128 ** 0.5 if softcap == 0 else softcap
        tol = 2.0 ** -18 * s + LSE_ABS
        assert np.abs(lse.cpu().numpy() - l).max() <= tol
        assert torch.isfinite(out).all() and torch.isfinite(acc).all()
        assert np.abs(acc.cpu().numpy()[0] - ws[0]).max() <= 8 * 2 * tol


def test_other_stream_and_graphs(orc):
    """Two captured graphs with a workspace each, replayed in turn; a call on another stream."""
    pb, q, d = _simple(orc, 2, 4, 8, 16, [400, 123])
    q = q.cuda()
    mods = dict(softcap=20.0, window=100, prefix=4)
    want_acc = torch.zeros((2, 8, 400), device="cuda")
    want, wl = call(2, q, d, 8, 16, 400, acc=want_acc, **mods)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    acc = torch.zeros_like(want_acc)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        out, lse = call(2, q, d, 8, 16, 400, acc=acc, stream=s, **mods)
        torch.cuda.synchronize()
    assert torch.equal(acc, want_acc) and torch.equal(out, want) and torch.equal(lse, wl)
    n = tq.scored_workspace_bytes(2, 2, 32, 8, 400, 100, 4, True)
    graphs = []
    for _ in range(2):
        a, ws = torch.zeros_like(want_acc), torch.empty(n, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(want), torch.empty_like(wl)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tq.decode_attention_weights(2, q, d["cache"], d["bt"], d["sl"], 400, 8, 16, d["signs"], d["cent"], out,
                                        lse, ws, a, **mods)
        graphs.append((g, a, out, lse))
    for _ in range(3):
        for g, *_ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for _, a, out, lse in graphs:
        assert torch.equal(out, want) and torch.equal(lse, wl)
        three = (want_acc + want_acc) + want_acc
        assert torch.equal(a, three)


@pytest.mark.parametrize("preset,Hk", [(0, 8), (2, 8), (2, 3), (1, 16)])
def test_cache_past_4_gib(preset, Hk):
    """Pages whose byte offsets pass 32 bits give what the same pages give in a small cache."""
    bs, n = 128, 600
    slot = tq.tq_get_layout(preset)["slot_size_aligned"]
    nb = (9 << 29) // (bs * Hk * slot) + 1           # about 4.5 GiB
    rng = np.random.default_rng(preset)
    c = tq.TQCache(preset, 5, bs, Hk)
    kv = torch.from_numpy(rng.normal(size=(2, 640, Hk, 128))).half().cuda()
    c.store(kv[0], kv[1], torch.arange(640, device="cuda"))
    big = torch.empty((nb,) + c.cache.shape[1:], dtype=torch.uint8, device="cuda")
    pages = [nb - 1, 0, nb - 2, nb // 2, nb - 7]
    for i, p in enumerate(pages):
        big[p] = c.cache[i]
    q = torch.from_numpy(rng.normal(size=(1, 4 * Hk, 128))).half().cuda()
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    d = dict(sl=sl, signs=c.signs, cent=c.centroids)
    got = []
    for cache, table in ((c.cache, [0, 1, 2, 3, 4]), (big, pages)):
        acc = torch.zeros((1, Hk, n), device="cuda")
        bt = torch.tensor([table], dtype=torch.int32, device="cuda")
        got.append((*call(preset, q, dict(d, cache=cache, bt=bt), Hk, bs, n, acc=acc, softcap=20.0), acc))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_two_streams_at_once(orc):
    """Calls that overlap on the GPU, each with a workspace and sums of its own, over one cache."""
    pb, q, d = _simple(orc, 1, 8, 8, 32, [900, 411, 0])
    q = q.cuda()
    kws = [dict(softcap=15.0), dict(window=333, prefix=2)]
    want = []
    for kw in kws:
        a = torch.zeros((3, 8, 900), device="cuda")
        want.append((*call(1, q, d, 8, 32, 900, acc=a, **kw), a))
    streams = [torch.cuda.Stream() for _ in kws]
    n = max(tq.scored_workspace_bytes(1, 3, 64, 8, 900, kw.get("window", 0), kw.get("prefix", 0), True) for kw in kws)
    bufs = [(torch.empty_like(want[0][0]), torch.empty_like(want[0][1]), torch.empty(n, dtype=torch.uint8, device="cuda"),
             torch.zeros_like(want[0][2])) for _ in kws]
    torch.cuda.synchronize()
    for rep in range(20):
        for s, kw, (out, lse, ws, acc) in zip(streams, kws, bufs):
            with torch.cuda.stream(s):
                acc.zero_()
            tq.decode_attention_weights(1, q, d["cache"], d["bt"], d["sl"], 900, 8, 32, d["signs"], d["cent"], out, lse,
                                        ws, acc, stream=s, **kw)
    torch.cuda.synchronize()
    for (o, l, a), (out, lse, _, acc) in zip(want, bufs):
        assert torch.equal(o, out) and torch.equal(l, lse) and torch.equal(a, acc)


def test_many_splits_and_long_context(orc):
    """A long sequence over many splits: every split count gives the same attention."""
    rng = np.random.default_rng(3)
    preset, Hk, G, bs, n = 3, 2, 4, 64, 5000
    nb = -(-n // bs) + 1
    c = tq.TQCache(preset, nb, bs, Hk)
    K = torch.from_numpy(rng.normal(size=(n, Hk, 128))).half().cuda()
    V = torch.from_numpy(rng.normal(size=(n, Hk, 128))).half().cuda()
    bt = torch.from_numpy(rng.permutation(nb - 1).astype(np.int32)).cuda().view(1, -1)
    t = torch.arange(n, device="cuda")
    c.store(K, V, bt[0].long()[t // bs] * bs + t % bs)
    ko, vo = torch.empty((n, Hk, 128), device="cuda"), torch.empty((n, Hk, 128), device="cuda")
    c.dequant(bt[0].long()[t // bs] * bs + t % bs, ko, vo)
    q = torch.from_numpy(rng.normal(size=(1, Hk * G, 128))).half()
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    for kw in (dict(softcap=10.0), dict(window=3001, prefix=100)):
        o, l, w = attend(to_f32(q[0]).astype(np.float64), ko.double().cpu().numpy(), vo.double().cpu().numpy(), n, **kw)
        for S in (0, 1, 7, 64, 256):
            acc = torch.zeros((1, Hk, n), device="cuda")
            ws = c.scored_workspace(1, Hk * G, n, S, kw.get("window", 0), kw.get("prefix", 0), True)
            out = torch.empty((1, Hk * G, 128), device="cuda")
            lse = torch.empty((1, Hk * G), device="cuda")
            c.decode_weights(q.cuda(), bt, sl, n, out, lse, ws, acc, num_splits=S, **kw)
            check_decode(out.cpu().numpy(), lse.cpu().numpy(), o[None], l[None], f"{kw} S={S}")
            _check_acc(acc.cpu().numpy(), np.zeros((1, Hk, n), np.float32), [w], [n], G)


@pytest.mark.parametrize("preset,Hk", [(2, 8), (0, 2), (2, 1)])
@pytest.mark.parametrize("B", [33, 40, 512, 520])
def test_large_ragged_batches(preset, Hk, B):
    """The plan of the splits for batches of more sequences than a warp has lanes, and than it plans for: every
    row equals the same sequence decoded alone, within the decode's bars."""
    gen = torch.Generator(device="cuda").manual_seed(B)
    rng = np.random.default_rng(B)
    G, bs = 4, 16
    lens = rng.integers(0, 200, B)
    lens[:4] = [700, 0, 1, 200]
    need = -(-lens // bs)
    c = tq.TQCache(preset, int(need.sum()) + 1, bs, Hk)
    bt = torch.full((B, int(need.max())), int(need.sum()), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = torch.arange(at, at + int(n), device="cuda")
        at += int(n)
    slots = torch.arange(int(need.sum()) * bs, device="cuda")
    kv = torch.randn((2, slots.numel(), Hk, 128), generator=gen, device="cuda").half()
    c.store(kv[0], kv[1], slots)
    q = torch.randn((B, Hk * G, 128), generator=gen, device="cuda").half()
    sl = torch.from_numpy(lens.astype(np.int32)).cuda()
    d = dict(cache=c.cache, bt=bt, sl=sl, signs=c.signs, cent=c.centroids)
    kw = dict(softcap=20.0, window=150, prefix=5)
    for S in (0, 1, 3):
        acc = torch.zeros((B, Hk, 704), device="cuda")
        out, lse = call(preset, q, d, Hk, bs, 700, acc=acc, num_splits=S, **kw)
        for b in (0, 1, 2, 3, B // 2, B - 1):
            one = dict(d, bt=bt[b:b + 1], sl=sl[b:b + 1])
            acc1 = torch.zeros((1, Hk, 704), device="cuda")
            o1, l1 = call(preset, q[b:b + 1].contiguous(), one, Hk, bs, 700, acc=acc1, num_splits=1, **kw)
            assert (out[b] - o1[0]).abs().max() <= 2e-5
            assert torch.equal(lse[b].isneginf(), l1[0].isneginf())
            assert (lse[b] - l1[0]).nan_to_num(0.0).abs().max() <= LSE_ABS
            assert ((acc[b] - acc1[0]).abs() <= 2 * LSE_ABS * acc1[0]).all()
        # every sequence with tokens weighs G in all
        total = acc.double().sum(-1)
        assert (total[sl > 0] - G).abs().max() <= G * 2 * LSE_ABS and (total[sl == 0] == 0).all()


@pytest.mark.parametrize("preset", [0, 2, 4])
@pytest.mark.parametrize("G", [4, 8])
def test_long_flat_softmax_keeps_fp32_accuracy(preset, G):
    """Averages of 40000 values: the two parts of a value sum (codes times scales, and zeros) cancel to a few
    thousandths of their size, and the error must not grow with the sum.

    The bound.  Per 32-token tile the accumulators give up m = (half the values' range) * (the tile's weight), then
    at most four MMAs add terms that come back to it; each rounds towards zero, by at most 2^-23 of an
    intermediate no larger than m.  Over all tiles: 4 * 2^-23 = 2^-21 of the weighted mean of half the range, per
    output element.  Scores (of size < 8) are off by up to 2^-20 of their size, weights by 8e-6, independently
    from token to token, their average by less than 1e-5 of itself.  (Sums that are not kept about the middle code
    round by 2^-23 of everything summed so far, some hundred tiles: a factor of ten and more above the bound.)"""
    n, Hk, bs = 40000, 8, 64
    gen = torch.Generator(device="cuda").manual_seed(preset)
    nb = -(-n // bs)
    c = tq.TQCache(preset, nb, bs, Hk)
    t = torch.arange(n, device="cuda")
    k, v = torch.empty((n, Hk, 128), device="cuda"), torch.empty((n, Hk, 128), device="cuda")
    c.store(torch.randn((n, Hk, 128), generator=gen, device="cuda").half(),
            torch.randn((n, Hk, 128), generator=gen, device="cuda").half(), t)
    c.dequant(t, k, v)
    q = torch.randn((1, Hk * G, 128), generator=gen, device="cuda").half()
    x = torch.einsum("hgd,nhd->hgn", q.double().view(Hk, G, 128), k.double()) * 128 ** -0.5
    w = torch.softmax(50.0 * torch.tanh(x / 50.0), -1)
    want = torch.einsum("hgn,nhd->hgd", w, v.double()).reshape(1, Hk * G, 128)
    out, lse = torch.empty((1, Hk * G, 128), device="cuda"), torch.empty((1, Hk * G), device="cuda")
    bt = torch.arange(nb, dtype=torch.int32, device="cuda").view(1, -1)
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    for S in (0, 3):
        c.decode_scored(q, bt, sl, n, out, lse, c.scored_workspace(1, Hk * G, n, S), num_splits=S, softcap=50.0)
        half = ((v.amax(-1) - v.amin(-1)) / 2).double()                  # (n, Hk)
        half = (w * half.t()[:, None]).sum(-1).max()
        bound = 2.0 ** -21 * half * want.numel() ** 0.5 + 1e-5 * want.norm()
        assert ((out.double() - want).norm() <= bound).item()
