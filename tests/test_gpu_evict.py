"""Eviction: the selection (whole numbers, equal to a plain sort) and the
in-place move (bytes, equal), and the store - decode - evict - decode chain."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_04_gb300 as tq
from _helpers import aos_to_soa, check_decode, paged_problem, to_f32
from _scored import attend, compact_ref, select_ref, sequence_kv

pytestmark = pytest.mark.gpu


def _select(acc, seq_lens, budget, prefix, recent, max_len=None):
    B, Hk, T = acc.shape
    keep = torch.full((B, Hk, budget), 77, dtype=torch.int32, device="cuda")
    new = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    sl = torch.tensor(list(seq_lens), dtype=torch.int32, device="cuda")
    tq.evict_select(acc, sl, T if max_len is None else max_len, budget, keep, new, prefix=prefix, recent=recent)
    return keep.cpu().numpy(), new.cpu().numpy()


def _sums(rng, kind, shape):
    x = rng.exponential(size=shape).astype(np.float32) ** 3
    if kind == "ties":
        x = np.round(rng.random(shape) * 4).astype(np.float32)
    elif kind == "zeros":
        x[rng.random(shape) < 0.7] = 0.0
        x[rng.random(shape) < 0.2] = -0.0
    elif kind == "special":
        for v, p in ((np.nan, .02), (np.inf, .02), (-np.inf, .02), (-np.nan, .01), (1e-42, .05), (-1e-42, .05)):
            x[rng.random(shape) < p] = v
        x[rng.random(shape) < 0.3] *= -1
    elif kind == "equal":
        x[:] = 0.25
    elif kind == "close":
        x = (np.float32(1.0) + rng.integers(0, 300, shape) * np.float32(2.0 ** -23)).astype(np.float32)
    return x


@pytest.mark.parametrize("kind", ["plain", "ties", "zeros", "special", "equal", "close"])
@pytest.mark.parametrize("T,budget,prefix,recent", [
    (1, 1, 0, 0), (2, 1, 0, 1), (33, 32, 4, 28), (130, 7, 3, 4), (1237, 311, 4, 32), (4096, 1, 0, 0),
    (4097, 4096, 1, 0), (20000, 5000, 16, 200), (70001, 1025, 0, 1024)])
def test_select(kind, T, budget, prefix, recent):
    rng = np.random.default_rng(T + budget)
    B, Hk = (2, 3) if T < 5000 else (1, 2)
    acc = _sums(rng, kind, (B, Hk, T))
    lens = [T, max(0, T - 5)][:B]
    keep, new = _select(torch.from_numpy(acc).cuda(), lens, budget, prefix, recent)
    rk, rn = select_ref(acc, lens, budget, prefix, recent)
    assert np.array_equal(new, rn)
    assert np.array_equal(keep, rk)


def test_select_lengths_and_strides():
    rng = np.random.default_rng(1)
    B, Hk, T = 7, 5, 900
    lens = [900, 0, 1, 299, 300, 301, -4]
    base = torch.from_numpy(_sums(rng, "ties", (B, Hk + 3, T + 41))).cuda()
    for acc in (base[:, 1:Hk + 1, 7:T + 7], base.transpose(0, 1)[1:Hk + 1, :, 3:T + 3].transpose(0, 1),
                base[:, 1:Hk + 1, 7:T + 7].transpose(0, 1).contiguous().transpose(0, 1)):
        keep, new = _select(acc, lens, 300, 10, 20)
        rk, rn = select_ref(acc.cpu().numpy(), lens, 300, 10, 20)
        assert np.array_equal(new, rn) and np.array_equal(keep, rk)


def test_select_many_rows():
    """More rows than the GPU holds at once."""
    rng = np.random.default_rng(2)
    acc = _sums(rng, "zeros", (70, 16, 513))
    lens = [int(x) for x in rng.integers(0, 514, 70)]
    keep, new = _select(torch.from_numpy(acc).cuda(), lens, 100, 2, 30)
    rk, rn = select_ref(acc, lens, 100, 2, 30)
    assert np.array_equal(new, rn) and np.array_equal(keep, rk)


@pytest.mark.parametrize("T", [100000, 262144, 1100003])
def test_select_long(T):
    """A row over 8 CTAs, and ones beyond the keys, or the bits, that 8 CTAs hold in shared memory."""
    rng = np.random.default_rng(T)
    acc = _sums(rng, "plain", (1, 2, T))
    acc[:, 1] = np.round(acc[:, 1] * 8) / 8
    keep, new = _select(torch.from_numpy(acc).cuda(), [T], 32768, 4, 1024)
    rk, rn = select_ref(acc, [T], 32768, 4, 1024)
    assert np.array_equal(new, rn) and np.array_equal(keep, rk)


def test_select_longer_than_max_seq_len():
    rng = np.random.default_rng(4)
    acc = _sums(rng, "plain", (3, 2, 500))
    keep, new = _select(torch.from_numpy(acc).cuda(), [500, 400, 90], 100, 0, 0, max_len=400)
    rk, rn = select_ref(acc, [500, 400, 90], 100, 0, 0)
    assert (keep[0] == -1).all() and new[0] == 500
    assert np.array_equal(keep[1:], rk[1:]) and np.array_equal(new[1:], rn[1:])


def _random_keep(rng, B, Hk, lens, budget):
    keep = np.full((B, Hk, budget), -1, np.int32)
    for b, n in enumerate(lens):
        for h in range(Hk):
            m = min(n, budget)
            keep[b, h, :m] = np.sort(rng.permutation(n)[:m])
    return keep


def _paged(rng, preset, lens, Hk, bs):
    """A random cache (any bytes are a record), and a table of distinct pages with two spare blocks."""
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 2
    slot = tq.tq_get_layout(preset)["slot_size_aligned"]
    cache = rng.integers(0, 256, (nb, bs, Hk, slot), dtype=np.uint8)
    bt = np.full((len(lens), max(need) + 1), nb - 1, np.int32)
    perm, at = rng.permutation(nb - 2), 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n]
        at += n
    return cache, bt


@pytest.mark.parametrize("preset", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("soa", [False, True])
@pytest.mark.parametrize("Hk,bs,lens,budget", [
    (8, 16, [300, 100, 50, 0], 100), (1, 32, [97], 1), (3, 64, [200, 333], 199), (5, 128, [129, 40], 64),
    (2, 16, [1200, 700], 650), (16, 16, [40], 39)])
def test_compact(orc, preset, soa, Hk, bs, lens, budget):
    rng = np.random.default_rng(preset + 10 * Hk + budget)
    B, T = len(lens), max(lens) + 3
    cache, bt = _paged(rng, preset, lens, Hk, bs)
    keep = _random_keep(rng, B, Hk, lens, budget)
    acc0 = rng.random((B, Hk, T)).astype(np.float32)
    want, wacc = compact_ref(cache, bt, keep, lens, bs, acc0)
    if soa:
        # records only: bytes of a block that no record covers do not exist (data + meta = slot)
        cache, want = (aos_to_soa(orc, preset, x) for x in (cache, want))
    for with_acc in (True, False):
        c, a = torch.from_numpy(cache).cuda(), torch.from_numpy(acc0).cuda()
        tq.evict_compact(preset | (tq.TQ_LAYOUT_SOA if soa else 0), torch.from_numpy(keep).cuda(),
                         torch.tensor(lens, dtype=torch.int32, device="cuda"), c, torch.from_numpy(bt).cuda(), Hk, bs,
                         acc=a if with_acc else None)
        assert np.array_equal(c.cpu().numpy(), want)
        assert np.array_equal(a.cpu().numpy(), wacc if with_acc else acc0)


@pytest.mark.parametrize("budget", [1, 3000, 9000])
def test_compact_few_rows(budget):
    """One row over many chunks: the moved slots overlap their sources everywhere."""
    rng = np.random.default_rng(budget)
    cache, bt = _paged(rng, 4, [9500], 1, 16)
    keep = _random_keep(rng, 1, 1, [9500], budget)
    want, _ = compact_ref(cache, bt, keep, [9500], 16)
    c = torch.from_numpy(cache).cuda()
    tq.evict_compact(4, torch.from_numpy(keep).cuda(), torch.tensor([9500], dtype=torch.int32, device="cuda"), c,
                     torch.from_numpy(bt).cuda(), 1, 16)
    assert np.array_equal(c.cpu().numpy(), want)


def test_compact_refuses_entries_outside():
    """Entries outside the sequence and pages outside the cache move nothing; the other rows are exact."""
    rng = np.random.default_rng(8)
    lens, Hk, bs, budget = [120, 120, 90], 2, 16, 40
    cache, bt = _paged(rng, 2, lens, Hk, bs)
    keep = _random_keep(rng, 3, Hk, lens, budget)
    keep[0, 0, 39], keep[0, 1, 38], keep[0, 1, 39] = 120, -1, 2 ** 31 - 1
    bad = bt.copy()
    gone = keep[1, 0, 39] // bs                  # a source page of sequence 1, past the destinations
    if gone < 3:
        keep[1, :, 39], gone = 119, 7
    bad[1, gone] = cache.shape[0] + 3
    want, _ = compact_ref(cache, bt, keep, lens, bs)
    for h in range(Hk):                          # slots from the missing page stay as they were
        for i in range(budget):
            if keep[1, h, i] // bs == gone:
                at = (bt[1, i // bs], i % bs, h)
                want[at] = cache[at]
    big = torch.zeros((cache.shape[0] + 8,) + cache.shape[1:], dtype=torch.uint8, device="cuda")
    big[:cache.shape[0]] = torch.from_numpy(cache).cuda()
    c = big[:cache.shape[0]]
    tq.evict_compact(2, torch.from_numpy(keep).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), c,
                     torch.from_numpy(bad).cuda(), Hk, bs)
    assert np.array_equal(c.cpu().numpy(), want)
    assert (big[cache.shape[0]:] == 0).all()


def test_compact_past_4_gib():
    """Slots whose byte offsets pass 32 bits."""
    Hk, bs, n, budget = 8, 128, 640, 200
    slot = tq.tq_get_layout(0)["slot_size_aligned"]
    nb = (9 << 29) // (bs * Hk * slot) + 1       # about 4.5 GiB
    cache = torch.zeros((nb, bs, Hk, slot), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(9)
    pages = np.array([nb - 1, 3, nb - 2, nb // 2, nb - 5], np.int32)
    data = rng.integers(0, 256, (5, bs, Hk, slot), dtype=np.uint8)
    for p, x in zip(pages, data):
        cache[int(p)] = torch.from_numpy(x).cuda()
    keep = _random_keep(rng, 1, Hk, [n], budget)
    want, _ = compact_ref(data, np.arange(5)[None], keep, [n], bs)
    tq.evict_compact(0, torch.from_numpy(keep).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), cache,
                     torch.from_numpy(pages[None]).cuda(), Hk, bs)
    for p, x in zip(pages, want):
        assert np.array_equal(cache[int(p)].cpu().numpy(), x)
    assert int(cache[10:nb // 2].max()) == 0


@pytest.mark.parametrize("preset,Hk,G", [(0, 8, 4), (2, 8, 8), (3, 3, 2), (1, 2, 16)])
def test_decode_evict_decode(orc, preset, Hk, G):
    """Decode steps that accumulate weights, an eviction by them, and a decode of what is left, as one run; the
    graph of the same run gives the same cache."""
    rng = np.random.default_rng(17 + preset)
    bs, lens, budget, steps = 16, [200, 90, 333], 96, 3
    pb = paged_problem(orc, preset, lens, Hk, bs, rng)
    B, Hq, T = len(lens), Hk * G, 352
    dev = torch.device("cuda")
    c = tq.TQCache(preset, pb["cache"].shape[0], bs, Hk)
    bt, sl = torch.from_numpy(pb["bt"]).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    q = torch.from_numpy(rng.normal(size=(steps + 1, B, Hq, 128)) * 2).half().to(dev)
    out, lse = torch.empty((B, Hq, 128), device=dev), torch.empty((B, Hq), device=dev)
    acc = torch.zeros((B, Hk, T), device=dev)
    ws = c.scored_workspace(B, Hq, T, weights=True)
    keep = torch.empty((B, Hk, budget), dtype=torch.int32, device=dev)
    new = torch.empty((B,), dtype=torch.int32, device=dev)

    def run():
        c.cache.copy_(torch.from_numpy(pb["cache"]), non_blocking=False) if not torch.cuda.is_current_stream_capturing() \
            else c.cache.copy_(saved)
        acc.zero_()
        for s in range(steps):
            c.decode_weights(q[s], bt, sl, T, out, lse, ws, acc, softcap=30.0)
        sums = acc.clone()
        c.evict(acc, bt, sl, T, budget, prefix=2, recent=16, keep=keep, new_lens=new)
        c.decode_scored(q[steps], bt, new, T, out, lse, ws, softcap=30.0)
        return sums

    saved = torch.from_numpy(pb["cache"]).to(dev)
    sums = run()
    torch.cuda.synchronize()
    rk, rn = select_ref(sums.cpu().numpy(), lens, budget, 2, 16)
    assert np.array_equal(keep.cpu().numpy(), rk) and np.array_equal(new.cpu().numpy(), rn)
    want, wacc = compact_ref(pb["cache"], pb["bt"], rk, lens, bs, sums.cpu().numpy())
    assert np.array_equal(c.cache.cpu().numpy(), want) and np.array_equal(acc.cpu().numpy(), wacc)
    o, l = np.zeros((B, Hq, 128)), np.zeros((B, Hq))
    for b in range(B):
        k, v = sequence_kv(orc, preset, want, pb["bt"][b], int(rn[b]), bs, pb["signs"], pb["c32"])
        o[b], l[b], _ = attend(to_f32(q[steps, b]).astype(np.float64), k, v, int(rn[b]), softcap=30.0)
    check_decode(out.cpu().numpy(), lse.cpu().numpy(), o, l, "after the eviction")
    first = (c.cache.clone(), acc.clone(), out.clone(), lse.clone(), keep.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, x in zip(first, (c.cache, acc, out, lse, keep)):
        assert torch.equal(a, x)


def test_evict_of_the_cache_object():
    """TQCache.evict makes its own index and length buffers, and asks for them with a stream of the caller's."""
    rng = np.random.default_rng(21)
    lens, Hk, bs, budget = [100, 30], 2, 16, 40
    cache, bt = _paged(rng, 2, lens, Hk, bs)
    c = tq.TQCache("turboquant_k3v4_nc", cache.shape[0], bs, Hk)
    c.cache.copy_(torch.from_numpy(cache))
    acc = rng.random((2, Hk, 112)).astype(np.float32)
    accd, sl = torch.from_numpy(acc).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        c.evict(accd, torch.from_numpy(bt).cuda(), sl, 112, budget, stream=torch.cuda.Stream())
    keep, new = c.evict(accd, torch.from_numpy(bt).cuda(), sl, 112, budget, prefix=3, recent=5)
    rk, rn = select_ref(acc, lens, budget, 3, 5)
    want, wacc = compact_ref(cache, bt, rk, lens, bs, acc)
    assert np.array_equal(keep.cpu().numpy(), rk) and np.array_equal(new.cpu().numpy(), rn)
    assert np.array_equal(c.cache.cpu().numpy(), want) and np.array_equal(accd.cpu().numpy(), wacc)
    # a sequence longer than max_seq_len is left alone, slots, sums and length
    c.cache.copy_(torch.from_numpy(cache))
    accd = torch.from_numpy(acc).cuda()
    keep, new = c.evict(accd, torch.from_numpy(bt).cuda(), sl, 99, 20)
    rk, _ = select_ref(acc, [0, 30], 20, 0, 0)
    want, wacc = compact_ref(cache, bt, rk, [0, 30], bs, acc)
    assert new.tolist() == [100, 20] and (keep[0] == -1).all()
    assert np.array_equal(c.cache.cpu().numpy(), want) and np.array_equal(accd.cpu().numpy(), wacc)
    # the lengths in place of the old ones are refused: they are read while the new ones are written
    with pytest.raises(tq.TQError):
        c.evict(accd, torch.from_numpy(bt).cuda(), sl, 112, 20, keep=keep, new_lens=sl)
