"""Eviction by accumulated weight and filling with positions, bit for bit against
the oracle, and a decode loop that runs them with attention."""
import numpy as np
import pytest
import torch

from decode_kv_cache_eviction_b200 import Batch, Engine, Offsets, RkvError
from decode_kv_cache_eviction_b200 import _binding as B
from oracle import rkv_oracle as ora

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ODD = [1, 0, 2, 31, 32, 33, 127, 511, 512, 513, 1025, 5000]


def offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def evict(lengths, acc, budget, w=8, sinks=0, live=None, pos=None, budgets=None, with_idx=True,
          alias=False):
    off = offsets(lengths)
    U, T = len(lengths), int(off[-1])
    eng = Engine(1, w, U, max(T, 1), redundancy="closed")
    b = Batch(None, None, None, off, device=DEV)
    a = dev(acc.astype(np.float32))
    lv = None if live is None else dev(live)
    keep = lv if alias else torch.full((T,), 9, dtype=torch.uint8, device=DEV)
    free = torch.full((T,), -7, dtype=torch.int32, device=DEV)
    nf = torch.full((U,), -7, dtype=torch.int32, device=DEV)
    out = a if alias else torch.full((T,), float("nan"), device=DEV)
    W = budget + sinks + w
    idx = torch.full((U, W), -7, dtype=torch.int32, device=DEV) if with_idx else None
    nk = torch.full((U,), -7, dtype=torch.int32, device=DEV) if with_idx else None
    eng.evict_accumulated(b, a, budget, keep, free, nf, live=lv,
                          pos=None if pos is None else dev(pos.astype(np.int32)),
                          budgets=None if budgets is None else dev(budgets.astype(np.int32)),
                          sinks=sinks, acc_out=out, idx=idx, n_kept=nk)
    eng.check_status()
    keep, free, nf, out = (t.cpu().numpy() for t in (keep, free, nf, out))
    for u in range(U):
        s = slice(int(off[u]), int(off[u + 1]))
        N = lengths[u]
        lu = np.ones(N) if live is None else live[s]
        pu = np.arange(N) if pos is None else pos[s]
        bu = budget if budgets is None else min(max(int(budgets[u]), 0), budget)
        acc32 = acc[s].astype(np.float32)
        kept = ora.evict_accumulated(acc32, pu, lu, w, bu, sinks)
        k_o, f_o = ora.evict_in_place(N, kept)
        assert np.array_equal(keep[s], k_o.astype(np.uint8)), u
        assert nf[u] == len(f_o), u
        assert np.array_equal(free[s][:len(f_o)], f_o) and np.all(free[s][len(f_o):] == -1), u
        want = np.where(k_o, acc32, np.float32(0))
        assert np.array_equal(out[s].view(np.int32), want.view(np.int32)), u
        if with_idx:
            row = idx[u].cpu().numpy()
            assert int(nk[u]) == len(kept) and np.array_equal(row[:len(kept)], kept), u
            assert np.all(row[len(kept):] == -1), u


@pytest.mark.parametrize("budget", [0, 1, 37, 512, 4990, 100000])
@pytest.mark.parametrize("positions", [False, True])
def test_evict_matches_oracle(budget, positions):
    rng = np.random.default_rng(budget)
    T = sum(ODD)
    pos = np.concatenate([rng.permutation(3 * n)[:n] for n in ODD]) if positions else None
    for live in (None, (rng.random(T) < 0.6).astype(np.uint8)):
        evict(ODD, rng.random(T) ** 4, budget, w=8, sinks=4, live=live, pos=pos)
        evict(ODD, rng.random(T) ** 4, budget, w=1, sinks=0, live=live, pos=pos, with_idx=False)


def test_evict_equal_weights_and_special_values():
    rng = np.random.default_rng(1)
    T = sum(ODD)
    evict(ODD, np.zeros(T), 100)
    evict(ODD, rng.integers(0, 3, T).astype(float), 100, sinks=2)
    a = rng.standard_normal(T)
    a[rng.random(T) < 0.2] = np.nan
    a[rng.random(T) < 0.2] = 0.0
    a[rng.random(T) < 0.2] = -0.0
    a[rng.random(T) < 0.05] = np.inf
    a[rng.random(T) < 0.05] = -np.inf
    for budget in (0, 1, 50, 300, 2500):
        evict(ODD, a, budget, sinks=3)
    evict(ODD, np.full(T, np.nan), 20)
    # keys that agree in their upper bits
    evict(ODD, 1.0 + np.arange(T) * 2.0 ** -23, 333)


def test_evict_per_unit_budgets_dead_units_and_aliases():
    rng = np.random.default_rng(2)
    T = sum(ODD)
    live = (rng.random(T) < 0.5).astype(np.uint8)
    off = offsets(ODD)
    live[off[7]:off[8]] = 0
    budgets = np.array([5, 0, -3, 7, 1000000, 1, 60, 3, 100, 0, 250, 2000])
    evict(ODD, rng.random(T), 2000, live=live, budgets=budgets, sinks=4)
    evict(ODD, rng.random(T), 2000, live=live, budgets=budgets, sinks=4, alias=True)


@pytest.mark.parametrize("n", [8192, 32768, 131072])
def test_evict_long_units(n):
    rng = np.random.default_rng(n)
    lengths = [n, n - 1, 17]
    T = sum(lengths)
    evict(lengths, np.exp(2 * rng.standard_normal(T)), n // 8, sinks=4,
          live=(rng.random(T) < 0.7).astype(np.uint8),
          pos=np.concatenate([rng.permutation(2 * k)[:k] for k in lengths]))
    evict(lengths, np.round(np.exp(rng.standard_normal(T)), 1), n // 3)


def test_evict_many_units():
    rng = np.random.default_rng(3)
    lengths = rng.integers(1, 300, 3000).tolist()
    evict(lengths, rng.random(sum(lengths)), 64, w=4, sinks=2)


def test_kept_rows_feed_compaction():
    lengths = [700, 90, 20]
    off = offsets(lengths)
    rng = np.random.default_rng(4)
    T = sum(lengths)
    K = dev(rng.standard_normal((T, 128)).astype(np.float32)).to(torch.bfloat16)
    V = K * 2
    b = Batch(K, V, None, off)
    eng = Engine(4, 8, 3, T, redundancy="closed")
    budget, sinks = 64, 4
    acc = dev(rng.random(T).astype(np.float32))
    keep, free, nf = eng.alloc_in_place(b)
    idx, nk, Ko, Vo = eng.alloc_outputs(b, budget + sinks)
    eng.evict_accumulated(b, acc, budget, keep, free, nf, sinks=sinks, idx=idx, n_kept=nk)
    eng.compact(b, idx, nk, budget + sinks, Ko, Vo)
    eng.check_status()
    for u in range(3):
        n = int(nk[u])
        rows = idx[u, :n].long() + int(off[u])
        assert n == min(lengths[u], budget + sinks + 8)
        assert torch.equal(Ko[u, :n], K[rows]) and torch.equal(Vo[u, :n], V[rows])


def test_more_rows_than_idx_holds_is_reported():
    eng = Engine(1, 2, 1, 100, redundancy="closed")
    b = Batch(None, None, None, [0, 100], device=DEV)
    keep = torch.zeros(100, dtype=torch.uint8, device=DEV)
    free, nf = torch.zeros(100, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    idx, nk = torch.full((1, 7), -7, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    pos = torch.full((100,), 5, dtype=torch.int32, device=DEV)        # every row the newest
    eng.evict_accumulated(b, torch.rand(100, device=DEV), 5, keep, free, nf, pos=pos, idx=idx, n_kept=nk)
    with pytest.raises(RkvError) as ei:
        eng.check_status()
    assert ei.value.code == B.RKV_ERR_DEVICE
    assert idx[0].tolist() == list(range(7)) and int(nk) == 7 and bool(keep.all()) and int(nf) == 0


def _fill_state(lengths, seed, free_frac=0.5):
    rng = np.random.default_rng(seed)
    off = offsets(lengths)
    T = int(off[-1])
    K = dev(rng.standard_normal((T, 128)).astype(np.float32)).to(torch.bfloat16)
    V = dev(rng.standard_normal((T, 128)).astype(np.float32)).to(torch.bfloat16)
    keep = (rng.random(T) >= free_frac).astype(np.uint8)
    free, nf = np.full(T, -1, np.int32), np.zeros(len(lengths), np.int32)
    for u in range(len(lengths)):
        f = np.flatnonzero(keep[off[u]:off[u + 1]] == 0)
        free[off[u]:off[u] + len(f)] = f
        nf[u] = len(f)
    return rng, off, K, V, keep, free, nf


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("seed", [0, 1])
def test_fill_with_positions(in_place, seed):
    lengths = [1, 0, 2, 33, 700, 300, 2000, 257]
    rng, off, K, V, keep, free, nf = _fill_state(lengths, seed)
    U, T = len(lengths), int(off[-1])
    counts = [int(rng.integers(0, n + 1)) if u % 3 else int(n) * (seed == 0) for u, n in enumerate(nf)]
    new = offsets(counts)
    n = int(new[-1])
    Kn, Vn = (dev(rng.standard_normal((n, 128)).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
    pos, pos_new = rng.integers(0, 99, T).astype(np.int32), rng.integers(100, 999, n).astype(np.int32)
    acc = rng.random(T).astype(np.float32)
    Kw, Vw = K.clone(), V.clone()
    kw, pw, aw, fw, nw = keep.copy(), pos.copy(), acc.copy(), np.full(T, -1, np.int32), nf.copy()
    for u in range(U):
        a, f, x = int(off[u]), free[off[u]:off[u] + nf[u]], slice(int(new[u]), int(new[u + 1]))
        to = a + f[:counts[u]].astype(np.int64)
        Kw[dev(to)], Vw[dev(to)] = Kn[x], Vn[x]
        kw[to], pw[to], aw[to] = 1, pos_new[x], 0
        left = f[counts[u]:]
        fw[a:a + len(left)] = left
        nw[u] = len(left)
    eng = Engine(1, 4, U, T, redundancy="closed")
    d = dict(keep=dev(keep), free=dev(free), nf=dev(nf), pos=dev(pos), acc=dev(acc))
    fo = None if in_place else torch.full((T,), -7, dtype=torch.int32, device=DEV)
    no = None if in_place else torch.full((U,), -7, dtype=torch.int32, device=DEV)
    eng.fill_slots_ex(Batch(K, V, None, off), Offsets(new, DEV), Kn, Vn, d["keep"], d["free"], d["nf"],
                      pos=d["pos"], pos_new=dev(pos_new), acc=d["acc"], free_out=fo, n_free_out=no)
    eng.check_status()
    assert torch.equal(K, Kw) and torch.equal(V, Vw)
    assert np.array_equal(d["keep"].cpu().numpy(), kw) and np.array_equal(d["pos"].cpu().numpy(), pw)
    assert np.array_equal(d["acc"].cpu().numpy(), aw)
    assert np.array_equal((d["free"] if in_place else fo).cpu().numpy(), fw)
    assert np.array_equal((d["nf"] if in_place else no).cpu().numpy(), nw)
    if not in_place:      # the input list is untouched
        assert np.array_equal(d["free"].cpu().numpy(), free) and np.array_equal(d["nf"].cpu().numpy(), nf)


@pytest.mark.parametrize("units,each", [(700, 1), (700, 100), (60, 150), (60, 3)])
@pytest.mark.parametrize("in_place", [True, False])
def test_fill_many_units(units, each, in_place):
    """More units than the grid, and fewer than SMs with more rows than a pass."""
    rng = np.random.default_rng(units + each)
    n, free_rows = 200, 170
    T = units * n
    slots = np.stack([np.sort(rng.permutation(n)[:free_rows]) for _ in range(units)])
    free = np.full((units, n), -1, np.int32)
    free[:, :free_rows] = slots
    keep = np.ones((units, n), np.uint8)
    np.put_along_axis(keep, slots, 0, axis=1)
    K = torch.zeros((T, 128), dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    Kn, Vn = (torch.randn((units * each, 128), device=DEV).to(torch.bfloat16) for _ in range(2))
    to = dev((slots[:, :each] + n * np.arange(units)[:, None]).reshape(-1).astype(np.int64))
    Kw, Vw = K.clone(), V.clone()
    Kw[to], Vw[to] = Kn, Vn
    np.put_along_axis(keep_want := keep.copy(), slots[:, :each], 1, axis=1)
    left = np.full((units, n), -1, np.int32)
    left[:, :free_rows - each] = slots[:, each:]
    k, f = dev(keep.reshape(-1)), dev(free.reshape(-1))
    c = torch.full((units,), free_rows, dtype=torch.int32, device=DEV)
    fo, no = (f, c) if in_place else (torch.full_like(f, -7), torch.full_like(c, -7))
    eng = Engine(1, 4, units, T, redundancy="closed")
    kw = {} if in_place else dict(free_out=fo, n_free_out=no)
    eng.fill_slots_ex(Batch(K, V, None, n * np.arange(units + 1)), Offsets(each * np.arange(units + 1), DEV),
                      Kn, Vn, k, f, c, **kw)
    eng.check_status()
    assert torch.equal(K, Kw) and torch.equal(V, Vw)
    assert np.array_equal(k.cpu().numpy(), keep_want.reshape(-1))
    assert np.array_equal(fo.cpu().numpy(), left.reshape(-1)) and bool((no == free_rows - each).all())


def test_fill_more_tokens_than_free_slots():
    rng, off, K, V, keep, free, nf = _fill_state([100, 50], 3, 0.2)
    eng = Engine(1, 4, 2, 150, redundancy="closed")
    Kn = torch.randn((90, 128), device=DEV).to(torch.bfloat16)
    k, f, c = dev(keep), dev(free), dev(nf)
    eng.fill_slots_ex(Batch(K, V, None, off), Offsets([0, 60, 90], DEV), Kn, Kn, k, f, c)
    with pytest.raises(RkvError) as ei:
        eng.check_status()
    assert ei.value.code == B.RKV_ERR_DEVICE
    assert bool(k.all()) and c.tolist() == [0, 0] and bool((f == -1).all())


def test_refusals():
    eng = Engine(1, 4, 2, 150, redundancy="closed")
    b = Batch(None, None, None, [0, 100, 150], device=DEV)
    acc = torch.rand(150, device=DEV)
    keep = torch.full((150,), 9, dtype=torch.uint8, device=DEV)
    free, nf = torch.zeros(150, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    for kw in (dict(budget=-1), dict(sinks=-1), dict(idx=torch.zeros((2, 14), dtype=torch.int32, device=DEV))):
        with pytest.raises(RkvError) as ei:
            eng.evict_accumulated(b, acc, kw.pop("budget", 10), keep, free, nf, **kw)
        assert ei.value.code == B.RKV_ERR_INVALID_ARG
    for kw in (dict(acc=acc[:100]), dict(acc=acc.double()), dict(live=keep.bool()),
               dict(idx=torch.zeros((2, 13), dtype=torch.int32, device=DEV), n_kept=nf)):
        with pytest.raises(ValueError):
            eng.evict_accumulated(b, kw.pop("acc", acc), 10, keep, free, nf, **kw)
    big = Engine(1, 4, 1, 150, redundancy="closed")
    with pytest.raises(RkvError):
        big.evict_accumulated(b, acc, 10, keep, free, nf)
    K = torch.zeros((150, 128), dtype=torch.bfloat16, device=DEV)
    kv = Batch(K, K.clone(), None, [0, 100, 150])
    with pytest.raises(ValueError):                       # offsets of three units
        eng.fill_slots_ex(kv, Offsets([0, 1, 2, 3], DEV), K[:3], K[:3], keep, free, nf)
    with pytest.raises(ValueError):                       # positions without new ones
        eng.fill_slots_ex(kv, Offsets([0, 1, 2], DEV), K[:2], K[:2], keep, free, nf, pos=free)
    with pytest.raises(ValueError):
        eng.fill_slots_ex(kv, Offsets([0, 1, 2], DEV), K[:2], K[:2], keep, free, nf, free_out=free)
    with pytest.raises(RkvError) as ei:                   # decreasing offsets
        eng.fill_slots_ex(kv, Offsets([0, 3, 2], DEV), K[:2], K[:2], keep, free, nf)
    assert ei.value.code == B.RKV_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((keep == 9).all())


def test_refusals_of_sizes():
    eng = Engine(1, 4, 2, 150, redundancy="closed")
    b = Batch(None, None, None, [0, 100, 150], device=DEV)
    acc, keep = torch.rand(150, device=DEV), torch.full((150,), 9, dtype=torch.uint8, device=DEV)
    free, nf = torch.zeros(150, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    for budget, sinks in ((2**32, 0), (10, 2**31)):
        with pytest.raises(ValueError):
            eng.evict_accumulated(b, acc, budget, keep, free, nf, sinks=sinks)
    eng.evict_accumulated(b, acc, 2**31 - 1, keep, free, nf, sinks=2**31 - 1)    # the largest: all stay
    torch.cuda.synchronize()
    assert bool((keep == 1).all()) and bool((nf == 0).all())


def test_decode_loop():
    """A decode loop on caches of fixed size: each step places one token in every
    unit, attends with accumulated weights, and evicts by them when a unit is
    full; against the same loop in float64."""
    G, w, cap, budget, sinks, U = 4, 4, 64, 40, 2, 3
    rng = np.random.default_rng(9)
    T = U * cap
    off = offsets([cap] * U)
    K, V = (torch.zeros((T, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    b = Batch(K, V, None, off)
    eng = Engine(G, w, U, T, redundancy="closed")
    keep = torch.zeros(T, dtype=torch.uint8, device=DEV)
    pos = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    acc = torch.zeros(T, device=DEV)
    free = torch.arange(cap, dtype=torch.int32, device=DEV).repeat(U)
    nf = torch.full((U,), cap, dtype=torch.int32, device=DEV)
    one = Offsets(np.arange(U + 1), DEV)
    out = torch.empty((U, G, 1, 128), dtype=torch.bfloat16, device=DEV)
    h = [dict(k=np.zeros((cap, 128)), v=np.zeros((cap, 128)), live=np.zeros(cap, bool),
              pos=np.full(cap, -1), acc=np.zeros(cap), free=list(range(cap))) for _ in range(U)]
    evictions = 0
    for step in range(150):
        kn, vn = (dev(rng.standard_normal((U, 128)).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
        q = dev(rng.standard_normal((U, G, 1, 128)).astype(np.float32) * 2).to(torch.bfloat16)
        at = torch.full((U,), step, dtype=torch.int32, device=DEV)
        eng.fill_slots_ex(b, one, kn, vn, keep, free, nf, pos=pos, pos_new=at, acc=acc)
        eng.attend(b, q, out, keep=keep, pos=pos, q_pos=at, acc=acc, acc_out=acc)
        full = len(h[0]["free"]) == 1
        if full:
            eng.evict_accumulated(b, acc, budget, keep, free, nf, live=keep, pos=pos, sinks=sinks, acc_out=acc)
            evictions += 1
        got, ga = out.double().cpu().numpy(), acc.double().cpu().numpy()
        for u in range(U):
            s = h[u]
            i = s["free"].pop(0)
            s["k"][i], s["v"][i] = kn[u].double().cpu().numpy(), vn[u].double().cpu().numpy()
            s["live"][i], s["pos"][i], s["acc"][i] = True, step, 0
            o, _, p, _ = ora.attend(q[u].double().cpu().numpy(), s["k"], s["v"], s["pos"], [step], s["live"])
            assert np.max(np.abs(got[u] - o)) <= 2.0 ** -8 * np.max(np.abs(o)) + 1e-4
            s["acc"] += p.sum((0, 1))
            if full:
                kept = ora.evict_accumulated(s["acc"], s["pos"], s["live"], w, budget, sinks)
                s["live"], f = ora.evict_in_place(cap, kept)
                s["free"], s["acc"] = list(f), np.where(s["live"], s["acc"], 0)
            r = slice(u * cap, (u + 1) * cap)
            assert np.array_equal(keep[r].cpu().numpy() != 0, s["live"]), (step, u)
            assert np.max(np.abs(ga[r] - s["acc"])) <= 1e-4
            assert nf[u] == len(s["free"])
    eng.check_status()
    assert evictions >= 5


def test_captured_decode_step():
    """Fill, attend and evict captured together: replays give the bits of eager steps."""
    G, w, cap, budget, U = 4, 4, 200, 90, 5
    off, T = offsets([cap] * U), 5 * cap
    one = Offsets(np.arange(U + 1), DEV)
    ends = []
    for captured in (False, True):
        torch.manual_seed(3)
        eng = Engine(G, w, U, T, redundancy="closed")
        K, V = (torch.randn((T, 128), device=DEV).to(torch.bfloat16) for _ in range(2))
        b = Batch(K, V, None, off)
        keep = torch.ones(T, dtype=torch.uint8, device=DEV)
        pos = torch.arange(cap, dtype=torch.int32, device=DEV).repeat(U)
        acc, acc2 = torch.rand(T, device=DEV), torch.zeros(T, device=DEV)
        free, nf = torch.full((T,), -1, dtype=torch.int32, device=DEV), torch.zeros(U, dtype=torch.int32, device=DEV)
        free2, nf2 = torch.zeros_like(free), torch.zeros_like(nf)
        kn, vn = (torch.zeros((U, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        q = torch.zeros((U, G, 1, 128), dtype=torch.bfloat16, device=DEV)
        at = torch.full((U,), cap, dtype=torch.int32, device=DEV)
        out = torch.empty_like(q)

        def step():
            eng.evict_accumulated(b, acc, budget, keep, free, nf, live=keep, pos=pos, sinks=3, acc_out=acc2)
            eng.fill_slots_ex(b, one, kn, vn, keep, free, nf, pos=pos, pos_new=at, acc=acc2,
                              free_out=free2, n_free_out=nf2)
            eng.attend(b, q, out, keep=keep, pos=pos, q_pos=at, acc=acc2, acc_out=acc)
            at.add_(1)

        step()                     # scratch is allocated outside the capture
        if captured:
            g = torch.cuda.CUDAGraph()
            state = [t.clone() for t in (keep, pos, acc, acc2, free, nf, free2, nf2, at, K, V)]
            with torch.cuda.graph(g):
                step()
            for t, x in zip((keep, pos, acc, acc2, free, nf, free2, nf2, at, K, V), state):
                t.copy_(x)
        log = []
        for i in range(20):
            torch.manual_seed(100 + i)
            kn.copy_(torch.randn(U, 128, device=DEV))
            vn.copy_(torch.randn(U, 128, device=DEV))
            q.copy_(torch.randn(U, G, 1, 128, device=DEV))
            if captured:
                g.replay()
            else:
                step()
            log.append([t.clone() for t in (out, keep, pos, acc, acc2, free, nf, free2, nf2)])
        eng.check_status()
        ends.append(log)
    for x, y in zip(*ends):
        for s, t in zip(x, y):
            assert torch.equal(s, t)
    assert int(ends[0][-1][6].sum()) > 0


def crowded(bits, equal, rng):
    """Weights of which a quarter each lies in one of four neighbouring bins of 2^bits keys when
    the range up to the largest is cut into 512, in an order of their own.  The second bin starts
    with a gap, so the range of its keys ends behind the bin if it is cut evenly from there, and
    the first key of the third occurs `equal` times."""
    size = 1 << bits
    i = np.arange(4 * size)
    key = np.concatenate([i[i != size], np.full(equal - 1, 2 * size), [512 * size - 1]])
    return rng.permutation((0x3f800000 + key).astype(np.uint32).view(np.float32))


@pytest.mark.parametrize("units,bits", [(600, 11), (150, 11), (24, 11), (24, 13)])
@pytest.mark.parametrize("equal", [1, 40, 300])
def test_evict_crowded_bins(units, bits, equal):
    """Budgets at the ends of the bins that the weights crowd into, in one CTA of 128 and 512
    threads per unit and in clusters of two and eight."""
    rng = np.random.default_rng(units + bits + equal)
    size = 1 << bits
    ends = np.cumsum([1, size, size + equal - 1, size - 1])          # rows above each bin
    budgets = (ends[:, None] + np.arange(-2, 4)).reshape(-1).clip(0)
    acc = [crowded(bits, equal, rng) for _ in range(units)]
    w, n = 2, len(acc[0])
    # the two newest rows stay anyway and are not ranked
    acc = np.concatenate([np.concatenate([a, [1.0, 1.0]]) for a in acc])
    evict([n + w] * units, acc, int(budgets.max()), w=w, budgets=np.resize(budgets, units), with_idx=units < 100)


@pytest.mark.parametrize("units,n", [(2048, 2176), (40, 32000)])
def test_evict_alike_weights_beside_a_small_one(units, n):
    """What decoding leaves where all rows are looked at alike and one is not."""
    rng = np.random.default_rng(10)
    acc = np.exp(0.1 * rng.standard_normal((units, n)))
    acc[:, n // 3] = 1e-20
    evict([n] * units, acc.reshape(-1), n, budgets=rng.integers(1, n, units), with_idx=False)
