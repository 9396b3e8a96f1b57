"""Attention over a live cache (rkv_attend, rkv_attend_shared) against the oracle.

Tolerances, elementwise, from the arithmetic:
* a logit is a sum of 128 exact products added in fp32, each addition off by at
  most 2^-23 of a partial sum (the tensor cores may truncate): dz = 2^-23 * 136 *
  max sum_d |q_d k_d| / sqrt(d), which also covers the scaling's roundings;
* a probability is then off by a factor of at most 1 + 2 dz + 2^-20 (numerator,
  denominator, two 2^x of 2 ulp each, sums of at most a few hundred terms per
  thread in fp32 joined in a tree: N 2^-24 / 64 more), and its two-bf16 form by 2^-16;
* out adds the accumulation of the p v (N terms in fp32: at most N 2^-23 of
  sum p |v|, in practice far less; a warp adds 16 per step) and one rounding to
  bf16, 2^-8 of the value at most;
* where a prefix has more than 4 query rows, or a unit more than 8, p is one bf16, half
  a step, 2^-8 of each p at most, on its share of sum p |v|, and 2^x may come from a
  polynomial that is off by 2.6e-6 < 2^-18 at most (numerator and denominator: 2^-17);
* lse: dz + 2^-20 + 2^-22 |lse|;  acc: |p| times the factor above, and 2^-23 of
  the sum.
"""
import numpy as np
import pytest
import torch

from decode_kv_cache_eviction_b200 import Batch, Engine, Prefix, RkvError
from decode_kv_cache_eviction_b200 import _binding as B
from oracle import rkv_oracle as ora

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def bf(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


class Case:
    """One call: inputs on the device and (float64) on the host."""

    def __init__(self, lengths, G, nq, seed=0, live=None, positions=False, local=0, sinks=0,
                 weights=False, scale=1.0, prefixes=None, unit_prefix=None):
        rng = np.random.default_rng(seed)
        self.lengths, self.G, self.nq, self.local, self.sinks = lengths, G, nq, local, sinks
        self.off = offsets(lengths)
        U, T = len(lengths), int(self.off[-1])
        self.K, self.V = bf(rng.standard_normal((T, 128)) * scale), bf(rng.standard_normal((T, 128)))
        self.Q = bf(rng.standard_normal((U, G, nq, 128)) * scale)
        self.keep = self.pos = self.q_pos = self.acc = None
        if live is not None:
            k = (rng.random(T) < live).astype(np.uint8)
            if U > 1:
                k[self.off[1]:self.off[2]] = 0          # one unit with no live row
            self.keep = torch.from_numpy(k).to(DEV)
        if positions:
            p = np.concatenate([rng.permutation(2 * n)[:n] for n in lengths]) if T else np.zeros(0)
            self.pos = torch.from_numpy(p.astype(np.int32)).to(DEV)
            self.q_pos = torch.from_numpy(np.array([2 * n - 1 for n in lengths], np.int32)).to(DEV)
        if weights:
            self.acc = torch.from_numpy(rng.random(T).astype(np.float32)).to(DEV)
        self.prefixes, self.unit_prefix = prefixes, unit_prefix
        if prefixes is not None:
            self.poff = offsets(prefixes)
            n = int(self.poff[-1])
            self.PK, self.PV = bf(rng.standard_normal((n, 128)) * scale), bf(rng.standard_normal((n, 128)))
        self.acc_out = torch.full((T,), float("nan"), device=DEV) if weights else None
        self.out = torch.full((U, G, nq, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((U, G, nq), float("nan"), device=DEV)

    def engine(self, **kw):
        return Engine(self.G, max(self.nq, 1), len(self.lengths), max(1, int(self.off[-1])),
                      redundancy="closed", **kw)

    def run(self, eng=None, stream=None):
        self.eng = eng or self.engine()
        b = Batch(self.K, self.V, None, self.off)
        kw = dict(keep=self.keep, pos=self.pos, q_pos=self.q_pos, local=self.local,
                  sinks=self.sinks, acc=self.acc, acc_out=self.acc_out, stream=stream)
        if self.prefixes is None:
            self.eng.attend(b, self.Q, self.out, self.lse, **kw)
        else:
            self.prefix = Prefix(self.PK, self.PV, self.poff, self.unit_prefix)
            self.eng.attend_shared(b, self.prefix, self.Q, self.out, self.lse, **kw)
        self.eng.check_status(stream)
        torch.cuda.synchronize()
        return self

    def wide(self):
        return self.G * self.nq > 8

    def unit(self, u):
        """Oracle arguments of unit u (prefix rows first) and its prefix length."""
        a, e = int(self.off[u]), int(self.off[u + 1])
        n = e - a
        k, v = f64(self.K[a:e]), f64(self.V[a:e])
        P = 0
        if self.prefixes is not None and self.unit_prefix[u] >= 0:
            x = self.unit_prefix[u]
            p0, p1 = int(self.poff[x]), int(self.poff[x + 1])
            P = p1 - p0
            k, v = np.concatenate([f64(self.PK[p0:p1]), k]), np.concatenate([f64(self.PV[p0:p1]), v])
        pos = np.arange(P + n)
        if self.pos is not None:
            pos[P:] = self.pos[a:e].cpu().numpy()
        newest = P + n - 1 if self.q_pos is None else int(self.q_pos[u])
        live = None
        if self.keep is not None:
            live = np.concatenate([np.ones(P), self.keep[a:e].cpu().numpy()])
        return k, v, pos, newest - (self.nq - 1) + np.arange(self.nq), live, P

    def check(self, units=None):
        out, lse = f64(self.out), f64(self.lse)
        for u in range(len(self.lengths)) if units is None else units:
            k, v, pos, qp, live, P = self.unit(u)
            q = f64(self.Q[u])
            o, s, p, seen = ora.attend(q, k, v, pos, qp, live, self.local, self.sinks)
            N = len(k)
            dz = 0.0 if N == 0 else 2.0 ** -23 * 136 * np.max(
                np.abs(q).reshape(-1, 128) @ np.abs(k).T) / np.sqrt(128)
            poly = 2.0 ** -17 if self.prefixes is not None or self.wide() else 0.0
            eps = 2 * dz + 2.0 ** -20 + N * 2.0 ** -30 + poly
            mass = p.reshape(-1, N) @ np.abs(v) if N else np.zeros((self.G * self.nq, 128))
            one = N if self.wide() else P        # rows whose p is one bf16
            pre = p[..., :one].reshape(-1, one) @ np.abs(v[:one]) if one else np.zeros_like(mass)
            tol = 2.0 ** -8 * np.abs(o) + (eps + 2.0 ** -16 + N * 2.0 ** -23) * mass.reshape(o.shape)
            tol += 2.0 ** -8 * pre.reshape(o.shape)
            assert np.all(np.abs(out[u] - o) <= tol), (u, np.max(np.abs(out[u] - o) - tol))
            none = np.isneginf(s)
            assert np.array_equal(np.isneginf(lse[u]), none), u
            assert np.all(out[u][none] == 0), u
            ok = ~none
            assert np.all(np.abs(lse[u][ok] - s[ok]) <= dz + poly + 2.0 ** -20 + 2.0 ** -22 * np.abs(s[ok])), u
            if self.acc_out is not None:
                a, e = int(self.off[u]), int(self.off[u + 1])
                w = p.sum((0, 1))[P:]
                want = f64(self.acc[a:e]) + w if self.acc is not None else w
                got = f64(self.acc_out[a:e])
                assert np.all(np.abs(got - want) <= eps * w + 2.0 ** -22 * want), u
                unseen = ~seen.any(0)[P:]
                base = f64(self.acc[a:e]) if self.acc is not None else np.zeros(e - a)
                assert np.array_equal(got[unseen], base[unseen]), u


ODD = [1, 0, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 300, 1000, 4097]


@pytest.mark.parametrize("G,nq", [(1, 1), (4, 1), (8, 1), (3, 2), (4, 4), (4, 8), (5, 7), (16, 4)])
def test_odd_lengths(G, nq):
    Case(ODD, G, nq, seed=G + nq, weights=True).run().check()


@pytest.mark.parametrize("live", [1.0, 0.5, 0.03])
@pytest.mark.parametrize("positions", [False, True])
@pytest.mark.parametrize("nq", [1, 3])
def test_live_mask_and_positions(live, positions, nq):
    Case(ODD, 4, nq, seed=7, live=live, positions=positions, weights=True).run().check()


@pytest.mark.parametrize("local,sinks", [(1, 0), (1, 4), (7, 4), (32, 0), (100, 4), (100, 200),
                                         (5000, 4), (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("positions", [False, True])
@pytest.mark.parametrize("nq", [1, 4])
def test_window_and_sinks(local, sinks, positions, nq):
    Case(ODD, 2, nq, seed=local % 97, local=local, sinks=sinks, positions=positions,
         live=0.7 if positions else None, weights=True).run().check()


def test_split_units_with_window_and_long_rows():
    Case([40000, 7, 33333], 4, 1, seed=3, weights=True).run().check()
    Case([40000, 7, 33333], 4, 2, seed=4, local=9000, sinks=70, weights=True).run().check()


def test_peaked_logits():
    """Logits of +-30: the running maximum moves, and most weights underflow."""
    Case([3000, 500, 17], 4, 2, seed=5, scale=3.0, weights=True).run().check()


def test_more_query_rows_than_one_pass():
    Case([2000, 40, 700], 16, 16, seed=6, weights=True).run().check()     # 256 rows


@pytest.mark.parametrize("G,nq", [(4, 8), (17, 1), (8, 16), (16, 16)])
@pytest.mark.parametrize("local,sinks", [(0, 0), (300, 4), (2000, 130)])
def test_many_query_rows(G, nq, local, sinks):
    """17 to 256 query rows over whole units."""
    Case([5000, 127, 128, 129, 1, 0, 2500], G, nq, seed=60 + G, local=local, sinks=sinks,
         weights=True).run().check()


def test_many_query_rows_peaked_and_long():
    Case([30000, 900], 4, 8, seed=61, scale=3.0).run().check()


def test_many_query_rows_and_values_that_are_not_finite():
    """Rows behind the window, of the next unit, and seen by the newest query alone."""
    c = Case([1500, 1000], 4, 8, seed=62, local=200, sinks=2, weights=True)
    c.run()
    assert c.wide()
    want = c.out.clone(), c.lse.clone(), c.acc_out.clone()
    nan, inf = float("nan"), float("inf")
    c.V[100:1000], c.K[100:900] = nan, inf        # before every window of unit 0
    c.V[1500 + 2], c.K[1500 + 2] = inf, nan       # unit 1: behind the sinks
    c.run(c.eng)
    assert torch.allclose(c.out.float(), want[0].float(), atol=2e-2)
    assert torch.allclose(c.lse, want[1], atol=1e-4) and torch.allclose(c.acc_out, want[2], atol=1e-4)
    c.V[2499] = nan
    c.run(c.eng)
    assert bool(c.out[1, :, 7].isnan().all()) and not bool(c.out[1, :, :7].isnan().any())
    assert torch.allclose(c.out[1, :, :7].float(), want[0][1, :, :7].float(), atol=2e-2)
    assert not bool(c.out[0].isnan().any())
    c.K[2499], c.V[2499] = inf, 0.0               # a logit that is not finite
    c.run(c.eng)
    assert bool(c.out[1, :, 7].isnan().any()) and not bool(c.out[1, :, :7].isnan().any())


def test_largest_finite_values_in_unseen_rows():
    """An unseen row's weight is 0 for every V, the type's largest and lowest too: through
    windows and causal masks of many query rows, and behind a prefix's end."""
    big = float(torch.finfo(torch.bfloat16).max)
    c = Case([1500, 1000], 4, 8, seed=63, local=200, sinks=2).run()
    want = c.out.clone()
    c.V[100:1000] = big                           # before every window of unit 0
    c.V[1500 + 2:1500 + 790] = -big               # unit 1: between the sinks and the windows
    c.run(c.eng)
    assert torch.allclose(c.out.float(), want.float(), atol=1e-2)
    c.check()
    c = Case([10] * 20 + [300] * 20, 2, 1, seed=64, prefixes=[500, 300], unit_prefix=[0] * 40,
             local=250).run()
    want = c.out.clone()
    c.PV[500:], c.PV[:200] = big, -big            # the next prefix, and rows nobody sees
    c.PV[400] = big                               # seen by the short units alone
    c.run(c.eng)
    assert torch.allclose(c.out[20:].float(), want[20:].float(), atol=1e-2)


@pytest.mark.parametrize("G,nq", [(4, 1), (2, 3), (4, 3)])
def test_logits_of_minus_infinity_weigh_nothing(G, nq):
    """A seen row whose logits are all -inf: its p is 0, in the sums and in the weights."""
    c = Case([300, 40], G, nq, seed=65, weights=True)
    c.Q.copy_(c.Q.abs().clamp_min(0.01))
    c.K[20] = float("-inf")
    c.run()
    assert not bool(c.out.isnan().any()) and not bool(c.acc_out.isnan().any())
    assert float(c.acc_out[20]) == float(c.acc[20])
    c.check([1])


def test_queries_that_stand_elsewhere():
    """q_pos without pos: queries behind the cache, inside it, and before it."""
    c = Case([300, 300, 300, 300], 4, 2, seed=8, local=50, sinks=3, weights=True)
    c.q_pos = torch.tensor([1000, 150, 0, -5], dtype=torch.int32, device=DEV)
    c.run().check()
    assert bool((c.out[3] == 0).all())


def test_what_lies_in_unseen_rows_does_not_matter():
    """Infinities and NaN in dead rows, behind the window, and in rows that only a
    later query sees."""
    c = Case([200, 200, 500], 4, 3, seed=9, live=0.5, local=60, sinks=4, weights=True)
    c.keep[200:400] = 1
    c.run()
    want = c.out.clone(), c.lse.clone(), c.acc_out.clone()
    dead = c.keep == 0
    bad = torch.tensor([float("nan"), float("inf"), float("-inf")], device=DEV).to(torch.bfloat16)
    c.K[dead], c.V[dead] = bad[0], bad[1]
    c.V[200 + 50:200 + 90] = bad[1]         # unit 1: behind the window of every query
    c.K[200 + 50:200 + 90] = bad[2]
    c.run(c.eng)
    assert torch.equal(c.out, want[0]) and torch.equal(c.lse, want[1])
    assert torch.equal(c.acc_out, want[2])
    # unit 1's newest row is seen by the newest query alone
    c.V[399], c.K[399] = bad[0], bad[0]
    c.run(c.eng)
    assert torch.equal(c.out[1, :, :2], want[0][1, :, :2])
    assert torch.equal(c.lse[1, :, :2], want[1][1, :, :2])
    assert bool(c.out[1, :, 2].isnan().all())
    assert torch.equal(c.out[[0, 2]], want[0][[0, 2]])


def test_infinite_values_in_seen_rows():
    c = Case([100, 3000], 2, 1, seed=10)
    c.V[50, 3] = float("inf")
    c.V[60, 5] = float("-inf")
    c.V[61, 5] = float("inf")
    c.run()
    out = c.out.float()
    assert bool((out[0, :, 0, 3] == float("inf")).all()) and bool(out[0, :, 0, 5].isnan().all())
    c.V[50, 3] = c.V[60, 5] = c.V[61, 5] = 0
    keep = [i for i in range(128) if i not in (3, 5)]
    rest = out[0][..., keep].clone()
    c.run(c.eng)
    assert torch.allclose(rest, c.out.float()[0][..., keep], atol=1e-2)
    c.check([1])


def test_repeats_and_streams_give_the_same_bits():
    c = Case([5000, 64, 1, 30000], 4, 2, seed=11, live=0.6, weights=True).run()
    want = c.out.clone(), c.lse.clone(), c.acc_out.clone()
    s = torch.cuda.Stream()
    for stream in (None, s):
        for t in (c.out, c.lse, c.acc_out):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        c.run(c.eng, stream=stream)
        s.synchronize()
        assert torch.equal(c.out, want[0]) and torch.equal(c.lse, want[1])
        assert torch.equal(c.acc_out, want[2])


def test_weights_in_place_and_from_zero():
    c = Case([700, 90], 4, 1, seed=12, weights=True).run()
    want = c.acc_out.clone()
    b = Batch(c.K, c.V, None, c.off)
    acc = c.acc.clone()
    c.eng.attend(b, c.Q, c.out, None, acc=acc, acc_out=acc)
    assert torch.equal(acc, want)
    zero = torch.full_like(acc, float("nan"))
    c.eng.attend(b, c.Q, c.out, None, acc_out=zero)
    c.acc, c.acc_out = None, zero
    c.check()


def test_captured_call_replays_on_new_inputs():
    c = Case([9000, 300, 5], 4, 1, seed=13, live=0.8, weights=True).run()
    b = Batch(c.K, c.V, None, c.off)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.eng.attend(b, c.Q, c.out, c.lse, keep=c.keep, acc=c.acc, acc_out=c.acc_out)
    c.Q.copy_(torch.randn_like(c.Q))
    c.keep.copy_((torch.rand(len(c.keep), device=DEV) < 0.4).to(torch.uint8))
    g.replay()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("G,nq,shared", [(4, 3, False), (4, 8, False), (4, 1, True), (4, 4, True)])
def test_captured_calls_of_one_engine(G, nq, shared):
    """Two captures that share the engine's scratch, replayed in turn on new inputs; their
    launches start early only where the one before is of the same call."""
    kw = dict(weights=True, live=0.7)
    if shared:
        kw.update(prefixes=[700, 90], unit_prefix=[0, 1, 0, -1])
    c = Case([2000, 300, 5, 64], G, nq, seed=66, **kw).run()
    d = Case([70, 1000, 0, 900], G, nq, seed=67, **kw)
    eng = Engine(G, nq, 4, 4000, redundancy="closed")
    c.run(eng)
    d.run(eng)
    graphs = []
    for x in (c, d):
        b = Batch(x.K, x.V, None, x.off)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a = dict(keep=x.keep, acc=x.acc, acc_out=x.acc_out)
            if shared:
                eng.attend_shared(b, x.prefix, x.Q, x.out, x.lse, **a)
            else:
                eng.attend(b, x.Q, x.out, x.lse, **a)
        graphs.append((b, g))
    for x in (c, d):
        x.Q.copy_(torch.randn_like(x.Q))
        x.acc.copy_(torch.rand_like(x.acc))
    for _ in range(3):
        for _, g in graphs:
            g.replay()
    torch.cuda.synchronize()
    c.check()
    d.check()


def test_two_engines_on_two_streams():
    cases = [Case([3000, 100], 4, 2, seed=68, weights=True), Case([900, 4000], 4, 8, seed=69, weights=True)]
    want = []
    for c in cases:
        c.run()
        want.append((c.out.clone(), c.lse.clone(), c.acc_out.clone()))
    streams = [torch.cuda.Stream() for _ in cases]
    batches = [Batch(c.K, c.V, None, c.off) for c in cases]
    for c in cases:
        c.out.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, b, s in zip(cases, batches, streams):
            c.eng.attend(b, c.Q, c.out, c.lse, acc=c.acc, acc_out=c.acc_out, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c.out, w[0]) and torch.equal(c.lse, w[1]) and torch.equal(c.acc_out, w[2])


def test_first_call_inside_a_capture_is_refused():
    c = Case([9000], 4, 1, seed=14)
    eng = c.engine()
    b = Batch(c.K, c.V, None, c.off)
    x = torch.zeros(8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(RkvError) as ei:
            eng.attend(b, c.Q, c.out)
        x += 1
    assert ei.value.code == B.RKV_ERR_INVALID_ARG
    g.replay()                                   # the capture itself stayed valid
    torch.cuda.synchronize()
    assert bool((x == 1).all())
    c.run(eng).check()


def test_offsets_beyond_32_bits():
    """17.2 million rows: element offsets pass 2^31, byte offsets 2^32."""
    n, U = 131072, 132
    off = offsets([n] * (U - 1) + [1000])
    T = int(off[-1])
    K = torch.zeros((T, 128), dtype=torch.bfloat16, device=DEV)
    V = torch.zeros((T, 128), dtype=torch.bfloat16, device=DEV)
    c = Case([1000], 4, 1, seed=15)
    a = int(off[U - 1])
    K[a:], V[a:] = c.K, c.V
    Q = torch.zeros((U, 4, 1, 128), dtype=torch.bfloat16, device=DEV)
    Q[U - 1] = c.Q[0]
    V[int(off[U - 2]):a] = 1.0
    out = torch.empty_like(Q)
    acc = torch.empty(T, device=DEV)
    eng = Engine(4, 1, U, T, redundancy="closed")
    eng.attend(Batch(K, V, None, off), Q, out, acc_out=acc)
    torch.cuda.synchronize()
    c.out, c.lse = out[U - 1:], c.lse
    c.eng = eng
    ref = Case([1000], 4, 1, seed=15).run()
    assert torch.allclose(out[U - 1].float(), ref.out[0].float(), atol=2e-2)
    assert bool((out[U - 2] == 1).all()) and bool((out[0] == 0).all())
    assert abs(float(acc[a:].double().sum()) - 4) < 1e-4
    assert abs(float(acc[int(off[U - 2]):a].double().sum()) - 4) < 1e-3


# ---------------------------------------------------------------- shared prefixes
@pytest.mark.parametrize("G,nq", [(1, 1), (4, 1), (4, 3), (8, 4)])
def test_shared_prefix(G, nq):
    Case([5, 1, 33, 200, 64, 17, 0, 90], G, nq, seed=20 + G, prefixes=[100, 1, 0, 1000],
         unit_prefix=[0, 3, -1, 3, 1, 0, 3, 2], weights=True).run().check()


@pytest.mark.parametrize("members", [1, 2, 9, 40, 100])
def test_shared_prefix_members(members):
    rng = np.random.default_rng(members)
    lengths = rng.integers(1, 60, members + 3).tolist()
    up = [1] * members + [0, 2, 0]
    rng.shuffle(up)
    Case(lengths, 4, 1, seed=30 + members, prefixes=[513, 3001, 129], unit_prefix=up,
         weights=True).run().check()


@pytest.mark.parametrize("local,sinks", [(20, 0), (20, 4), (300, 4), (2000, 0)])
def test_shared_prefix_with_window(local, sinks):
    """The window of a short sequence reaches into the prefix, a long one's does not;
    every sequence of a prefix has its own."""
    Case([5, 400, 33, 64, 17, 150, 1, 700], 4, 2, seed=40, prefixes=[1000, 260],
         unit_prefix=[0, 0, 0, 1, 1, 0, -1, 0], local=local, sinks=sinks, weights=True).run().check()


def test_shared_prefix_with_live_mask_and_positions():
    c = Case([50, 60, 300], 4, 2, seed=41, prefixes=[400], unit_prefix=[0, 0, 0], live=0.5,
             positions=True, local=500, sinks=4, weights=True)
    c.pos += 400
    c.q_pos += 400
    c.run().check()


@pytest.mark.parametrize("local,sinks", [(20, 0), (250, 4), (2000, 200)])
def test_shared_prefix_wide_with_window(local, sinks):
    rng = np.random.default_rng(local)
    lengths = rng.integers(0, 400, 60).tolist()
    Case(lengths, 4, 2, seed=45, prefixes=[1000, 260], unit_prefix=[int(i % 3 == 0) for i in range(60)],
         local=local, sinks=sinks, weights=True).run().check()


def test_shared_prefix_wide_values_that_are_not_finite():
    c = Case([10] * 20 + [300] * 20, 2, 1, seed=46, prefixes=[500, 300], unit_prefix=[0] * 40,
             local=250, weights=True).run()
    want = c.out.clone(), c.acc_out.clone()
    c.PV[400], c.PK[400] = float("nan"), float("inf")   # seen by the short units alone
    c.PV[500:] = float("nan")                             # the next prefix, behind this one's end
    c.PV[100], c.PK[90] = float("inf"), float("nan")      # seen by nobody
    c.run(c.eng)
    assert bool(c.out[:20].isnan().all())
    assert torch.allclose(c.out[20:].float(), want[0][20:].float(), atol=2e-2)
    assert torch.allclose(c.acc_out[200:], want[1][200:], atol=1e-4)


def test_shared_prefix_long():
    Case([100] * 40, 4, 1, seed=42, prefixes=[30000], unit_prefix=[0] * 40).run().check([0, 7, 39])


def test_shared_prefix_values_that_one_unit_does_not_see():
    """A window that leaves a row of the prefix to one unit alone: what it holds
    reaches that unit only."""
    c = Case([10, 200], 2, 1, seed=43, prefixes=[300], unit_prefix=[0, 0], local=150).run()
    want = c.out.clone()
    c.PV[200], c.PK[200] = float("nan"), float("inf")   # 161 .. 299 for unit 0; unit 1 sees none
    c.PV[100] = float("nan")                              # nobody
    c.run(c.eng)
    assert torch.equal(c.out[1], want[1]) and bool(c.out[0].isnan().all())


def test_shared_call_without_any_prefix():
    c = Case([100, 33], 4, 1, seed=44, prefixes=[50], unit_prefix=[-1, -1], weights=True).run()
    c.check()
    d = Case([100, 33], 4, 1, seed=44, prefixes=[], unit_prefix=[-1, -1], weights=True).run()
    assert torch.equal(c.out, d.out)


@pytest.mark.parametrize("units", [2, 40])
def test_prefixes_without_rows(units):
    up = [i % 2 for i in range(units)]
    c = Case([100] * units, 4, 1, seed=47, prefixes=[0, 0], unit_prefix=up, weights=True).run()
    c.check()
    Case([30] * units, 4, 1, seed=48, prefixes=[0, 200], unit_prefix=up, weights=True).run().check()


@pytest.mark.parametrize("G,nq", [(4, 1), (2, 3), (4, 4), (8, 4)])
@pytest.mark.parametrize("local,sinks", [(0, 0), (2500, 40)])
def test_shared_prefix_and_long_own_rows(G, nq, local, sinks):
    """Many members of a long prefix, own rows in several parts: both kernels' parts are
    joined; the timing names the kernels that ran."""
    lengths = [2000, 1900, 0, 1, 700] * 8
    for n, units in ((6000, None), (40000, [0, 1, 2, 3, 9])):
        c = Case(lengths, G, nq, seed=70 + G, prefixes=[n, 100], local=local, sinks=sinks, weights=True,
                 unit_prefix=[int(u % 5 == 3) for u in range(40)])
        eng = c.engine()
        eng.set_timing(True)
        c.run(eng).check(units)
    if not local:      # 32 units would read 40000 rows each
        assert eng.read_timing()["shared"][1] == 1


@pytest.mark.parametrize("G,nq", [(1, 1), (4, 1), (2, 3), (4, 4), (8, 4)])
@pytest.mark.parametrize("weights", [False, True])
def test_each_unit_reads_its_prefix(G, nq, weights):
    """Few members: one launch over prefix and own rows, in one chunk or in many."""
    for lengths, prefixes in (([40, 3, 0, 260], [70, 33]), ([500, 2000, 1, 64], [3000, 1])):
        c = Case(lengths, G, nq, seed=80 + G, prefixes=prefixes, unit_prefix=[0, 1, 0, -1], weights=weights,
                 live=0.8)
        eng = c.engine()
        eng.set_timing(True)
        c.run(eng).check()
        assert eng.read_timing()["shared"][1] == 0


# ---------------------------------------------------------------- refusals
def test_refusals():
    c = Case([100, 33], 4, 2, seed=50, weights=True)
    eng = c.engine()
    b = Batch(c.K, c.V, None, c.off)
    f = lambda code, **kw: _refused(code, lambda: eng.attend(b, kw.pop("Q", c.Q), c.out, **kw))
    f(B.RKV_ERR_INVALID_ARG, local=-1)
    f(B.RKV_ERR_INVALID_ARG, sinks=-1)
    f(B.RKV_ERR_INVALID_ARG, pos=torch.zeros(133, dtype=torch.int32, device=DEV))   # no q_pos
    f(B.RKV_ERR_INVALID_ARG, acc=c.acc)                                             # no acc_out
    one = Engine(4, 1, 2, 133, redundancy="closed")
    _refused(B.RKV_ERR_UNSUPPORTED, lambda: one.attend(b, c.Q, c.out))              # n_q > window
    small = Engine(4, 2, 1, 133, redundancy="closed")
    _refused(B.RKV_ERR_CAPACITY, lambda: small.attend(b, c.Q, c.out))
    small = Engine(4, 2, 2, 132, redundancy="closed")
    _refused(B.RKV_ERR_CAPACITY, lambda: small.attend(b, c.Q, c.out))
    short = Engine(4, 2, 2, 133, redundancy="closed", max_unit_tokens=99)
    _refused(B.RKV_ERR_UNSUPPORTED, lambda: short.attend(b, c.Q, c.out))
    for kw in (dict(lse=torch.empty(2, 4, 1, device=DEV)), dict(keep=torch.ones(133, device=DEV)),
               dict(keep=torch.ones(132, dtype=torch.uint8, device=DEV)),
               dict(acc_out=torch.empty(133, dtype=torch.float64, device=DEV)),
               dict(acc_out=torch.empty(133))):
        with pytest.raises(ValueError):
            eng.attend(b, c.Q, c.out, **kw)
    for q in (c.Q.float(), c.Q[:1], c.Q.transpose(0, 1), c.Q[:, :, :, :64]):
        with pytest.raises(ValueError):
            eng.attend(b, q, c.out)
    x = Prefix(c.K, c.V, [0, 133], [0])
    _refused(B.RKV_ERR_INVALID_ARG, lambda: eng.attend_shared(b, x, c.Q, c.out))     # 1 unit, not 2
    with pytest.raises(ValueError):
        Prefix(c.K, c.V, [0, 100], [0, 0])
    # nothing ran: the outputs are as they were
    torch.cuda.synchronize()
    assert bool(c.out.isnan().all())


def test_refusals_of_sizes_and_overlap():
    c = Case([100, 33], 4, 2, seed=51)
    eng, b = c.engine(), Batch(c.K, c.V, None, c.off)
    q = c.Q.clone()
    _refused(B.RKV_ERR_INVALID_ARG, lambda: eng.attend(b, q, q))     # out is Q's memory
    for kw in (dict(local=2**32 + 5), dict(sinks=2**31)):
        with pytest.raises(ValueError):
            eng.attend(b, q, c.out, **kw)
    torch.cuda.synchronize()
    assert torch.equal(q, c.Q) and bool(c.out.isnan().all())


def _refused(code, call):
    with pytest.raises(RkvError) as ei:
        call()
    assert ei.value.code == code


def test_tampered_prefix_plan_is_refused():
    c = Case([100, 33, 5], 4, 1, seed=51, prefixes=[50, 7], unit_prefix=[0, 1, 0])
    eng = c.engine()
    b = Batch(c.K, c.V, None, c.off)
    for k, i, v in ((1, 0, 5), (1, 0, -2), (3, 1, 1), (3, 0, 3), (2, 1, 3), (0, 1, 1 << 31)):
        x = Prefix(c.PK, c.PV, c.poff, c.unit_prefix)
        x._host[k][i] = v                       # the host copies are what is checked
        with pytest.raises(RkvError):
            eng.attend_shared(b, x, c.Q, c.out)


def test_allocation_fault_then_recovers():
    c = Case([9000], 4, 1, seed=52)
    eng = c.engine()
    eng.inject_fault(B.RKV_FAULT_ALLOC)
    _refused(B.RKV_ERR_OOM, lambda: c.run(eng))
    c.run(eng).check()


def test_no_units_and_empty_units():
    eng = Engine(4, 1, 4, 100, redundancy="closed")
    empty = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    q0 = torch.empty((0, 4, 1, 128), dtype=torch.bfloat16, device=DEV)
    eng.attend(Batch(empty, empty, None, [0]), q0, q0.clone())
    q = torch.randn((3, 4, 1, 128), device=DEV).to(torch.bfloat16)
    out = torch.full_like(q, 7)
    lse = torch.zeros((3, 4, 1), device=DEV)
    eng.attend(Batch(empty, empty, None, [0, 0, 0, 0]), q, out, lse)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())


@pytest.mark.parametrize("lengths,G,nq,shared", [([300, 40], 2, 3, False), ([9000, 9000], 4, 8, False),
                                                 ([40] * 40, 4, 1, True)])
def test_tensor_map_that_cannot_be_made_enqueues_nothing(lengths, G, nq, shared):
    """The weights pass from K, the wide kernel over units, and a prefix: their maps are made
    before the first launch."""
    kw = dict(prefixes=[9000], unit_prefix=[0] * 40) if shared else {}
    c = Case(lengths, G, nq, seed=53, weights=True, **kw).run()
    for t in (c.out, c.lse, c.acc_out):
        t.fill_(float("nan"))
    n = c.eng.launches
    c.eng.inject_fault(B.RKV_FAULT_TENSOR_MAP)
    _refused(B.RKV_ERR_CUDA, lambda: c.run(c.eng))
    torch.cuda.synchronize()
    assert c.eng.launches == n
    assert all(bool(t.isnan().all()) for t in (c.out, c.lse, c.acc_out))
    c.run(c.eng).check([0])


@pytest.mark.parametrize("units,G,nq", [(4, 4, 1), (65536, 16, 16), (4096, 4, 8)])
@pytest.mark.parametrize("shared", [False, True])
def test_scratch_of_the_first_call(units, G, nq, shared):
    """At most what the header says (to 4 MB of the allocators): 15 MB + 4 max_units (G w + 1), and
    35 MB + max_units (1044 G w + 4) for shared calls."""
    c = Case([40, 3], G, nq, seed=54, **(dict(prefixes=[70], unit_prefix=[0, 0]) if shared else {}))
    eng = Engine(G, nq, units, 43, redundancy="closed")
    rows = units * G * nq
    most = 35e6 + 1044 * rows + 4 * units if shared else 15e6 + 4 * (rows + units)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    b = Batch(c.K, c.V, None, c.off)
    if shared:
        eng.attend_shared(b, Prefix(c.PK, c.PV, c.poff, c.unit_prefix), c.Q, c.out)
    else:
        eng.attend(b, c.Q, c.out)
    torch.cuda.synchronize()
    assert free - torch.cuda.mem_get_info()[0] <= most + (1 << 22)


def test_output_over_a_part_of_the_queries_is_refused():
    c = Case([100, 33, 7], 4, 2, seed=55)
    eng, b = c.engine(), Batch(c.K, c.V, None, c.off)
    buf = torch.cat([c.Q, c.Q])
    was = buf.clone()
    for q0, o0 in ((0, 1), (1, 0), (2, 0), (0, 2)):
        _refused(B.RKV_ERR_INVALID_ARG, lambda: eng.attend(b, buf[q0:q0 + 3], buf[o0:o0 + 3]))
    torch.cuda.synchronize()
    assert torch.equal(buf, was)
    eng.attend(b, buf[:3], buf[3:], c.lse)        # side by side
    c.out = buf[3:]
    torch.cuda.synchronize()
    c.check()


def test_more_query_rows_than_one_grid_dimension_holds():
    """65600 units of 256 query rows behind one prefix: 65600 blocks of 256 rows."""
    U = 65600
    c = Case([0, 5], 16, 16, seed=56, prefixes=[300], unit_prefix=[0, 0])
    Q = torch.zeros((U, 16, 16, 128), dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(Q, float("nan"))
    Q[0], Q[-1] = c.Q
    eng = Engine(16, 16, U, 5, redundancy="closed")
    eng.set_timing(True)
    b = Batch(c.K, c.V, None, np.array([0] * U + [5]))
    eng.attend_shared(b, Prefix(c.PK, c.PV, c.poff, [0] * U), Q, out)
    eng.check_status()
    assert eng.read_timing()["shared"][1] == 1
    eng.close()
    c.run()                                       # the two alone, for their log-sums
    c.out = torch.stack([out[0], out[-1]])
    c.check()
    # queries of 0 weigh alike what they see, query t the rows up to 284 + t
    v = c.PV.double()
    for t in range(16):
        mean, size = v[:285 + t].mean(0), v[:285 + t].abs().mean(0)
        assert bool(((out[1, 0, t].double() - mean).abs() <= 2.0 ** -8 * (mean.abs() + size)).all()), t
    assert bool((out[1:-1] == out[1, :1]).all())
