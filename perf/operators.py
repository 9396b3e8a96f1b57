"""Measured cases of the cache-attention operators: decode attention over a live cache (attend), the same
with a prefix that several sequences share (attend_shared), eviction by accumulated attention weight
(evict_accumulated) and new tokens into freed slots with their positions (fill_slots_ex).

A *unit* is one (sequence, layer, KV head); unit u owns rows off[u] .. off[u+1]-1 of K and V ([T, 128] bf16).
"""
import math
import random

import torch

own = False
D = 128
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one Llama-3-8B layer, one new token: the smallest call of a decode step, latency counts
        dict(name="attend_one_layer", op="attend", units=8, lo=4096, hi=4096, group=4, queries=1, live=1.0,
             positions=False, local=0, sinks=0, weights=False, lens=1),
        # the whole R1-Llama-8B cache after its 128-step trigger (B = 2048 + 128), weights accumulated
        dict(name="attend_cadence_weights", op="attend", units=2048, lo=2176, hi=2176, group=4, queries=1, live=1.0,
             positions=False, local=0, sinks=0, weights=True, lens=2),
        # a ragged serving batch evicted in place: a third of the slots live, reused out of order
        dict(name="attend_in_place_ragged", op="attend", units=256, lo=2048, hi=8192, group=4, queries=1, live=0.35,
             positions=True, local=0, sinks=0, weights=True, lens=3),
        # sliding window with four sinks over caches that were never trimmed
        dict(name="attend_window_sinks", op="attend", units=509, lo=7001, hi=8192, group=4, queries=1, live=1.0,
             positions=False, local=1024, sinks=4, weights=False, lens=4),
        # eight drafted tokens checked at once (32 query rows per unit)
        dict(name="attend_eight_queries", op="attend", units=64, lo=15000, hi=16384, group=4, queries=8, live=1.0,
             positions=False, local=0, sinks=0, weights=False, lens=5),
        # 32K reasoning traces, uncompressed: the largest read
        dict(name="attend_long_trace", op="attend", units=128, lo=32768, hi=32768, group=4, queries=1, live=1.0,
             positions=False, local=0, sinks=0, weights=False, lens=6),
        # four samples of one prompt, one layer: 16 query rows per prefix
        dict(name="shared_few", op="shared", prefixes=8, members=4, plo=2048, phi=2048, lo=64, hi=512, group=4,
             queries=1, local=0, sinks=0, weights=False, lens=7),
        # 64 samples of one 16K prompt, four layers: 256 query rows per prefix, weights of the own rows
        dict(name="shared_many", op="shared", prefixes=32, members=64, plo=16384, phi=16384, lo=33, hi=511, group=4,
             queries=1, local=0, sinks=0, weights=True, lens=8),
        # the trigger of the R1-Llama-8B cache: 128 of 2176 rows leave
        dict(name="evict_cadence", op="evict", units=2048, lo=2176, hi=2176, recent=8, sinks=4, budget=2036, live=1.0,
             positions=False, lens=9),
        # 32K traces cut to 4096 rows, half of the slots already free, slots out of order
        dict(name="evict_long_in_place", op="evict", units=64, lo=30001, hi=32768, recent=8, sinks=4, budget=4084,
             live=0.5, positions=True, lens=10),
        # one decode step of one layer: a token for each of 8 units
        dict(name="fill_one_layer", op="fill", units=8, lo=4224, hi=4224, free=128, new_lo=1, new_hi=1, lens=11),
        # a block of tokens into a ragged in-place cache
        dict(name="fill_block_ragged", op="fill", units=512, lo=2048, hi=4096, free=640, new_lo=100, new_hi=300, lens=12),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "shared", "shared", "evict", "fill"])
    lens = rng.randrange(1 << 20)
    if op == "attend":
        hi = _log(rng, 16, 32768)
        queries = rng.choice([1, 1, 1, 2, 3, 8])
        group = rng.choice([1, 2, 4, 4, 5, 8])
        units = max(1, min(_log(rng, 1, 2048), min(1 << 22, (1 << 25) // (group * queries)) // hi))
        local = rng.choice([0, 0, _log(rng, 16, 4096)])
        return dict(op=op, units=units, lo=max(1, int(hi * rng.uniform(0.3, 1.0))), hi=hi, group=group, queries=queries,
                    live=rng.choice([1.0, round(rng.uniform(0.05, 1.0), 3)]), positions=rng.random() < 0.4,
                    local=local, sinks=rng.choice([0, 4, 7]) if local else 0, weights=rng.random() < 0.5, lens=lens)
    if op == "shared":
        phi = _log(rng, 100, 32768)
        group, queries = rng.choice([1, 4, 4, 8]), rng.choice([1, 1, 2, 4])
        members = min(_log(rng, 1, 96), (1 << 27) // (phi * group * queries))
        prefixes = max(1, min(_log(rng, 1, 32), (1 << 19) // phi, (1 << 27) // (phi * group * queries * members)))
        hi = _log(rng, 1, 1024)
        local = rng.choice([0, 0, _log(rng, 64, 8192)])
        return dict(op=op, prefixes=prefixes, members=members, plo=max(1, int(phi * rng.uniform(0.5, 1.0))), phi=phi,
                    lo=max(1, int(hi * rng.uniform(0.1, 1.0))), hi=hi, group=group, queries=queries, local=local,
                    sinks=4 if local else 0,
                    weights=rng.random() < 0.4, lens=lens)
    hi = _log(rng, 64, 32768)
    units = max(1, min(_log(rng, 1, 2048), (1 << 21) // hi))
    lo = max(32, int(hi * rng.uniform(0.4, 1.0)))
    if op == "evict":
        return dict(op=op, units=units, lo=lo, hi=hi, recent=rng.choice([1, 8, 32]), sinks=rng.choice([0, 4]),
                    budget=_log(rng, 1, hi), live=rng.choice([1.0, round(rng.uniform(0.2, 1.0), 3)]),
                    positions=rng.random() < 0.5, lens=lens)
    free = _log(rng, 2, lo)
    new_lo = rng.randrange(0, free)
    return dict(op=op, units=units, lo=lo, hi=hi, free=free, new_lo=new_lo, new_hi=rng.randint(new_lo, free), lens=lens)


def _lengths(n, lo, hi, seed):
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(n)]


def _offsets(lengths):
    off = [0]
    for n in lengths:
        off.append(off[-1] + n)
    return off


def _case_lengths(case):
    units = case["units"] if "units" in case else case["prefixes"] * case["members"]
    return _lengths(units, case["lo"], case["hi"], case["lens"])


def _live_count(n, frac):
    return max(1, round(n * frac))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _cache(rows, g):
    """Keys and values of `rows` tokens: keys of varying strength, values with a mean per channel."""
    k = torch.randn((rows, D), generator=g, device=DEV, dtype=torch.bfloat16)
    v = torch.randn((rows, D), generator=g, device=DEV, dtype=torch.bfloat16)
    v += torch.randn(D, generator=g, device=DEV, dtype=torch.bfloat16) * 0.25
    return k, v


def _queries(units, case, k, starts, g):
    """Queries [U, G, n_q, d]: noise, and a part along the unit's first key (the sink that every head looks at)."""
    q = torch.randn((units, case["group"], case["queries"], D), generator=g, device=DEV) * 1.5
    return (q + 0.4 * k[starts].float()[:, None, None, :]).to(torch.bfloat16)


def _pad(off, g=None):
    """Row index [U, Nmax] of every unit's rows (0 beyond its length) and which of them are its own."""
    n = off[1:] - off[:-1]
    at = torch.arange(int(n.max()), device=DEV)
    inside = at[None, :] < n[:, None]
    return torch.where(inside, off[:-1, None] + at[None, :], 0), inside


def _live_and_positions(case, off, g):
    """A live mask with a fixed count in each unit (or None), and positions of the rows in an order of their own (or None).
    The newest token is live."""
    rows, inside = _pad(off)
    n = off[1:] - off[:-1]
    keep = pos = None
    total = int(off[-1])
    newest = n - 1                       # the row that holds the newest position
    if case["positions"]:
        # slots were reused: positions are a permutation of each unit's range, spread over 3 N
        score = torch.rand(rows.shape, generator=g, device=DEV).masked_fill(~inside, 2.0)
        rank = score.argsort(dim=1).argsort(dim=1)
        pos = torch.empty(total, dtype=torch.int32, device=DEV)
        pos[rows[inside]] = (rank * 3 + 1)[inside].to(torch.int32)
        newest = torch.where(inside, rank, -1).argmax(dim=1)
    if case["live"] < 1.0:
        score = torch.rand(rows.shape, generator=g, device=DEV).masked_fill(~inside, 2.0)
        score.scatter_(1, newest[:, None], -1.0)
        count = (n.double() * case["live"]).round().clamp(min=1).long()
        alive = score.argsort(dim=1).argsort(dim=1) < count[:, None]
        keep = torch.zeros(total, dtype=torch.uint8, device=DEV)
        keep[rows[inside]] = alive[inside].to(torch.uint8)
    return keep, pos


def prepare(case, seed):
    g = _gen(seed)
    lengths = _case_lengths(case)
    host_off = _offsets(lengths)
    off = torch.tensor(host_off, device=DEV)
    U, T = len(lengths), host_off[-1]
    s = dict(case=case, off=off, host_off=host_off)
    if case["op"] in ("attend", "shared"):
        s["K"], s["V"] = _cache(T, g)
        s["keep"] = s["pos"] = s["q_pos"] = s["acc"] = s["acc_out"] = s["prefix"] = None
        if case["op"] == "attend":
            s["Q"] = _queries(U, case, s["K"], off[:-1], g)
            s["keep"], s["pos"] = _live_and_positions(case, off, g)
            if s["pos"] is not None:   # the newest query stands at the newest position
                s["q_pos"] = ((off[1:] - off[:-1] - 1) * 3 + 1).to(torch.int32)
        else:
            pre = _offsets(_lengths(case["prefixes"], case["plo"], case["phi"], case["lens"] + 1))
            s["PK"], s["PV"] = _cache(pre[-1], g)
            s["pre_host"], s["pre"] = pre, torch.tensor(pre, device=DEV)
            # unit = (sequence, head): the units of one prefix are `prefixes` apart, as a cache lays them out
            s["unit_prefix"] = [u % case["prefixes"] for u in range(U)]
            s["up"] = torch.tensor(s["unit_prefix"], device=DEV)
            s["Q"] = _queries(U, case, s["PK"], s["pre"][s["up"]], g)
        if case["weights"]:
            s["acc"] = torch.rand(T, generator=g, device=DEV) * 4.0
            s["acc_out"] = torch.empty(T, device=DEV)
        s["out"] = torch.empty_like(s["Q"])
        s["lse"] = torch.empty(s["Q"].shape[:3], device=DEV)
    elif case["op"] == "evict":
        # weights as decoding leaves them: a few heavy rows, many light ones, some equal
        w = torch.exp(2.0 * torch.randn(T, generator=g, device=DEV) - 3.0)
        tie = torch.rand(T, generator=g, device=DEV) < 0.2
        s["acc"] = torch.where(tie, (w * 8).round() / 8, w)
        s["live"], s["pos"] = _live_and_positions(case, off, g)
        s["keep"] = torch.empty(T, dtype=torch.uint8, device=DEV)
        s["free"] = torch.empty(T, dtype=torch.int32, device=DEV)
        s["n_free"] = torch.empty(U, dtype=torch.int32, device=DEV)
        s["acc_out"] = torch.empty(T, device=DEV)
    else:
        s["K"], s["V"] = _cache(T, g)
        n = off[1:] - off[:-1]
        rows, inside = _pad(off)
        score = torch.rand(rows.shape, generator=g, device=DEV).masked_fill(~inside, 2.0)
        dead = score.argsort(dim=1).argsort(dim=1) < case["free"]       # case["free"] <= lo
        s["keep"] = torch.ones(T, dtype=torch.uint8, device=DEV)
        s["keep"][rows[dead]] = 0
        slots = dead.long().argsort(dim=1, descending=True, stable=True)  # dead slots first, ascending
        at = torch.arange(rows.shape[1], device=DEV)[None, :]
        s["free"] = torch.empty(T, dtype=torch.int32, device=DEV)
        s["free"][rows[inside]] = torch.where(at < case["free"], slots, -1)[inside].to(torch.int32)
        s["n_free"] = torch.full((U,), case["free"], dtype=torch.int32, device=DEV)
        s["free_out"], s["n_free_out"] = torch.empty_like(s["free"]), torch.empty_like(s["n_free"])
        s["pos"] = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
        s["acc"] = torch.rand(T, generator=g, device=DEV)
        new = _offsets(_lengths(U, case["new_lo"], case["new_hi"], case["lens"] + 1))
        s["new_host"], s["new"] = new, torch.tensor(new, device=DEV)
        s["K_new"], s["V_new"] = _cache(new[-1], g)
        s["pos_new"] = torch.randint(1 << 20, 1 << 21, (new[-1],), generator=g, device=DEV, dtype=torch.int32)
    if own:
        from decode_kv_cache_eviction_b200 import Batch, Engine, Offsets, Prefix
        kv = s.get("K")
        if kv is None:   # eviction by weight reads no keys
            s["batch"] = Batch(None, None, None, host_off, device=off.device)
        else:
            s["batch"] = Batch(kv, s["V"], None, host_off)
        s["engine"] = Engine(case.get("group", 1), max(case.get("queries", 1), case.get("recent", 1)), U, max(T, 1),
                             redundancy="closed")
        if case["op"] == "shared":
            s["prefix"] = Prefix(s["PK"], s["PV"], s["pre_host"], s["unit_prefix"])
        if case["op"] == "fill":
            s["offsets"] = Offsets(s["new_host"], off.device)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"attend": _run_attend, "shared": _run_shared, "evict": _run_evict, "fill": _run_fill}[s["case"]["op"]](s)


def _result(s):
    got = {"out": s["out"], "lse": s["lse"]}
    if s["acc"] is not None:
        got["acc"] = s["acc_out"]
    return got


def _seen(p, qp, local, sinks):
    """Which positions p the queries at qp see: not later, and inside the window or a sink."""
    v = p <= qp
    return v & ((p > qp - local) | (p < sinks)) if local else v


def _run_attend(s):
    c = s["case"]
    if own:
        s["engine"].attend(s["batch"], s["Q"], s["out"], s["lse"], keep=s["keep"], pos=s["pos"], q_pos=s["q_pos"],
                           local=c["local"], sinks=c["sinks"], acc=s["acc"], acc_out=s["acc_out"])
        return _result(s)
    U, G, n, _ = s["Q"].shape
    rows, inside = _pad(s["off"])
    length = s["off"][1:] - s["off"][:-1]
    p = s["pos"][rows].long() if s["pos"] is not None else torch.arange(rows.shape[1], device=DEV)[None, :].expand_as(rows)
    last = s["q_pos"].long() if s["q_pos"] is not None else length - 1
    qp = last[:, None] - (n - 1) + torch.arange(n, device=DEV)[None, :]              # [U, n]
    see = inside[:, None, :] & _seen(p[:, None, :], qp[:, :, None], c["local"], c["sinks"])  # [U, n, N]
    if s["keep"] is not None:
        see &= (s["keep"][rows] != 0)[:, None, :]
    q = s["Q"].float().reshape(U, G * n, D)
    z = (q @ s["K"][rows].float().transpose(1, 2)).reshape(U, G, n, -1) / math.sqrt(D)
    z.masked_fill_(~see[:, None], float("-inf"))
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    w = torch.where(total > 0, e / total, 0.0)
    v = s["V"][rows].float().masked_fill_(~see.any(1)[:, :, None], 0.0)
    s["out"].copy_((w.reshape(U, G * n, -1) @ v).reshape(U, G, n, D))
    s["lse"].copy_((m + torch.log(total))[..., 0])
    if s["acc"] is not None:
        s["acc_out"].copy_(s["acc"])
        s["acc_out"][rows[inside]] += w.sum((1, 2))[inside]
    return _result(s)


def _run_shared(s):
    c = s["case"]
    if own:
        s["engine"].attend_shared(s["batch"], s["prefix"], s["Q"], s["out"], s["lse"], local=c["local"],
                                  sinks=c["sinks"], acc=s["acc"], acc_out=s["acc_out"])
        return _result(s)
    U, G, n, _ = s["Q"].shape
    P = c["prefixes"]
    M = U // P
    order = torch.arange(U, device=DEV).reshape(M, P).t()          # [P, M] units of each prefix
    plen = s["pre"][1:] - s["pre"][:-1]
    prows, pin = _pad(s["pre"])
    rows, inside = _pad(s["off"])
    length = s["off"][1:] - s["off"][:-1]
    qp = (plen[s["up"]] + length)[:, None] - n + torch.arange(n, device=DEV)[None, :]     # [U, n]
    # the prefix: all its members' queries in one product
    q = s["Q"][order].float().reshape(P, M * G * n, D)
    pk, pv = s["PK"][prows].float(), s["PV"][prows].float().masked_fill_(~pin[:, :, None], 0.0)
    zp = (q @ pk.transpose(1, 2)).reshape(P, M, G, n, -1) / math.sqrt(D)
    seep = pin[:, None, None, :] & _seen(torch.arange(prows.shape[1], device=DEV), qp[order][..., None], c["local"], c["sinks"])
    zp.masked_fill_(~seep[:, :, None], float("-inf"))
    # the units' own rows
    p = plen[s["up"]][:, None] + torch.arange(rows.shape[1], device=DEV)[None, :]
    see = inside[:, None, :] & _seen(p[:, None, :], qp[:, :, None], c["local"], c["sinks"])
    zo = (s["Q"].float().reshape(U, G * n, D) @ s["K"][rows].float().transpose(1, 2)).reshape(U, G, n, -1) / math.sqrt(D)
    zo.masked_fill_(~see[:, None], float("-inf"))
    mp = torch.empty((U, G, n, 1), device=DEV)
    mp[order] = zp.amax(-1, keepdim=True)
    m = torch.maximum(mp, zo.amax(-1, keepdim=True))
    m = torch.where(m == float("-inf"), 0.0, m)
    ep, eo = torch.exp(zp - m[order]), torch.exp(zo - m)
    op, tp = torch.empty((U, G, n, D), device=DEV), torch.empty((U, G, n, 1), device=DEV)
    op[order] = (ep.reshape(P, M * G * n, -1) @ pv).reshape(P, M, G, n, D)
    tp[order] = ep.sum(-1, keepdim=True)
    total = tp + eo.sum(-1, keepdim=True)
    v = s["V"][rows].float().masked_fill_(~see.any(1)[:, :, None], 0.0)
    o = op + (eo.reshape(U, G * n, -1) @ v).reshape(U, G, n, D)
    s["out"].copy_(torch.where(total > 0, o / total, 0.0))
    s["lse"].copy_((m + torch.log(total))[..., 0])
    if s["acc"] is not None:
        s["acc_out"].copy_(s["acc"])
        s["acc_out"][rows[inside]] += torch.where(total > 0, eo / total, 0.0).sum((1, 2))[inside]
    return _result(s)


def _run_evict(s):
    c = s["case"]
    got = {"keep": s["keep"], "free": s["free"], "n_free": s["n_free"], "acc": s["acc_out"]}
    if own:
        s["engine"].evict_accumulated(s["batch"], s["acc"], c["budget"], s["keep"], s["free"], s["n_free"],
                                      live=s["live"], pos=s["pos"], sinks=c["sinks"], acc_out=s["acc_out"])
        return got
    rows, inside = _pad(s["off"])
    at = torch.arange(rows.shape[1], device=DEV)[None, :].expand_as(rows)
    alive = inside & (s["live"][rows] != 0) if s["live"] is not None else inside
    p = s["pos"][rows].long() if s["pos"] is not None else at
    newest = torch.where(alive, p, -1).amax(1, keepdim=True)
    safe = alive & ((p < c["sinks"]) | (p > newest - c["recent"]))
    score = torch.where(alive & ~safe, s["acc"][rows], float("-inf"))
    order = score.argsort(dim=1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, at)
    kept = safe | (alive & (rank < c["budget"]))
    s["keep"][rows[inside]] = kept[inside].to(torch.uint8)
    dead = inside & ~kept
    n_free = dead.sum(1)
    slots = dead.long().argsort(dim=1, descending=True, stable=True)
    s["free"][rows[inside]] = torch.where(at < n_free[:, None], slots, -1)[inside].to(torch.int32)
    s["n_free"].copy_(n_free)
    s["acc_out"][rows[inside]] = torch.where(kept, s["acc"][rows], 0.0)[inside]
    return got


def _run_fill(s):
    got = {n: s[n] for n in ("K", "V", "keep", "pos", "acc", "free_out", "n_free_out")}
    if own:
        s["engine"].fill_slots_ex(s["batch"], s["offsets"], s["K_new"], s["V_new"], s["keep"], s["free"], s["n_free"],
                                  pos=s["pos"], pos_new=s["pos_new"], acc=s["acc"], free_out=s["free_out"],
                                  n_free_out=s["n_free_out"])
        return got
    U = s["off"].numel() - 1
    count = s["new"][1:] - s["new"][:-1]
    unit = torch.repeat_interleave(torch.arange(U, device=DEV), count, output_size=s["K_new"].shape[0])
    nth = torch.arange(unit.numel(), device=DEV) - s["new"][unit]
    base = s["off"][unit]
    to = base + s["free"][base + nth].long()
    s["K"][to], s["V"][to], s["pos"][to] = s["K_new"], s["V_new"], s["pos_new"]
    s["keep"][to] = 1
    s["acc"][to] = 0.0
    rows, inside = _pad(s["off"])
    at = torch.arange(rows.shape[1], device=DEV)[None, :]
    left = s["n_free"].long() - count
    moved = s["free"][torch.gather(rows, 1, (at + count[:, None]).clamp(max=rows.shape[1] - 1))]
    s["free_out"][rows[inside]] = torch.where(at < left[:, None], moved, -1)[inside]
    s["n_free_out"].copy_(left)
    return got


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    lengths = _case_lengths(case)
    T, U = sum(lengths), len(lengths)
    if case["op"] in ("attend", "shared"):
        R, n = case["group"] * case["queries"], case["queries"]
        span = case["local"] + n - 1 + case["sinks"]
        bytes_ = U * R * (4 * D + 4) + (8 * T if case["weights"] else 0)
        if case["op"] == "attend":
            # positions are 3 apart where slots were reused
            near = span * case["live"] / (3 if case["positions"] else 1)
            seen = sum(min(_live_count(x, case["live"]), math.ceil(near)) if case["local"] else _live_count(x, case["live"])
                       for x in lengths)
            bytes_ += seen * 4 * D + (T if case["live"] < 1.0 else 0) + (4 * T if case["positions"] else 0)
            return {"bytes": bytes_, "flops": 4 * D * R * seen}
        pre = _lengths(case["prefixes"], case["plo"], case["phi"], case["lens"] + 1)
        seen = pseen = 0
        pread = [0] * len(pre)
        for u, x in enumerate(lengths):
            q = u % case["prefixes"]
            a = min(x, case["local"] + n - 1) if case["local"] else x
            b = min(pre[q], max(0, case["local"] - x) + case["sinks"]) if case["local"] else pre[q]
            seen, pseen, pread[q] = seen + a, pseen + b, max(pread[q], b)
        return {"bytes": bytes_ + (seen + sum(pread)) * 4 * D, "flops": 4 * D * R * (seen + pseen)}
    if case["op"] == "evict":
        return {"bytes": T * (4 + 1 + 4 + 4 + (1 if case["live"] < 1.0 else 0) + (4 if case["positions"] else 0)), "flops": T}
    new = sum(_lengths(U, case["new_lo"], case["new_hi"], case["lens"] + 1))
    return {"bytes": new * (8 * D + 4 + 4 + 1 + 4) + 4 * (U * case["free"] + T) + 8 * U, "flops": new}


# ------------------------------------------------------------------ the definition in 64 bits, unit by unit
def exact(case, seed):
    s = _inputs_of(case, seed)
    off = s["host_off"]
    U = len(off) - 1
    if case["op"] in ("attend", "shared"):
        G, n = case["group"], case["queries"]
        out = torch.zeros((U, G, n, D), dtype=torch.float64, device=DEV)
        lse = torch.full((U, G, n), -math.inf, dtype=torch.float64, device=DEV)
        acc = s["acc"].double() if s["acc"] is not None else None
        for u in range(U):
            a, b = off[u], off[u + 1]
            N = b - a
            k, v = s["K"][a:b].double(), s["V"][a:b].double()
            P = 0
            if case["op"] == "shared":
                p0, p1 = s["pre_host"][s["unit_prefix"][u]], s["pre_host"][s["unit_prefix"][u] + 1]
                P = p1 - p0
                k, v = torch.cat([s["PK"][p0:p1].double(), k]), torch.cat([s["PV"][p0:p1].double(), v])
            p = torch.arange(P + N, device=DEV)
            newest = P + N - 1
            if s["pos"] is not None:
                p, newest = s["pos"][a:b].long(), int(3 * (N - 1) + 1)
            for t in range(n):
                at = newest - (n - 1 - t)
                seen = p <= at
                if case["local"]:
                    seen &= (p > at - case["local"]) | (p < case["sinks"])
                if s["keep"] is not None:
                    seen &= s["keep"][a:b] == 1
                i = seen.nonzero()[:, 0]
                if i.numel() == 0:
                    continue
                z = s["Q"][u, :, t].double() @ k[i].T / D ** 0.5
                lse[u, :, t] = torch.logsumexp(z, -1)
                w = torch.softmax(z, -1)
                out[u, :, t] = w @ v[i]
                if acc is not None:
                    mine = i >= P
                    acc[a + i[mine] - P] += w.sum(0)[mine]
        return {"out": out, "lse": lse, **({"acc": acc} if acc is not None else {})}
    if case["op"] == "evict":
        acc = s["acc"].double().cpu()
        live = s["live"].cpu() if s["live"] is not None else torch.ones(off[-1], dtype=torch.uint8)
        pos = s["pos"].long().cpu() if s["pos"] is not None else None
        keep = torch.zeros(off[-1], dtype=torch.uint8)
        free = torch.full((off[-1],), -1, dtype=torch.int32)
        n_free = torch.zeros(U, dtype=torch.int32)
        for u in range(U):
            a, b = off[u], off[u + 1]
            p = pos[a:b] if pos is not None else torch.arange(b - a)
            there = live[a:b].nonzero()[:, 0]
            newest = p[there].max() if there.numel() else 0
            fixed = (p[there] < case["sinks"]) | (p[there] > newest - case["recent"])
            ranked = there[~fixed]
            best = ranked[torch.sort(acc[a:b][ranked], descending=True, stable=True).indices[: case["budget"]]]
            keep[a + there[fixed]] = 1
            keep[a + best] = 1
            gone = (keep[a:b] == 0).nonzero()[:, 0]
            free[a:a + gone.numel()] = gone.int()
            n_free[u] = gone.numel()
        return {"keep": keep, "free": free, "n_free": n_free, "acc": torch.where(keep == 1, acc, 0.0)}
    K, V, acc = s["K"].double(), s["V"].double(), s["acc"].double()
    keep, pos = s["keep"].clone(), s["pos"].clone()
    free, left = torch.full_like(s["free"], -1), s["n_free"].clone()
    for u in range(U):
        a, x, y = off[u], s["new_host"][u], s["new_host"][u + 1]
        to = a + s["free"][a:a + y - x].long()
        K[to], V[to], pos[to] = s["K_new"][x:y].double(), s["V_new"][x:y].double(), s["pos_new"][x:y]
        keep[to], acc[to] = 1, 0.0
        left[u] -= y - x
        free[a:a + case["free"] - (y - x)] = s["free"][a + y - x:a + case["free"]]
    return {"K": K, "V": V, "keep": keep, "pos": pos, "acc": acc, "free_out": free, "n_free_out": left}


def _inputs_of(case, seed):
    """The inputs alone, without the framework's objects."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was
