"""Host-side checks of the attention and weight-eviction calls (no GPU needed):
argument checks of the C entry points and the binding, struct layouts, and the
oracle's definitions pinned by hand."""
import ctypes
import glob
import os
import re
import subprocess
import sys
import tempfile

import numpy as np
import pytest
import torch

import decode_kv_cache_eviction_b200 as rkv
from decode_kv_cache_eviction_b200 import _binding as B
from oracle import rkv_oracle as ora

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    from decode_kv_cache_eviction_b200 import build
    build.build()


def test_struct_layouts_match_header():
    fields = {"rkv_attention": B.RkvAttention, "rkv_prefix": B.RkvPrefix}
    lines = []
    for name, s in fields.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in s._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "rkv.h"\nint main(void){' + "".join(lines) + "return 0;}"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                        c, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for s in fields.values():
        want.append(ctypes.sizeof(s))
        want += [getattr(s, f).offset for f, _ in s._fields_]
    assert got == want


def test_null_arguments():
    L = rkv.lib()
    n = None
    att = B.RkvAttention()
    assert L.rkv_attend(n, n, n, n) == B.RKV_ERR_INVALID_ARG
    assert L.rkv_attend(n, n, ctypes.byref(att), n) == B.RKV_ERR_INVALID_ARG
    assert L.rkv_attend_shared(n, n, n, ctypes.byref(att), n) == B.RKV_ERR_INVALID_ARG
    assert L.rkv_evict_accumulated(n, n, n, n, n, 4, n, 0, n, n, n, n, n, n, n) == B.RKV_ERR_INVALID_ARG
    assert L.rkv_fill_slots_ex(n, n, n, n, n, n, n, n, n, n, n, n, n, n, n, n, n) == B.RKV_ERR_INVALID_ARG


def test_prefix_plan_arguments():
    kv = torch.zeros((10, 128), dtype=torch.bfloat16)
    for off, up in (([1, 10], [0]), ([0, 10, 5], [0]), ([0, 10], [1]), ([0, 10], [-2]), ([0], [0])):
        with pytest.raises(ValueError):
            rkv.Prefix(kv, kv, off, up)
    with pytest.raises(ValueError):                 # not on a GPU
        rkv.Prefix(kv, kv, [0, 10], [0, 0])


def test_batch_of_offsets_needs_a_device():
    with pytest.raises(ValueError):
        rkv.Batch(None, None, None, [0, 5])
    b = rkv.Batch(None, None, None, [0, 5], device="cpu")
    assert b.num_units == 1 and b.num_tokens == 5
    with pytest.raises(ValueError):
        rkv.Offsets([[0, 1]], "cpu")


def test_oracle_attend_by_hand():
    """Two keys along one axis: z = 1 and 0, p = e / (e + 1)."""
    d = 4
    q = np.zeros((1, 2, d))
    q[0, :, 0] = 2.0
    k = np.zeros((3, d))
    k[0, 0] = 1.0
    v = np.array([[1.0] * d, [3.0] * d, [100.0] * d])
    out, lse, p, seen = ora.attend(q, k, v, [0, 1, 2], [1, 2], live=[1, 1, 0])
    a = np.e / (np.e + 1)
    assert np.allclose(p[0], [[a, 1 - a, 0]] * 2) and np.allclose(lse, np.log(np.e + 1))
    assert np.allclose(out[0], a + 3 * (1 - a))
    assert seen.tolist() == [[True, True, False]] * 2
    # a window of one position, with and without a sink; a query before everything
    out, lse, p, _ = ora.attend(q[:, :1], k, v, [0, 1, 2], [2], local=1)
    assert np.allclose(out, 100.0)
    _, _, p, _ = ora.attend(q[:, :1], k, v, [0, 1, 2], [2], local=1, sinks=1)
    assert np.allclose(p[0, 0], [a, 0, 1 - a])
    out, lse, _, _ = ora.attend(q[:, :1], k, v, [0, 1, 2], [-1])
    assert np.all(out == 0) and np.all(np.isneginf(lse))


def test_oracle_attend_matches_importance():
    """Without masks, the mean of p over queries and heads is the importance."""
    rng = np.random.default_rng(0)
    Q, K = rng.standard_normal((2, 3, 8)), rng.standard_normal((20, 8))
    _, _, p, _ = ora.attend(Q, K, K, np.arange(20), 17 + np.arange(3))
    assert np.allclose(p, ora.attention_probs(Q, K))


def test_oracle_evict_accumulated_by_hand():
    acc = np.array([9.0, 1.0, 5.0, 5.0, np.nan, 0.0, 2.0])
    kept = lambda *a, **k: ora.evict_accumulated(acc, *a, **k).tolist()
    assert kept(range(7), [1] * 7, 1, 2) == [0, 2, 6]          # newest 6, then 9 and the first 5
    assert kept(range(7), [1] * 7, 1, 5, sinks=1) == [0, 1, 2, 3, 4, 5, 6]
    assert kept(range(7), [1] * 7, 1, 4, sinks=1) == [0, 1, 2, 3, 5, 6]   # NaN goes last
    assert kept([6, 5, 4, 3, 2, 1, 0], [1] * 7, 2, 1, sinks=1) == [0, 1, 2, 6]
    assert kept(range(7), [0, 1, 0, 1, 1, 1, 0], 1, 1) == [3, 5]
    assert kept(range(7), [0] * 7, 3, 5) == []


def host_engine(group=4, window=8, device=0):
    """An engine's Python side alone: what it refuses before the library is called."""
    eng = object.__new__(rkv.Engine)
    eng.h, eng.group, eng.window, eng.device = None, group, window, device
    return eng


def test_offsets_on_another_device_are_refused():
    """A batch of offsets alone has no K that would be checked in their place."""
    eng = host_engine()
    rows = torch.zeros(5)
    for device in ("cpu", "meta"):
        b = rkv.Batch(None, None, None, [0, 5], device=device)
        with pytest.raises(ValueError, match="offsets are on"):
            eng.evict_accumulated(b, rows, 2, rows, rows, rows)


def test_no_read_only_loads_of_what_a_running_launch_writes():
    """The second kernels of an attention call start while the first still writes its parts and
    sums.  A race cannot be shown by its results, so the source is looked at: read-only loads
    are for the caller's inputs."""
    scratch = r"__ldg\(&?p\w*\.(part_o|part_ml|pre_o|pre_ml|lse2|z|count)\b"
    files = glob.glob(os.path.join(ROOT, "decode_kv_cache_eviction_b200", "csrc", "attend*"))
    assert len(files) >= 4
    assert [(os.path.basename(f), m.group()) for f in files for m in re.finditer(scratch, open(f).read())] == []


def test_tensor_map_fault_needs_an_engine():
    L = rkv.lib()
    assert L.rkv_inject_fault(None, B.RKV_FAULT_TENSOR_MAP) == B.RKV_ERR_INVALID_ARG


def test_tensor_check_built_for_another_pytorch(tmp_path, monkeypatch):
    """It is built again although its source is older, and it does not load."""
    from decode_kv_cache_eviction_b200 import build
    so = tmp_path / "_tensors.so"
    monkeypatch.setattr(build, "TENSORS", str(so))
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        build.build()
    load = [sys.executable, "-c", f"import sys, torch; sys.path.insert(0, {str(tmp_path)!r}); import _tensors"]
    got = subprocess.run(load, capture_output=True, text=True)
    assert got.returncode != 0 and "ImportError: it was built for PyTorch 0.0.1" in got.stderr
    was = so.stat().st_mtime_ns
    build.build()
    assert so.stat().st_mtime_ns > was
    assert subprocess.run(load).returncode == 0
    was = so.stat().st_mtime_ns
    build.build()
    assert so.stat().st_mtime_ns == was


@pytest.mark.parametrize("big", [2**31, 2**32 + 5, -2**31 - 1, -2**32 + 5])
def test_numbers_beyond_32_bits_are_refused(big):
    """ctypes would pass their low 32 bits on."""
    eng = host_engine()
    b = rkv.Batch(None, None, None, [0, 5], device="cpu")
    b.device = eng.device
    q, rows = torch.zeros((1, 4, 1, 128), dtype=torch.bfloat16), torch.zeros(5)
    for kw in (dict(local=big), dict(sinks=big)):
        with pytest.raises(ValueError, match="must fit into 32 bits"):
            eng.attend(b, q, q, **kw)
    for budget, sinks in ((big, 0), (2, big)):
        with pytest.raises(ValueError, match="must fit into 32 bits"):
            eng.evict_accumulated(b, rows, budget, rows, rows, rows, sinks=sinks)
