"""How the backward of the windowed attention is cut into units, against the workspace
that is sized without knowing the documents (CPU: the host functions, compiled alone)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from conftest import ROOT



@pytest.fixture(scope="module")
def units(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    so = str(tmp_path_factory.mktemp("units") / "units.so")
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "-Xcompiler", "-fPIC",
                        "-I", os.path.join(ROOT, "include"), "-I",
                        os.path.join(ROOT, "long_context_sequence_head_gb300", "csrc"), "-shared", "-o", so,
                        os.path.join(ROOT, "tests", "window_units.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(so)
    i64, i32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
    lib.window_bounds.argtypes = [i64, i64, i64, i32, i32, i64, vp]
    lib.window_bounds.restype = lib.window_units.restype = None
    lib.window_units.argtypes = [i64, i32, i32, vp, i32, i32, i64, vp]
    lib.window_workspace.argtypes = [i64, i64, i32, i32, i64, i64, i32, i32]
    lib.window_workspace.restype = ctypes.c_size_t
    return lib


def counts(lib, N, window, sinks, cu, tile, nprob):
    """What the call takes and what there is room for: units, slots, joins, chunks."""
    need, room = (ctypes.c_int64 * 4)(), (ctypes.c_int64 * 4)()
    docs = len(cu) - 1 if cu else 0
    arr = (ctypes.c_int32 * len(cu))(*cu) if cu else None
    lib.window_units(N, window, sinks, arr, docs, tile, nprob, need)
    lib.window_bounds(N, window, sinks, docs, tile, nprob, room)
    return list(need), list(room)


def layout(rng, N, window, sinks):
    """Documents of lengths where the bounds are tight, and of any."""
    kind, cu = rng.randrange(6), [0]
    tight = rng.choice([window + 1, window + 129, window + rng.randrange(1, 300), 128 * rng.randrange(1, 9),
                        window + sinks + 1, window + 127 + rng.randrange(3), 64 * rng.randrange(1, 20) + 1])
    while cu[-1] < N:
        step = (tight if kind < 3 else rng.choice([0, 1, tight, rng.randrange(1, 2 * tight + 2)]) if kind == 3 else
                rng.randrange(N + 1) if kind == 4 else int(N ** rng.random()))
        cu.append(min(N, cu[-1] + step))
        if len(cu) > 3000:
            cu.append(N)
    if rng.random() < 0.3:
        cu[1:1] = [min(cu[1], rng.randrange(130))]
    return cu


@pytest.mark.parametrize("seed", range(8))
def test_every_call_fits_its_workspace(units, seed):
    rng = random.Random(seed)
    for _ in range(1500):
        N = int(round(2 ** rng.uniform(0, 17)))
        window = min(N, int(round(2 ** rng.uniform(0, 12))))
        sinks = 0 if window == N else min(N, rng.choice([0, 1, 4, 33, 64, 65, 130, 200, 320, 321, 513, 5000, 9000,
                                                         rng.randrange(400)]))
        cu = layout(rng, N, window, sinks) if rng.random() < 0.75 else None
        tile, nprob = rng.choice([64, 128]), rng.choice([1, 2, 8, 16, 64, 300])
        need, room = counts(units, N, window, sinks, cu, tile, nprob)
        assert all(a <= b for a, b in zip(need, room)), (N, window, sinks, cu and len(cu), tile, nprob, need, room)


@pytest.mark.parametrize("N,window,sinks,docs,tile", [
    (65536, 64, 320, 500, 128), (131072, 32, 320, 2000, 128), (65536, 100, 130, 600, 128), (65536, 1024, 4, 60, 128),
    (65536, 1000, 400, 64, 128), (32768, 256, 4, 100, 64), (65536, 4096, 4, 0, 128), (65536, 64, 65535, 0, 128)])
def test_slots_are_not_many_times_what_a_call_takes(units, N, window, sinks, docs, tile):
    """Against the largest of many layouts, drawn or even, that the documents may have."""
    rng = random.Random(N + docs)
    most = 0
    for i in range(200 if docs else 1):
        if not docs:
            cu = None
        elif i % 2:
            # even documents, the rest without tokens; all begin at a tile's end, so that their
            # sinks lie in as many tiles as they can
            step = (window + rng.choice([0, tile, tile * rng.randrange(40)])) // tile * tile + tile
            cu = [0] + sorted(min(N, tile - 1 + j * step) for j in range(docs - 1)) + [N]
        else:
            cu = [0] + sorted(rng.randrange(N + 1) for _ in range(docs - 1)) + [N]
        need, room = counts(units, N, window, sinks, cu, tile, 8)
        most = max(most, need[1])
    assert room[1] <= 2.5 * most + 8


def test_workspace(units):
    """Bytes: eight problems of four heads."""
    size = lambda *a: units.window_workspace(8, a[0], 4, 1, *a[1:], 2)
    base = size(65536, 64, 0, 500)
    assert size(65536, 64, 320, 500) - base <= 1.5 * 2 ** 30
    assert size(65536, 64, 65535, 0) - base <= 2 ** 20  # walks that are never cut have no sums
