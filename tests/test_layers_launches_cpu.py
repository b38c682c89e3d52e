"""The network operators' launches without a GPU: a stand-in takes the place of the HIP runtime and
looks at each launch (`host_runtime.cpp`), in a process of its own, where no torch has loaded the other."""
from __future__ import annotations

import json
import os
import subprocess
import sys

import pytest

from test_layers_abi_cpu import NORM, ROTARY, attention_args, layers  # noqa: F401 - a fixture

HERE = os.path.dirname(os.path.abspath(__file__))
NAMES = ("launches", "blocks", "too_many_threads", "too_much_lds", "attributes")

CHILD = """
import ctypes, json, sys
stand_in = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
out, counts = [], (ctypes.c_int64 * 5)()
for device, refuses, name, kind, args in json.load(sys.stdin):
    stand_in.stand_in_device(device)
    stand_in.stand_in_refuses(refuses)
    ctype = {"b": lambda v: bytes.fromhex(v), "p": ctypes.c_void_p, "q": ctypes.c_int64, "i": ctypes.c_int32,
             "f": ctypes.c_float, "Q": ctypes.c_uint64, "d": ctypes.c_double}
    before = list(counts)
    rc = getattr(lib, name)(*(ctype[k](v) for k, v in zip(kind, args)))
    stand_in.stand_in_counts(counts)
    out.append([rc] + [a - b for a, b in zip(counts, before)])
print(json.dumps(out))
"""


@pytest.fixture(scope="module")
def stand_in(layers, tmp_path_factory):  # noqa: F811
    """calls -> [{rc, launches, ...}] of a process that makes them in order."""
    so = tmp_path_factory.mktemp("runtime") / "host_runtime.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    os.path.join(HERE, "host_runtime.cpp"), "-o", str(so)], check=True)

    def calls(*jobs):
        r = subprocess.run([sys.executable, "-c", CHILD, str(so), layers.LIBRARY], input=json.dumps(jobs), text=True,
                           capture_output=True, timeout=120)
        assert r.returncode == 0, r.stderr
        return [dict(zip(("rc", *NAMES), row)) for row in json.loads(r.stdout)]

    return calls


def attention(layers, backward=0, device=0, refuses=0, **kw):  # noqa: F811
    name = "lic_attention_backward" if backward else "lic_attention_forward"
    return [device, refuses, name, "bpQp", [attention_args(layers, **kw).hex(), 256, 1 << 46, 0]]


def norm(backward=0, device=0, **kw):
    a = {**NORM, "dy": 256, "dx": 512, "bytes": 1 << 46, **kw}
    if backward:
        return [device, 0, "lic_group_norm_backward", "pqqpqqiqiiippiipppqqpppQp",
                [a["dy"], a["xs"], a["xr"], a["x"], a["xs"], a["xr"], a["n"], a["s"], a["c"], a["g"], a["dtype"],
                 a["w"], a["b"], a["pdtype"], a["act"], a["mean"], a["rstd"], a["dx"], a["xs"], a["xr"], 4096, 8192,
                 a["ws"], a["bytes"], 0]]
    return [device, 0, "lic_group_norm_forward", "pqqiqiiippifipqqpppQp",
            [a["x"], a["xs"], a["xr"], a["n"], a["s"], a["c"], a["g"], a["dtype"], a["w"], a["b"], a["pdtype"],
             a["eps"], a["act"], a["y"], a["ys"], a["yr"], a["mean"], a["rstd"], a["ws"], a["bytes"], 0]]


def rotary(layers, **kw):  # noqa: F811
    a = {**ROTARY, **kw}
    args = layers._ROTARY.pack(*(a[k] for k in ("q", "k", "qo", "ko", "cos", "sin", "pos", "status", "step")),
                               *a["strides"], *(a[k] for k in ("b", "s", "h", "kh", "d", "r", "rows", "dtype",
                                                               "inter", "inv")))
    return [0, 0, "lic_rotary", "bp", [args.hex(), 0]]


def every_kernel(layers, device):  # noqa: F811
    """Calls of all types, widths, kinds of masks and loads, of few and of many queries; norms of one launch."""
    jobs = []
    for dtype in (0, 1, 2):
        for d in (32, 64, 96, 128, 30, 60, 90, 126):
            odd = {"strides": (4097, 65, 17) * 8}
            for mask in ({}, {"mask": 256, "mask_strides": (0, 0, 512, 1)}, {"mask": 256, "mask_strides": (0, 0, 1, 512)}):
                for sizes in (dict(b=64, n=512, m=512), dict(b=2, n=3, m=900), dict(b=64, n=512, m=512, right=0)):
                    for layout in ({}, odd):
                        for backward in (0, 1):
                            jobs.append(attention(layers, backward, device, dtype=dtype, d=d, **sizes, **mask, **layout))
        for act in range(4):
            for backward in (0, 1):  # 96 and 125 KiB of values in one launch
                s = (384 if backward else 1000) * (2 if dtype else 1)
                jobs.append(norm(backward, device, n=256, c=32, g=1, s=s, dtype=dtype, act=act))
    return jobs


@pytest.mark.slow
def test_each_device_is_told_of_large_kernels(layers, stand_in):  # noqa: F811
    """What needs more than 64 KiB of LDS is allowed it on whatever device a call runs, once."""
    there = [every_kernel(layers, device) for device in (0, 1, 0, 5)]
    n = len(there[0])
    rows = stand_in(*(job for jobs in there for job in jobs))
    assert all(r["rc"] == 0 and r["launches"] >= 1 for r in rows)
    assert sum(r["too_much_lds"] for r in rows) == 0
    told = [sum(r["attributes"] for r in rows[i:i + n]) for i in range(0, 4 * n, n)]
    assert told[0] == told[1] == told[3] > 0 and told[2] == 0


def test_a_device_without_the_lds_is_an_error(layers, stand_in):  # noqa: F811
    jobs = []
    for refuses in (1, 0):  # and it is asked again
        jobs += [attention(layers, backward, 0, refuses, b=64, n=512, m=512, d=128) for backward in (0, 1)]
        jobs.append(norm(n=256, c=32, g=1, s=1000))
        jobs[-1][1] = refuses
    rows = stand_in(*jobs)
    assert [r["rc"] for r in rows] == [-8] * 3 + [0] * 3
    assert sum(r["too_much_lds"] for r in rows) == 0 and sum(r["launches"] for r in rows[:3]) == 0

def test_no_launch_has_more_threads_than_it_can(layers, stand_in):  # noqa: F811
    """Past 2^32 threads a call is several launches."""
    few, many = dict(b=1 << 20, n=1, m=1, h=17, kv=17, d=8), dict(b=1 << 20, n=200, m=200, h=32, kv=32, d=8)
    wide = (1 << 50, 1 << 20, 1 << 10) * 8
    jobs, least = [], []
    for sizes, blocks in ((few, 17 << 20), (many, 2 * (32 << 20))):
        for backward in (0, 1):
            jobs.append(attention(layers, backward, strides=wide, **sizes))
            least.append(blocks * (2 if backward else 1))
    jobs.append(rotary(layers, strides=wide[:12], s=1 << 20, h=1366, kh=0, d=6, r=6, rows=1 << 20))
    least.append((1 << 20) * 1366 * 3 // 256)
    jobs.append([0, 0, "lic_rotary_table", "pqiiddddddppp",
                 [256, 1 << 31, 1, 64, 1e4, 1.0, 0.0, 0.0, 0.0, 1.0, 512, 1024, 0]])
    least.append((1 << 31) * 32 // 256)
    for backward in (0, 1):
        jobs.append(norm(backward, n=65535, c=192, g=192, s=4096, dtype=2))  # one launch of 512 threads a group
        least.append(65535 * 192)
        jobs.append(norm(backward, n=65535, c=65533, g=1, s=9))              # single channels, three launches
        least.append(2 * 65535 * (65533 // 256))
    for row, blocks in zip(stand_in(*jobs), least):
        assert row["rc"] == 0 and row["too_many_threads"] == 0 and row["launches"] >= 2 and row["blocks"] >= blocks


def test_sizes_that_no_count_holds_are_refused(layers, stand_in):  # noqa: F811
    row, = stand_in(rotary(layers, b=1 << 20, s=1 << 20, h=65536, kh=65536, d=65536, r=2, rows=1 << 20))
    assert row["rc"] == -1 and row["launches"] == 0
