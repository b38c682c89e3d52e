"""Compile the HIP libraries for gfx950 in-tree (hipcc, no GPU needed).

Each translation unit is compiled to an object in its own hipcc process (in
parallel), then the objects are linked into ``librans_hip.so`` (the coder) and
``liblic_layers.so`` (the network operators around it).
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "librans_hip.so")
SOURCES = ["rans_prep.hip", "rans_encode.hip", "rans_decode.hip", "rans_tables.hip", "rans_latent.hip",
           "rans_interleaved.hip", "rans_noalloc.hip", "rans_abi.hip"]
LAYERS_LIBRARY = os.path.join(PKG, "liblic_layers.so")
LAYERS_SOURCES = ["layers_norm.hip", "layers_rms.hip", "layers_rotary.hip", "layers_attention.hip",
                  "layers_attention_f32.hip", "layers_attention_f16.hip",
                  "layers_attention_bf16.hip", "layers_linear.hip", "layers_linear_f32.hip",
                  "layers_linear_f16.hip", "layers_linear_bf16.hip", "layers_clip.hip"]
ARCH = os.environ.get("RANS_HIP_ARCH", "gfx950")

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # packed fp32 instructions stay off: only the compiler's scalar forms are used
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _jobs(sources: int) -> int:
    try:
        n = len(os.sched_getaffinity(0))
    except AttributeError:  # pragma: no cover
        n = os.cpu_count() or 1
    return max(1, min(n, 16, sources))


def build(verbose: bool = False, extra=()) -> str:
    libraries = {LIBRARY: SOURCES, LAYERS_LIBRARY: LAYERS_SOURCES}
    with tempfile.TemporaryDirectory(prefix="rans_build_") as tmpdir:
        def run(cmd):
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)

        def compile_one(name):
            obj = os.path.join(tmpdir, name + ".o")
            run(["hipcc", *FLAGS, "-I", INCLUDE, "-I", CSRC, *extra, "-c",
                 os.path.join(CSRC, name), "-o", obj])
            return obj

        names = [s for sources in libraries.values() for s in sources]
        with ThreadPoolExecutor(max_workers=_jobs(len(names))) as ex:
            objs = dict(zip(names, ex.map(compile_one, names)))
        for library, sources in libraries.items():
            tmp = f"{library}.tmp{os.getpid()}"
            run(["hipcc", f"--offload-arch={ARCH}", "-shared", "-fPIC",
                 *(objs[s] for s in sources), "-o", tmp])
            os.replace(tmp, library)
    return LIBRARY


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
