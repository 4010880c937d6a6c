"""Build libmqa_topk.so (the HIP kernels and the C ABI) in-tree for gfx950."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB_DIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIB_DIR, "libmqa_topk.so")
SOURCES = ["fused.hip", "dense.hip", "probe.hip", "api.hip", "kvcache.hip", "attend.hip",
           "attend_narrow.hip", "attend_list.hip", "attend_wide.hip", "attend_api.hip"]
HEADERS = ["common.h", "launch.h", "attend.h", "attend_tiles.h"]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
         # packed fp32 VALU forms are kept out of the generated code
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include")]


def run(args: list[str]) -> None:
    res = subprocess.run([hipcc()] + args, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + res.stdout + res.stderr)


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + \
           [os.path.join(ROOT, "include", h) for h in ("mqa_topk.h", "mqa_attend.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = True) -> str:
    """Compile the library (always when force, else only when missing/stale)."""
    if not force and not stale():
        return LIB
    os.makedirs(LIB_DIR, exist_ok=True)
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, name + ".o") for name in SOURCES]
        with concurrent.futures.ThreadPoolExecutor(min(len(SOURCES), os.cpu_count() or 1, 8)) as pool:
            list(pool.map(lambda i: run(FLAGS + ["-c", os.path.join(CSRC, SOURCES[i]), "-o",
                                                 objects[i]]), range(len(SOURCES))))
        run(["--offload-arch=gfx950", "-shared", "-fPIC", "-o", LIB + ".tmp"] + objects)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True))
