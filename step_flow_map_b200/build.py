"""Build the C-ABI library libflashmap_b200.so for sm_100a with nvcc.

Usage: python -m step_flow_map_b200.build [--verbose]
The library lands next to this file, so it travels with the source tree.
"""
from __future__ import annotations

import hashlib
import os
import re
import subprocess
import sys
import time

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libflashmap_b200.so")
SRCS = [os.path.join(HERE, "csrc", f) for f in ("fm_api.cu", "fm_cache_api.cu")]
OBJ_DIR = os.path.join(HERE, "_build")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def compile_command(src: str, obj: str, extra=()) -> list:
    return [
        nvcc(), "-O3", "-std=c++17", "-c", "-Xcompiler", "-fPIC",
        "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
        "-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc"),
        "--expt-relaxed-constexpr", "--extended-lambda",
        *extra, src, "-o", obj,
    ]


def link_command(objs, out: str = LIB) -> list:
    return [nvcc(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs, "-o", out]


def sources() -> list:
    csrc = os.path.join(HERE, "csrc")
    files = [os.path.join(csrc, f) for f in os.listdir(csrc)]
    files += [os.path.join(ROOT, "include", "flashmap.h"), os.path.join(HERE, "build.py")]
    return files


def object_file(src: str, extra=()) -> str:
    """Where a source's object is kept: one file for every way to compile it."""
    cmd = "\n".join(compile_command(src, "", extra)).replace(ROOT, "")
    return os.path.join(OBJ_DIR, f"{os.path.basename(src)}.{hashlib.sha1(cmd.encode()).hexdigest()[:12]}.o")


def _linked() -> str:
    return os.path.join(OBJ_DIR, os.path.basename(LIB) + ".linked")


def up_to_date(extra=()) -> bool:
    """Whether the library is newer than its sources and, where it is known what it
    was linked from, was compiled with these flags."""
    if not os.path.exists(LIB):
        return False
    if os.path.exists(_linked()):
        with open(_linked(), encoding="utf-8") as f:
            if f.read().split() != [os.path.basename(object_file(s, extra)) for s in SRCS]:
                return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in sources())


def _newest(src: str, seen=None) -> float:
    """Latest change of a source, of the headers it includes and of this file."""
    seen = set() if seen is None else seen
    seen.add(src)
    t = max(os.path.getmtime(src), os.path.getmtime(os.path.join(HERE, "build.py")))
    for name in re.findall(r'#include "([^"]+)"', open(src, encoding="utf-8").read()):
        for d in (os.path.dirname(src), os.path.join(ROOT, "include")):
            f = os.path.join(d, name)
            if os.path.exists(f) and f not in seen:
                t = max(t, _newest(f, seen))
    return t


def _run(cmds, verbose: bool) -> None:
    """Run the commands side by side; raise if one fails."""
    if verbose:
        for c in cmds:
            print(" ".join(c), flush=True)
    procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
             for c in cmds]
    outs = [p.communicate()[0] for p in procs]
    bad = any(p.returncode != 0 for p in procs)
    if verbose or bad:
        sys.stderr.write("".join(outs))
    if bad:
        raise RuntimeError("nvcc failed building libflashmap_b200.so")


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile every source (side by side) and link the library.  Objects
    newer than their source and its headers, and compiled with the same flags,
    are kept unless `force`.  Every file appears under its name when it is whole, so
    processes that build at once do no harm."""
    if not force and up_to_date(extra):
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    start = time.time()            # a source that changes from here on is newer than what is made of it
    tmp = f".{os.getpid()}.tmp"
    objs = [object_file(src, extra) for src in SRCS]
    stale = [(src, obj) for src, obj in zip(SRCS, objs)
             if force or not os.path.exists(obj) or os.path.getmtime(obj) < _newest(src)]
    try:
        _run([compile_command(src, obj + tmp, extra) for src, obj in stale], verbose)
        for _, obj in stale:
            _appear(obj, tmp, start)
        _run([link_command(objs, LIB + tmp)], verbose)
        with open(_linked() + tmp, "w", encoding="utf-8") as f:
            f.write(" ".join(map(os.path.basename, objs)))
        _appear(LIB, tmp, start)
        _appear(_linked(), tmp, start)
    finally:
        for f in [*objs, LIB, _linked()]:
            if os.path.exists(f + tmp):
                os.remove(f + tmp)
    return LIB


def _appear(path: str, tmp: str, when: float) -> None:
    os.utime(path + tmp, (when, when))
    os.replace(path + tmp, path)


if __name__ == "__main__":
    v = "--verbose" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else []
    print(build(force=True, verbose=v, extra=extra))
