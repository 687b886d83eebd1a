"""Builds the HIP library liblrsort.so in-tree for gfx950 with hipcc.

Run ``python -m sorting_lsd_radix_sort_amd.build``; ``__graft_entry__.build()``
calls :func:`build` too.  The library is two translation units, compiled side
by side: the sort (``csrc/lrsort.hip`` with the kernels of ``csrc/kernels.hpp``)
and the row operators (``csrc/rows.hip`` with those of ``csrc/row_kernels.hpp``
and ``csrc/group_kernels.hpp``).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = [os.path.join(PKG, "csrc", "lrsort.hip"), os.path.join(PKG, "csrc", "rows.hip")]
DEPS = SOURCES + [os.path.join(PKG, "csrc", "kernels.hpp"), os.path.join(PKG, "csrc", "row_kernels.hpp"),
                  os.path.join(PKG, "csrc", "group_kernels.hpp"),
                  os.path.join(ROOT, "include", "lrsort.h"), os.path.join(ROOT, "include", "lrsort_prof.h"),
                  os.path.join(ROOT, "include", "lrsort_rows.h")]
LIB = os.path.join(PKG, "liblrsort.so")
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found; the HIP library cannot be built")


def command(args: list[str]) -> list[str]:
    return [hipcc(), "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
            # packed fp32 instructions stay off
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(ROOT, "include")] + args


def _wait(cmd: list[str], proc: subprocess.Popen, verbose: bool) -> None:
    out, err = proc.communicate()
    noise = "is not a recognized feature for this target"
    msgs = [ln for ln in (out + err).splitlines() if noise not in ln]
    if proc.returncode != 0:
        raise RuntimeError("hipcc failed: %s\n%s" % (" ".join(cmd), "\n".join(msgs)))
    if verbose and msgs:
        print("\n".join(msgs))


def build(verbose: bool = False) -> str:
    """Compiles liblrsort.so (always recompiles) and returns its path."""
    tmp = LIB + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as objs:
        obj = [os.path.join(objs, os.path.basename(s) + ".o") for s in SOURCES]
        steps = [[command(["-c", "-o", o, s]) for o, s in zip(obj, SOURCES)], [command(["-shared", "-o", tmp] + obj)]]
        for cmds in steps:
            if verbose:
                print("\n".join(" ".join(c) for c in cmds), flush=True)
            procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True) for c in cmds]
            try:
                for cmd, proc in zip(cmds, procs):
                    _wait(cmd, proc, verbose)
            finally:
                for proc in procs:  # after a failure, none is left running
                    if proc.poll() is None:
                        proc.kill()
                        proc.communicate()
    os.replace(tmp, LIB)
    return LIB


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(d) > t for d in DEPS)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
