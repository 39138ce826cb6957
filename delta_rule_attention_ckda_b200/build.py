"""Build libckda.so (the CKDA C-ABI library) in-tree with nvcc for sm_100a."""
from __future__ import annotations

import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libckda.so")
SELFTEST_LIB = os.path.join(PKG, "libckda_selftest.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = [*ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills", "-Xptxas", "-v"]
# Kernels that move registers between their warps, by part of their name: the file and constant that
# say how many a thread is compiled to. Such a split adds up against no other number.
SPLITS = {"chain_fwd_kernel": ("kernels/gated_chain.cuh", "kRegLaunch"), "chain_bwd_kernel": ("kernels/gated_chain.cuh", "kRegLaunch")}


TARGETS = {LIB: ["ckda_api.cu", "gated_api.cu"], SELFTEST_LIB: ["selftest.cu"]}
OBJ = os.path.join(PKG, "_build")


def _inputs(src: str):
    """The files `src` is compiled from: itself and every file of this package it includes."""
    seen, todo = set(), [os.path.join(CSRC, src)]
    while todo:
        f = todo.pop()
        if f in seen:
            continue
        seen.add(f)
        for name in re.findall(r'^\s*#include "([^"]+)"', open(f).read(), re.M):
            for d in (os.path.dirname(f), CSRC, os.path.join(ROOT, "include")):
                if os.path.exists(os.path.join(d, name)):
                    todo.append(os.path.normpath(os.path.join(d, name)))
                    break
    return seen | {os.path.abspath(__file__)}


def _check_registers(log: str) -> None:
    """The compiler's report (-Xptxas -v) against SPLITS."""
    entry = None
    for line in log.splitlines():
        m = re.search(r"Compiling entry function '(\S+)'", line)
        if m:
            entry = m.group(1)
        m = re.search(r"Used (\d+) registers", line)
        if m and entry:
            for part, (file, name) in SPLITS.items():
                if part in entry:
                    want = int(re.search(rf"\b{name} = (\d+)", open(os.path.join(CSRC, file)).read()).group(1))
                    if int(m.group(1)) != want:
                        raise RuntimeError(f"{entry} was compiled to {m.group(1)} registers a thread; its split between warps needs {want}")
            entry = None


def _newer(out: str, files) -> bool:
    return os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(f) for f in files)


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)


def _build_one(lib: str, sources, force: bool, verbose: bool, extra) -> None:
    inputs = {src: _inputs(src) for src in sources}
    if not force and _newer(lib, set().union(*inputs.values())):
        return
    os.makedirs(OBJ, exist_ok=True)
    objects, procs = [], []
    for src in sources:                        # one object per source, compiled side by side
        obj = os.path.join(OBJ, src + ".o")
        objects.append(obj)
        if not force and _newer(obj, inputs[src]):
            continue
        tmp = obj + f".tmp{os.getpid()}"
        cmd = [NVCC, *FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c",
               os.path.join(CSRC, src), "-o", tmp]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        log = open(tmp + ".log", "w+")
        procs.append((subprocess.Popen(cmd, stderr=log), log, tmp, obj, cmd))
    failed = None
    for p, log, tmp, obj, cmd in procs:
        p.wait()
        with log:
            log.seek(0)
            said = log.read()
        os.remove(log.name)
        for line in said.splitlines():
            if verbose or not re.search(r"^ptxas info|bytes stack frame|^$", line):
                print(line, file=sys.stderr)
        try:
            if p.returncode != 0:
                raise subprocess.CalledProcessError(p.returncode, cmd)
            _check_registers(said)
            os.replace(tmp, obj)
        except (subprocess.CalledProcessError, RuntimeError) as e:
            failed = e
    if failed:
        raise failed
    tmp = lib + f".tmp{os.getpid()}"
    _run([NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objects, "-o", tmp], verbose)
    os.replace(tmp, lib)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Build libckda.so and the test-only libckda_selftest.so; returns libckda.so's path."""
    for lib, sources in TARGETS.items():
        _build_one(lib, sources, force, verbose, extra)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
