"""Build the sm_100a shared library ``libfa_b200.so`` in-tree with nvcc.

    python -m exact_io_aware_93_b200.build [--verbose]

The library statically links the CUDA runtime and reaches the driver's
tensor-map encoder through the runtime's entry-point query, so it loads on a
machine without a GPU (the exported symbols can be inspected there) and needs
only the NVIDIA driver at run time.
"""
from __future__ import annotations

import concurrent.futures
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIB_NAME = "libfa_b200.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
# the same sources compiled with FA_CHECKS: every kernel bounds-checks its TMA coordinates
# and global indices and reports a violation in the device status word (include/fa.h)
CHECKS_LIB_PATH = os.path.join(PKG, "libfa_b200_checks.so")
SOURCES = ["fa_api.cu", "fa_cache.cu", "fa_paged.cu", "fa_paged_bf16.cu", "fa_paged_bf16_e4m3.cu", "fa_paged_f16.cu",
           "fa_paged_f16_e4m3.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa_b200.so")
    return cand


def _deps():
    out = []
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh", ".h")):
            out.append(os.path.join(CSRC, f))
    out.append(os.path.join(os.path.dirname(PKG), "include", "fa.h"))
    return out


def up_to_date(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(p) <= t for p in _deps())


# Kernels whose warpgroups rebalance registers with setmaxnreg: the split assumes that ptxas
# gives every instantiation exactly the launch allocation named by the constant.
# (Keys are patterns of mangled names.)
REG_CONTRACT = {
    "fa_fwd_kernel": ("fa_fwd_kernel.cuh", "kLaunchRegs"),
    "fa_bwd_main_kernel": ("fa_bwd_kernel.cuh", "kBwdLaunchRegs"),
    "fa_paged_kernel.*ELb0E": ("fa_paged_kernel.cuh", "kPagedLaunchRegs"),
    "fa_paged_kernel.*ELb1E": ("fa_paged_kernel.cuh", "kPagedLaunchRegsConv"),
}


def _constant(header: str, name: str) -> int:
    with open(os.path.join(CSRC, header)) as f:
        m = re.search(r"constexpr\s+uint32_t\s+" + name + r"\s*=\s*(\d+)", f.read())
    if not m:
        raise RuntimeError(f"{name} not found in {header}")
    return int(m.group(1))


def ptxas_registers(log: str):
    """(mangled entry name, registers) for every entry function in a `-Xptxas -v` report."""
    out, current = [], None
    for line in log.splitlines():
        m = re.search(r"Compiling entry function '([^']+)'", line)
        if m:
            current = m.group(1)
            continue
        m = re.search(r"Used (\d+) registers", line)
        if m and current is not None:
            out.append((current, int(m.group(1))))
            current = None
    return out


def check_register_contract(log: str) -> None:
    """Fail when a setmaxnreg kernel was compiled to a register count other than its launch
    allocation: the warpgroups' register split would then not add up."""
    regs = ptxas_registers(log)
    bad = []
    for kernel, (header, const) in REG_CONTRACT.items():
        want = _constant(header, const)
        found = [(name, n) for name, n in regs if re.search(kernel, name)]
        if not found:
            bad.append(f"{kernel}: no instantiation in the ptxas report")
        bad += [f"{name}: {n} registers, the split assumes {want}" for name, n in found if n != want]
    if bad:
        raise RuntimeError("register contract broken:\n  " + "\n  ".join(bad))


def _compile(src: str, obj: str, defines):
    """One source to one object; (command, ptxas report) or a RuntimeError with nvcc's output."""
    cmd = [_nvcc(), *ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v", *defines,
           "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    return cmd, res.returncode, res.stdout + res.stderr


def _build_one(path: str, defines, log_name: str, verbose: bool) -> None:
    """Compile every source (at the same time, one nvcc each) and link the library."""
    tmp = f"{path}.{os.getpid()}.tmp"
    objs = [f"{tmp}.{s}.o" for s in SOURCES]
    try:
        with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
            done = list(pool.map(lambda a: _compile(a[0], a[1], defines), zip(SOURCES, objs)))
        if all(rc == 0 for _, rc, _ in done):
            cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "static", *objs, "-o", tmp]
            res = subprocess.run(cmd, capture_output=True, text=True)
            done.append((cmd, res.returncode, res.stdout + res.stderr))
    finally:
        for o in objs:
            if os.path.exists(o):
                os.unlink(o)
    report = "".join(" ".join(cmd) + "\n" + text for cmd, _, text in done)
    log = os.path.join(PKG, log_name)
    with open(log, "w") as f:
        f.write(report)
    bad = [text for _, rc, text in done if rc != 0]
    if bad:
        raise RuntimeError(f"nvcc failed (see {log}):\n{bad[0][-4000:]}")
    try:
        check_register_contract(report)
    except RuntimeError:
        os.unlink(tmp)
        raise
    os.replace(tmp, path)
    if verbose:
        print(report)


def build(force: bool = False, verbose: bool = False, checks: bool = True) -> str:
    """Build the release library and (checks=True) the checking build; returns the release
    library's path."""
    jobs = [(LIB_PATH, [], "build.log")]
    if checks:
        jobs.append((CHECKS_LIB_PATH, ["-DFA_CHECKS"], "build_checks.log"))
    jobs = [j for j in jobs if force or not up_to_date(j[0])]
    with concurrent.futures.ThreadPoolExecutor(max_workers=2) as pool:
        for f in [pool.submit(_build_one, *j, verbose) for j in jobs]:
            f.result()
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB_PATH)
