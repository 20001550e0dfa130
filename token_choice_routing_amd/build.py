"""Builds libmoe_mi355x.so for gfx950 with hipcc, and the binding's argument checks
(_marshal.so) with g++ against torch's headers, in-tree.

    python -m token_choice_routing_amd.build

Every call compiles all sources (one hipcc process per file, in parallel) and
links the shared libraries next to this file. Without a C++ compiler or torch's
headers the HIP library is built all the same, with a warning: the binding's row
operators then refuse to run, the others do not need the checks.
"""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libmoe_mi355x.so")
SOURCES = ["api.hip", "route.hip", "permute.hip", "ffn.hip", "combine.hip", "aux.hip", "backward.hip", "validate.hip",
           "dispatch_grad.hip", "act8.hip"]
MARSHAL = os.path.join(HERE, "_marshal.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-result",
    # packed float32 VALU ops stay off: only ordinary float code is emitted
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in r.stdout.splitlines() if "packed-fp32-ops" not in l)
    return r.returncode, out


def _marshal_cmd(out):
    """g++ line of the binding's argument checks (host code: Python and torch, no GPU)."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-isystem", os.path.join(root, "include"),
            "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "marshal.cpp"), "-o", out,
            "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]


def _compile_marshal(out) -> str:
    """Compiles the argument checks; returns what went wrong ("" if nothing did)."""
    try:
        rc, text = _run(_marshal_cmd(out))
    except OSError as e:  # no such compiler
        rc, text = 1, str(e)
    return (text or f"g++ status {rc}") if rc else ""


def _install_marshal(new, problem):
    """Puts the compiled checks in place. If they did not compile, those of an earlier build
    do not stay either: they may not match the sources or torch."""
    if not problem:
        os.replace(new, MARSHAL)
        return
    if os.path.exists(MARSHAL):
        os.remove(MARSHAL)
    print(f"warning: {MARSHAL} is not built, the Python binding's row operators will refuse to run:\n{problem}",
          file=sys.stderr)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    objs, cmds = [], []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".hip", ".o"))
        objs.append(obj)
        cmds.append([HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj])
    with ThreadPoolExecutor(max_workers=min(len(cmds), os.cpu_count() or 4, 8)) as ex:
        marshal = ex.submit(_compile_marshal, MARSHAL + ".tmp")
        results = list(ex.map(_run, cmds))
    for cmd, (rc, out) in zip(cmds, results):
        if out.strip() and (verbose or rc):
            print(out, file=sys.stderr)
        if rc:
            raise RuntimeError(f"compiler failed: {' '.join(cmd)}")
    tmp = LIB + ".tmp"
    rc, out = _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs])
    if rc:
        print(out, file=sys.stderr)
        raise RuntimeError("link failed")
    os.replace(tmp, LIB)
    _install_marshal(MARSHAL + ".tmp", marshal.result())
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
