"""Build libgdr.so (the C-ABI CUDA library) in-tree with nvcc for sm_100a."""
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libgdr.so")
# Two translation units, compiled side by side.
UNITS = ("gdr_lib", "ssm_lib")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-Xptxas", "-warn-spills",
]

_INCLUDE = re.compile(r'^\s*#\s*include\s+"([^"]+)"', re.M)


def _sources(unit):
    """A unit's .cu file and every header it includes, directly or not."""
    todo, seen = [os.path.join(CSRC, unit + ".cu")], []
    while todo:
        path = todo.pop()
        if path in seen:
            continue
        seen.append(path)
        with open(path) as f:
            for name in _INCLUDE.findall(f.read()):
                for d in (CSRC, os.path.join(ROOT, "include")):
                    if os.path.exists(os.path.join(d, name)):
                        todo.append(os.path.join(d, name))
    return seen


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the units that are older than their sources and link libgdr.so; nothing where it is newer than them all."""
    if not force and os.path.exists(LIB):
        t = os.path.getmtime(LIB)
        if all(os.path.getmtime(s) <= t for unit in UNITS for s in _sources(unit)):
            return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    pid = os.getpid()
    running, objects = [], []
    for unit in UNITS:
        obj = os.path.join(CSRC, unit + ".o")
        objects.append(obj)
        if not force and os.path.exists(obj):
            t = os.path.getmtime(obj)
            if all(os.path.getmtime(s) <= t for s in _sources(unit)):
                continue
        tmp = obj + ".tmp%d.o" % pid
        cmd = [nvcc] + NVCC_FLAGS + ["-I", os.path.join(ROOT, "include"), "-c", "-o", tmp,
                                     os.path.join(CSRC, unit + ".cu")]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd))
        running.append((subprocess.Popen(cmd), tmp, obj, cmd))
    codes = [p.wait() for p, _, _, _ in running]
    for code, (_, tmp, obj, cmd) in zip(codes, running):
        if code:
            raise subprocess.CalledProcessError(code, cmd)
        os.replace(tmp, obj)
    if running or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objects):
        tmp = LIB + ".tmp%d" % pid
        subprocess.check_call([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp] + objects)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
