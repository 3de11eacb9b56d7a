"""Builds libokls.so (HIP for gfx950) in-tree with hipcc."""
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCES = ["csrc/okls_api.cpp", "csrc/okls_kernels.hip", "csrc/linear_api.cpp", "csrc/linear_kernels.hip",
           "csrc/optim_api.cpp", "csrc/optim_kernels.hip", "csrc/experts_api.cpp", "csrc/experts_kernels.hip"]
OUT = os.path.join(HERE, "libokls.so")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def compile_command(source, out):
    return ["hipcc", *FLAGS, "-c", os.path.join(HERE, source), "-o", out]


def link_command(objects, out):
    return ["hipcc", "--offload-arch=gfx950", "-fPIC", "-shared", *objects, "-o", out]


def _finish(command, process):
    out = process.communicate()[0]
    if process.returncode != 0:
        sys.stderr.write(out)
        raise RuntimeError("hipcc failed: " + " ".join(command))


def build(verbose=False):
    """Every source by a compiler of its own, at once; then the library."""
    with tempfile.TemporaryDirectory() as place:
        objects = [os.path.join(place, os.path.basename(s) + ".o") for s in SOURCES]
        commands = [compile_command(s, o) for s, o in zip(SOURCES, objects)]
        running = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in commands]
        try:
            for command, process in zip(commands, running):
                _finish(command, process)
        finally:
            for process in running:
                if process.poll() is None:
                    process.kill()
                    process.wait()
        tmp = OUT + ".tmp"
        command = link_command(objects, tmp)
        _finish(command, subprocess.Popen(command, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    os.replace(tmp, OUT)
    if verbose:
        print("built", OUT)
    return OUT


if __name__ == "__main__":
    build(verbose=True)
