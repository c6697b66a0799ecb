"""Build libric.so in-tree with hipcc for gfx950.

Run ``python -m ragged_input_compilation_amd.build`` (or call ``build()``).
The library links only the HIP runtime; nothing here imports torch."""
import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libric.so")
SOURCES = [os.path.join(CSRC, n) for n in ("ric_kernels.hip", "ric_attention.hip", "ric_logprobs.hip", "ric_pages.hip",
                                           "ric_host.cpp", "ric_ops_host.cpp")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Wall", "-Wno-unused-function",
    # no packed-fp32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I" + os.path.join(ROOT, "include"),
]


def build(verbose: bool = False, extra_flags=()) -> str:
    """Compile every source (at the same time), then link."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as objects:
        cmds = [[HIPCC] + FLAGS + list(extra_flags) + ["-x", "hip", "-c", src, "-o",
                                                       os.path.join(objects, os.path.basename(src) + ".o")]
                for src in SOURCES]
        jobs = []
        for cmd in cmds:
            if verbose:
                print(" ".join(cmd), flush=True)
            jobs.append(subprocess.Popen(cmd))
        codes = [j.wait() for j in jobs]
        for cmd, code in zip(cmds, codes):
            if code:
                raise subprocess.CalledProcessError(code, cmd)
        link = [HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared"] + list(extra_flags) + [c[-1] for c in cmds] + \
            ["-o", tmp]
        if verbose:
            print(" ".join(link), flush=True)
        subprocess.check_call(link)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-q" not in sys.argv))
