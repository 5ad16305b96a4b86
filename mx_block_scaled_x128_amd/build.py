"""Build libmxfp8.so (HIP kernels + C ABI) for gfx950 with hipcc, in-tree, and
_mx_tensors.so, the Python extension with the MX operators' tensor functions.

The sources compile to objects in parallel (the GEMM once per pair of operand
formats, plus its host dispatch; the MXFP4 product once per format of its left
operand), which hipcc then links into the library.

Usage: python -m mx_block_scaled_x128_amd.build   (always recompiles)
"""
import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmxfp8.so")
TENSORS = os.path.join(HERE, "_mx_tensors.so")
ARCH = "gfx950"
# (source, extra flags, object name)
UNITS = [("api.cpp", [], "api"), ("mx_api.cpp", [], "mx_api"), ("mx_quant.hip", [], "mx_quant"),
         ("mx_act.hip", [], "mx_act"),
         ("mxfp4_gemm.hip", ["-DMXFP4_GEMM_FMT=-1"], "mxfp4_gemm_dispatch"),
         ("quant.hip", [], "quant"), ("gaussws.hip", [], "gaussws"),
         ("gemm.hip", ["-DMXFP8_GEMM_FMT=-1"], "gemm_dispatch")] + \
        [("gemm.hip", ["-DMXFP8_GEMM_FMT=%d" % k], "gemm_fmt%d" % k) for k in range(4)] + \
        [("mxfp4_gemm.hip", ["-DMXFP4_GEMM_FMT=%d" % k], "mxfp4_gemm_fmt%d" % k) for k in range(3)]

FLAGS = [
    "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC",
    "-Wall", "-Wno-unused-command-line-argument",
    # keep packed-fp32 instructions out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def hipcc():
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    raise RuntimeError("hipcc not found")


def _run(cmd):
    proc = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the GPU feature flag; that warning is harmless
    err = "\n".join(l for l in proc.stderr.splitlines() if "packed-fp32-ops" not in l)
    if proc.returncode != 0:
        raise RuntimeError("hipcc failed: %s\n%s" % (" ".join(cmd), err))
    return err


def tensors_command(cc, out):
    """The extension: host code against torch's headers and libraries."""
    import torch
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    return [cc, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-DTORCH_EXTENSION_NAME=_mx_tensors",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI] + \
        [a for d in inc for a in ("-isystem", d)] + [os.path.join(CSRC, "tensors.cpp"), "-L" + os.path.join(base, "lib")] + \
        ["-l" + n for n in ("c10", "c10_hip", "torch_cpu", "torch", "torch_python")] + ["-o", out]


def build(verbose=False, jobs=None):
    """Build the library and the extension; return the library's path.  The library needs hipcc
    alone and is in place before an error of the extension (no torch, or a failed compilation)
    is raised."""
    cc = hipcc()
    tmpdir = tempfile.mkdtemp(prefix="mxfp8_build_")
    parts = []

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        err = _run(cmd)
        if verbose and err.strip():
            print(err, file=sys.stderr)

    def put(make, path):
        """make(path) written next to its place, then moved there."""
        part = path + ".tmp"
        parts.append(part)
        run(make(part))
        os.replace(part, path)

    try:
        cmds = [[cc] + FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", os.path.join(tmpdir, name + ".o")]
                for src, extra, name in UNITS]
        jobs = jobs or min(len(cmds) + 1, max(1, os.cpu_count() or 1))
        with concurrent.futures.ThreadPoolExecutor(max_workers=jobs) as pool:
            tensors = pool.submit(put, lambda out: tensors_command(cc, out), TENSORS)  # the longest first
            list(pool.map(run, cmds))
            put(lambda out: [cc, "--offload-arch=" + ARCH, "-shared", "-fPIC"] +
                [os.path.join(tmpdir, name + ".o") for _, _, name in UNITS] + ["-o", out], LIB)
            tensors.result()
    finally:
        shutil.rmtree(tmpdir, ignore_errors=True)
        for part in parts:
            if os.path.exists(part):
                os.remove(part)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
