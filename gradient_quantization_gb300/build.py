"""Build libagoq.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each translation unit under csrc/ is compiled in parallel, then linked into
gradient_quantization_gb300/libagoq.so with the CUDA runtime linked
statically.  Every unit is compiled with -fmad=false so that no
multiply and add are contracted into one rounding (the kernels also use the
explicitly rounded intrinsics).  Run ``python -m gradient_quantization_gb300.build``.
"""
import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libagoq.so")
ROOT = os.path.dirname(HERE)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          "-I" + os.path.join(ROOT, "include")]
UNITS = {
    "agoq_api.cu": ["-fmad=false"],
    "laaq.cu": ["-fmad=false"],
    "quangrad.cu": ["-fmad=false"],
    "wgrad_gemm.cu": ["-fmad=false"],
    "wgrad_gemm_k64.cu": ["-fmad=false"],
    "rmsnorm.cu": ["-fmad=false"],
    "fwd_gemm.cu": ["-fmad=false"],
    "fwd_gemm_k64.cu": ["-fmad=false"],
    "layernorm.cu": ["-fmad=false"],
    "grad_norm.cu": ["-fmad=false"],
    "token_logprobs.cu": ["-fmad=false"],
    "fp4_quant.cu": ["-fmad=false"],
    "fp4_gemm.cu": ["-fmad=false"],
    "preference.cu": ["-fmad=false"],
}
HEADERS = ["agoq_device.cuh", "agoq_launch.h", "gemm_common.cuh", "wgrad_gemm_impl.cuh", "fwd_gemm_impl.cuh",
           "typed_io.cuh", "row_units.h", "fp4_format.cuh", "fp4_split.h"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force=False, verbose=False, ptxas_info=False):
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "agoq.h")]
    objs, jobs = [], []
    for unit, extra in UNITS.items():
        src = os.path.join(CSRC, unit)
        obj = os.path.join(BUILD, unit + ".o")
        objs.append(obj)
        if force or _stale(obj, [src, __file__] + hdrs):
            cmd = [nvcc, *ARCH, *COMMON, *extra, "-c", src, "-o", obj]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
    for cmd, r in zip(jobs, results):
        if verbose or ptxas_info or r.returncode:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode:
            raise RuntimeError("nvcc failed for " + cmd[-3])
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        subprocess.run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                ptxas_info="--ptxas-info" in sys.argv))
