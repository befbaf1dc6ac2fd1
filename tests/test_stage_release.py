"""Shared memory that asynchronous copies fill again is released only once no load of it can be in
flight (CPU, from the sources: an arrival on a barrier does not wait for loads issued before it, and
a copy is not ordered behind them; the race is too rare to provoke)."""
import os
import re

from gradient_quantization_gb300 import agoq


def _source(name):
    text = open(os.path.join(agoq.HERE, "csrc", name)).read()
    return re.sub(r"//.*", "", text)


def test_scales_of_the_fp4_product():
    """Released when the loaded scales have been written to tensor memory."""
    code = _source("fp4_gemm.cu")
    assert code.count("mbar_arrive(&sempty[s])") == 1
    start = code.index("uint32_t w[S::kScaleCols];")
    order = [code.index(s, start) for s in ("tmem_st16(to + c, w + c)", "tcgen05.wait::st.sync.aligned",
                                            "__syncwarp()", "mbar_arrive(&sempty[s])")]
    assert order == sorted(order)


def _kernel(code, name):
    """The text from a kernel's name to the next kernel or launch."""
    start = code.index(name + "(")
    ends = [code.find(s, start) for s in ("__global__", "cudaError_t launch")]
    return code[start:min(e for e in ends if e > 0)]


def test_the_staged_accumulation():
    """Released when the results, which need every loaded value, have been stored."""
    code = _kernel(_source("quangrad.cu"), "grad_accum_staged_kernel")
    assert code.count("mbar_arrive(&empty[stage])") == 1
    order = [code.index(s) for s in ("accum_block<MID>(", "reinterpret_cast<uint2 *>(master)[blk * 16 + j] = out",
                                     "__syncwarp()", "mbar_arrive(&empty[stage])")]
    assert order == sorted(order)


def test_the_staged_reduce():
    """Released behind a fence between the loads and copies to come, executed by every lane."""
    code = _kernel(_source("quangrad.cu"), "reduce_shards_staged_kernel")
    release = r"reads_before_copies\(\);\s*__syncwarp\(\);\s*if \(lane == 0\) mbar_arrive\(&empty\[stage\]\);"
    assert len(re.findall(release, code)) == code.count("mbar_arrive(") == 2
    assert "fence.proxy.async.shared::cta" in _source("gemm_common.cuh")


def test_the_weight_gradient_of_rmsnorm():
    """The same fence."""
    code = _kernel(_source("rmsnorm.cu"), "rmsnorm_dw_tma_kernel")
    release = r"reads_before_copies\(\);\s*__syncwarp\(\);\s*if \(lane == 0\) mbar_arrive\(&empty\[s\]\);"
    assert len(re.findall(release, code)) == code.count("mbar_arrive(") == 1


def test_the_codes_of_the_weight_gradient_product():
    """As it was: released after the stores of what the codes were turned into."""
    code = _source("wgrad_gemm_impl.cuh")
    assert code.count("mbar_arrive(&sh.empty_x[sx])") == 1
    stores, release = code.index("*reinterpret_cast<uint4 *>(dst) = y;"), code.index("mbar_arrive(&sh.empty_x[sx])")
    assert stores < code.index("fence.proxy.async.shared::cta", stores) < release
