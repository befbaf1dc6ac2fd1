"""The FP4 product's thread that issues MMAs waits for those in flight before its CTA frees tensor
memory, however its loop ends (CPU, from the source: a wait that runs out is not provoked)."""
import os
import re

from gradient_quantization_gb300 import agoq

SOURCE = os.path.join(agoq.HERE, "csrc", "fp4_gemm.cu")


def _mma_warp():
    text = open(SOURCE).read()
    kernel = text[text.index("fp4_gemm_kernel("):]
    start = kernel.index("} else if (warp == kMmaWarp) {")
    return kernel[start:kernel.index("} else if (warp < kScaleWarp0 + S::kScaleWarps)", start)]


def test_every_stage_that_is_issued_is_drained():
    """One place waits for a stage, it marks that MMAs may be in flight, every issue follows it, and
    the drain asks for nothing else."""
    code = re.sub(r"//.*", "", _mma_warp())
    assert len(re.findall(r"&full\[", code)) == 1 and code.count("issued = true") == 1
    wait = re.search(r"auto stage_there = \[&\] \{(.*?)\n\s*\};", code, re.S).group(1)
    order = [wait.index(s) for s in ("&full[ring.s]", "return false", "tc_fence_after()", "issued = true",
                                     "return true")]
    assert order == sorted(order)
    # the first issue of each of the three loops comes after a stage that is there
    loops = [m.start() for m in re.finditer(r"\bstage_there\(\)", code)]
    firsts = [m.start() for m in re.finditer(r"\bissue\((?:ring\.)?s, ", code)]
    assert len(loops) == 3 and len(firsts) == 3
    assert all(a < b for a, b in zip(loops, firsts)) and all(b < a for a, b in zip(loops[1:], firsts))
    drain = code[code.index("if (issued)"):]
    assert "drain" in drain and "wait_bar(drain, 0u, abort, status, true)" in drain
