"""Products of every variant from six threads on streams of their own, for some seconds: CTAs of
different calls share SMs, and each result is the one of a call alone, bit for bit."""
import random
import threading
import time

import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests.test_gpu_fp4_gemm import FORMATS, _gemm, _operand

pytestmark = pytest.mark.gpu
SIZES = [(1, 11008, 4096), (1, 11008, 4096), (40, 300, 2200), (3, 200, 8300), (300, 200, 9000), (512, 1024, 2048),
         (1001, 4090, 3999), (517, 5003, 1999)]


def test_products_at_once():
    ops = [(_operand(M, K, fmt, 1), _operand(N, K, fmt, 2), fmt) for M, N, K in SIZES for fmt in FORMATS]
    want = [_gemm(*op) for op in ops]
    torch.cuda.synchronize()
    stop, bad, calls = time.time() + 6, [], []

    def work(seed):
        pick, stream = random.Random(seed), torch.cuda.Stream()
        with torch.cuda.stream(stream):
            while time.time() < stop:
                some = [pick.randrange(len(ops)) for _ in range(20)]
                got = [_gemm(*ops[i]) for i in some]
                stream.synchronize()
                bad.extend(i for i, d in zip(some, got) if not torch.equal(d, want[i]))
                calls.append(len(some))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    agoq.agoq_device_status()
    assert not bad and sum(calls) > 0, (len(bad), sum(calls))
