"""The kernels whose shared memory bulk copies fill again and again, from six threads on streams of
their own beside products that share their SMs: each result is the one of a call alone, bit for
bit."""
import random
import threading
import time

import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests.test_gpu_fp4_gemm import _gemm, _operand

pytestmark = pytest.mark.gpu


def _at_once(calls, seconds=4):
    """`calls`: functions that return tensors, the same at every call."""
    a, b = _operand(1, 4096, agoq.NVFP4, 1), _operand(4096, 4096, agoq.NVFP4, 2)
    calls = calls + [lambda: [_gemm(a, b, agoq.NVFP4)]]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    stop, bad, done = time.time() + seconds, [], []

    def work(seed):
        pick, stream = random.Random(seed), torch.cuda.Stream()
        with torch.cuda.stream(stream):
            while time.time() < stop:
                some = [pick.randrange(len(calls)) for _ in range(10)]
                got = [calls[i]() for i in some]
                stream.synchronize()
                bad.extend(i for i, r in zip(some, got) if not all(torch.equal(x, y) for x, y in zip(r, want[i])))
                done.append(len(some))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    agoq.agoq_device_status()
    assert not bad and sum(done) > 0, (len(bad), sum(done))


def test_accumulations():
    calls = []
    for seed, n in ((1, 1 << 20), (2, 96 * 128 * 152 * 7 + 512)):     # one tile a CTA or none; several
        g = torch.Generator(device="cuda").manual_seed(seed)
        grad = torch.randn(n, generator=g, device="cuda").bfloat16()
        start = torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(n // 128, device="cuda")
        agoq.agoq_grad_accum_fp8(*start, torch.randn(n, generator=g, device="cuda").bfloat16())

        def call(grad=grad, start=start):
            master, scales = (t.clone() for t in start)
            return agoq.agoq_grad_accum_fp8(master, scales, grad)
        calls.append(call)
    _at_once(calls)


def test_reduces():
    calls = []
    for W, n, count in ((3, 1 << 18, False), (8, 1 << 20, True), (13, 64 * 128 * 152 * 3 + 512, False)):
        g = torch.Generator(device="cuda").manual_seed(W)
        shards = torch.randint(0, 120, (W, n), generator=g, device="cuda").to(torch.uint8)
        scales = torch.rand(W, n // 128, generator=g, device="cuda")

        def call(W=W, n=n, count=count, shards=shards, scales=scales):
            c = torch.zeros(1, dtype=torch.int64, device="cuda") if count else None
            out = agoq.agoq_reduce_fp8_shards(shards, scales, W, n, naive_overflow_count=c)
            return list(out) + ([c] if count else [])
        calls.append(call)
    _at_once(calls)


def test_rmsnorm_backwards():
    calls = []
    for T, H, bits in ((512, 512, 4), (4096, 1024, 8), (8192, 4096, 4)):
        g = torch.Generator(device="cuda").manual_seed(T)
        x, dy = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
        w = torch.randn(H, generator=g, device="cuda").bfloat16()
        codes, scales = agoq.agoq_quant_act(x, bits)
        calls.append(lambda a=(codes, scales, dy, w, T, H, bits): list(agoq.agoq_rmsnorm_backward(*a, 1e-5)))
    _at_once(calls)
