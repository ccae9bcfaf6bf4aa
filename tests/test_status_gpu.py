"""Where the 8-bit calls record a wait that ran out, on the GPU."""
import os
import subprocess
import sys
import threading
import time

import pytest
import torch

from bit_nf4_quantized_20_b200 import inputs

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def Q():
    import bit_nf4_quantized_20_b200 as q
    return q


FIRST_USE = r"""
import torch
import bit_nf4_quantized_20_b200 as q
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(40, 256, device="cuda", generator=g).to(torch.bfloat16)
w = torch.randn(64, 256, device="cuda", generator=g).to(torch.bfloat16)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):          # the library's first calls of this process
    x8 = q.quantize_int8(x)
    w8 = q.quantize_int8(w)
    y = q.linear_int8(x8, w8)
graph.replay()
q.get_error()
want = q.linear_int8(x, q.quantize_int8(w))
assert torch.equal(y.view(torch.int16), want.view(torch.int16))
# a wait that runs out on the word that the graph was given
q.wait_selftest(1000, noalloc=True)
try:
    q.get_error()
except q.QLoraError as e:
    assert e.status == 7
else:
    raise AssertionError("the timeout was not reported")
q.get_error()
graph.replay()
q.get_error()
assert torch.equal(y.view(torch.int16), want.view(torch.int16))
del graph
print("ok")
"""


def test_first_use_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST_USE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["ok"], r.stderr[-2000:]


def test_every_name_of_the_device():
    q = Q()
    for made in ("cuda", "cuda:0", None):
        for asked in ("cuda", "cuda:0", None, 0):
            q.wait_selftest(500, made)
            with pytest.raises(q.QLoraError) as e:
                q.get_error(asked)
            assert e.value.status == 7
            q.get_error(asked)


def test_two_threads_at_the_first_use():
    """Both get the same word."""
    q = Q()
    dev = torch.device("cuda", torch.cuda.current_device())
    kept = q._STATUS.pop(dev, None)
    try:
        for _ in range(20):
            q._STATUS.pop(dev, None)
            start, got = threading.Barrier(2), []

            def first():
                start.wait()
                got.append(q._status(dev))

            threads = [threading.Thread(target=first) for _ in range(2)]
            for t in threads:
                t.start()
            for t in threads:
                t.join()
            assert len(got) == 2 and got[0] == got[1] == q._STATUS[dev].data_ptr()
    finally:
        if kept is not None:
            q._STATUS[dev] = kept


def test_a_null_word_is_the_fixed_arrays():
    """A timeout there is reported by noalloc_get_error; a call with a null word runs."""
    q = Q()
    x8 = q.quantize_int8(inputs.normal_bf16((40, 256), 1.0, 1, "cuda"))
    w8 = q.quantize_int8(inputs.normal_bf16((64, 256), 0.02, 2, "cuda"))
    y = torch.empty(40, 64, dtype=torch.bfloat16, device="cuda")
    q._int8_call(x8.device, "qlora_linear_int8_q", x8._ref, w8._ref, y.data_ptr(), None)
    q.noalloc_get_error()
    assert torch.equal(y.view(torch.int16), q.linear_int8(x8, w8).view(torch.int16))


def test_both_bounded_waits_run_out():
    """The two waits of the pipelines (the 8-bit kernels' producers and issuers
    use the one that does not suspend) give up one after the other, each after
    its limit, and the 8-bit calls' status word says so once."""
    q = Q()
    dev = torch.device("cuda", torch.cuda.current_device())
    w8 = q.quantize_int8(inputs.normal_bf16((64, 256), 0.02, 2, "cuda"))
    x = inputs.normal_bf16((40, 256), 1.0, 1, "cuda")
    want = q.linear_int8(x, w8)
    q.get_error()
    limit_us = 20000
    t0 = time.perf_counter()
    assert q.lib().qlora_wait_selftest(q._status(dev), 256, limit_us, q._raw_stream(dev.index)) == 0
    with pytest.raises(q.QLoraError) as e:
        q.get_error()
    assert e.value.status == 7
    assert 2e-6 * limit_us <= time.perf_counter() - t0 < 5.0
    q.get_error()
    assert torch.equal(q.linear_int8(x, w8).view(torch.int16), want.view(torch.int16))
