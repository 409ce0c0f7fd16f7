"""Bounded waits whose limit runs out about when the barrier completes, so that some lanes, warps and blocks see a
completed phase and others give up: the calls return, and a call that nothing gave up in (the error word is 0) gives
the right results.  With the default bound back, so does every call."""
import pytest
import torch

from test_nodes_gpu import BF16, F16, Case, fc  # noqa: F401

pytestmark = pytest.mark.gpu

LIMITS = [int(100 * 1.3 ** i) for i in range(28)]     # 100 ns to 0.12 ms


def race(fc, call, reps=4):  # noqa: F811
    """call() returns tensors; runs it under every limit.  Returns how many of the calls gave up."""
    clean = call()
    torch.cuda.synchronize()
    assert fc.device_error() == 0
    gave_up = 0
    try:
        for limit in LIMITS:
            fc.set_wait_timeout(limit)
            for _ in range(reps):
                got = call()
                torch.cuda.synchronize()
                if fc.device_error():
                    gave_up += 1
                else:
                    assert all(torch.equal(a, b) for a, b in zip(clean, got)), limit
    finally:
        fc.set_wait_timeout(0)
    got = call()
    torch.cuda.synchronize()
    assert fc.device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(clean, got))
    return gave_up


@pytest.mark.parametrize("d,kv,dtype", [(64, 4, BF16), (128, 2, F16)])
def test_attention_waits_race_their_limit(fc, d, kv, dtype):  # noqa: F811
    c = Case([700, 450], None, 4, kv, d, dtype, cap=8.0, hide=0.1)

    def call():
        outs, bars = c.run(fc)
        return [t for t in (*outs, *bars) if t is not None]
    assert race(fc, call) > 0
