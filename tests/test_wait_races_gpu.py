"""Bounded waits whose limit runs out about when the barrier completes, so that some lanes, warps and blocks see a
completed phase and others give up: the calls return, and a call that nothing gave up in (the error word is 0) gives
the right results.  With the default bound back, so does every call."""
import pytest
import torch

from cartesian_tensor_products_b200 import workloads as W
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


@pytest.mark.parametrize("nodes", [20, 600])
def test_ladder_waits_race_their_limit(fc, nodes):  # noqa: F811
    """20 nodes: blocks whose copies all fit the stages, so that the copying role itself has nothing to wait for when
    another gives up.  The weight gradients are summed by atomic additions, so that only the rest is bit-equal."""
    L, C, order = 3, 128, 3
    lad = W.ladder_inputs(nodes, L, C, order, 23)
    A1, pw, mw, gz = (torch.from_numpy(lad[k]).cuda() for k in ("A1", "path_w", "mix_w", "gz"))

    def call():
        states, z = fc.product_ladder(L, order, A1, pw, mw)
        a1b = fc.product_ladder_vjp(L, order, A1, pw, mw, states, gz)[0]
        return [states, z, a1b]
    assert race(fc, call) > 0


@pytest.mark.parametrize("nodes", [8, 300])
def test_full_ladder_waits_race_their_limit(fc, nodes):  # noqa: F811
    L, C, order = 2, 128, 3
    fl = W.full_ladder_inputs(nodes, L, C, order, 12)
    A, W1, Wq = (torch.from_numpy(fl[k]).cuda() for k in ("A", "W1", "Wq"))
    gz = torch.randn_like(fc.full_ladder(L, order, A, W1, Wq)[1])

    def call():
        states, z = fc.full_ladder(L, order, A, W1, Wq)
        a_bar = fc.full_ladder_vjp(L, order, A, W1, Wq, states, gz)[0]
        return [states, z, a_bar]
    assert race(fc, call) > 0
