"""The tcgen05 attention kernels at every small count of stream tiles of a block (64 rows each), and at counts around
the depth of their rings, against the plain 64-bit forms.  The senders and receivers are few enough blocks, or many
enough, that the streamed side is split or is not."""
import pytest
import torch

from test_nodes_gpu import BF16, F16, Case, fc  # noqa: F401

pytestmark = pytest.mark.gpu


def on_tcgen05(fc, c):  # noqa: F811
    """The case, once it is sure that both directions take the tcgen05 kernels."""
    sizes = len(c.rp) - 1, int(c.rp[-1]), int(c.sp[-1])
    assert all(fc.node_attention_on_tcgen05(c.dtype, c.h, c.kv, c.d, *sizes, vjp) for vjp in (False, True))
    return c


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, F16)])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 17])
def test_tile_counts(fc, tiles, d, dtype):  # noqa: F811
    """96 structures of 128 receivers are more blocks than the card takes at once, so that no structure is split."""
    send = [64 * tiles - (b % 3) * (31 if tiles > 1 else 0) for b in range(96)]
    on_tcgen05(fc, Case([128] * 96, send, 2, 2, d, dtype, cap=5.0, seed=tiles)).check(fc)


@pytest.mark.parametrize("tiles", [4, 6, 9, 13, 29])
def test_tile_counts_of_split_structures(fc, tiles):  # noqa: F811
    """One structure: its senders, and in the gradient its receivers, are shared by several blocks."""
    on_tcgen05(fc, Case([64 * tiles - 7], None, 2, 1, 64, BF16, cap=5.0, hide=0.1, seed=tiles)).check(fc)


def test_many_tiles_repeat_exactly(fc):  # noqa: F811
    """What reads a product before it is complete reads different values from run to run."""
    c = on_tcgen05(fc, Case([2100, 1500], None, 8, 8, 64, BF16, cap=9.0, hide=0.1))
    first = c.run(fc)
    for _ in range(30):
        again = c.run(fc)
        for a, b in zip([*first[0], *first[1]], [*again[0], *again[1]]):
            assert a is None or torch.equal(a, b)
    assert fc.device_error() == 0


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("apart", [False, True])
def test_a_gradient_does_not_depend_on_the_others_asked_for(fc, apart, bias):  # noqa: F811
    recv = [330, 150]
    c = on_tcgen05(fc, Case(recv, [200, 410] if apart else None, 4, 2, 64, BF16, cap=6.0, bias=bias, hide=0.1))
    (out, lse, o32), bars = c.run(fc)
    q, k, v = c.parts(c.qw.cuda(), c.kw.cuda())
    move = lambda t: None if t is None else t.cuda()  # noqa: E731
    kw = dict(c.kwargs(move), send_ptr=c.sp.cuda(), send_mask=c.mask.cuda())
    names = ("q", "k", "v", "pos", "pos_send", "slope")
    for want in (("q",), ("k",), ("v",), ("k", "v"), ("q", "k"), ("pos",), ("slope",), ("k", "slope"), ("v", "pos"), ("q", "v", "slope")):
        got = fc.node_attention_vjp(q, k, v, o32, lse, c.g.cuda(), c.rp.cuda(), want=want, **kw)
        for n, a, b in zip(names, got, bars):
            asked = n in want or n == "pos_send" and "pos" in want
            assert (a is None) == (b is None or not asked), (want, n)
            assert a is None or torch.equal(a, b), (want, n)


@pytest.mark.parametrize("power", [-10, 10])
@pytest.mark.parametrize("d", [8, 16, 32])
def test_score_factors_far_from_one_of_narrow_heads(fc, power, d):  # noqa: F811
    """Queries and keys times 2^power and scale times 4^-power are the same scores (exact in BF16), here at lengths at
    which narrow heads take the tcgen05 kernels: their polynomial has scale / cap in its coefficients."""
    c = on_tcgen05(fc, Case([400], None, 2, 2, d, BF16, cap=3.0))
    c.qw *= 2.0 ** power
    c.kw[:, : c.kv] *= 2.0 ** power
    c.scale *= 4.0 ** -power
    c.check(fc)


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, F16), (64, F16)])
def test_kernels_of_both_kinds_meet_on_uneven_batches(fc, d, dtype):  # noqa: F811
    """One long structure among many short and empty ones: a call has one kernel, whatever each structure is."""
    for short in (3, 12, 60):     # one structure of 900 and so many of 0 to 12 nodes
        lens = [(5 * i) % 13 for i in range(short)]
        Case(lens[: short // 2] + [900] + lens[short // 2:], None, 4, 2, d, dtype, cap=6.0, hide=0.1, lead=3, tail=20).check(fc)
