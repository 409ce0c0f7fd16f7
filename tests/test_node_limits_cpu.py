"""Limits of the node operators that are decided on the host."""
import pytest
import torch

from test_nodes_cpu import ARG, attn, fc  # noqa: F401


@pytest.mark.parametrize("vjp", [False, True])
def test_attention_refuses_structures_that_the_tile_search_cannot_count(fc, vjp):  # noqa: F811
    """The search for a tile's structure looks up to 31 places past n_struct + 1 in 32 bits."""
    for b in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 3, 2 ** 31 - 64):
        assert attn(fc, vjp, b=b) == ARG, b


def test_factors_in_tensors_are_read_at_every_call(fc):  # noqa: F811
    """Descriptors are kept by their values; a tensor of one element that is changed in place is another value."""
    for make, name in ((lambda t: fc._attn_desc(0, 1, 1, 8, t, 0.0), "scale"), (lambda t: fc._attn_desc(0, 1, 1, 8, 1.0, t), "cap"),
                       (lambda t: fc._head_desc(0, 1, 1, 8, 0, t), "eps")):
        t = torch.tensor(0.5)
        assert getattr(make(t), name) == 0.5
        t.mul_(4)
        assert getattr(make(t), name) == 2.0
        assert make(0.25) is make(0.25)
    t = torch.tensor(1)
    assert fc._head_desc(0, t, 1, 8, 0, 1.0).heads_q == 1
    t.add_(2)
    assert fc._head_desc(0, t, 1, 8, 0, 1.0).heads_q == 3


def test_every_argument_can_be_named(fc):  # noqa: F811
    """Also the first: the call gets as far as finding that its tensors are on the CPU."""
    x, i = torch.zeros(4, 3, 8), torch.zeros(4, dtype=torch.int32)
    for f, kw in ((fc.species_embed, dict(species=i, table=x[0])), (fc.species_embed_vjp, dict(species=i, g=x[:, 0], n_species=3)),
                  (fc.head_norm_rotate, dict(x=x, heads_q=2)), (fc.head_norm_rotate_vjp, dict(x=x, g=x, heads_q=2)),
                  (fc.node_attention, dict(q=x, k=x, v=x, recv_ptr=i)),
                  (fc.node_attention_vjp, dict(q=x, k=x, v=x, out_f32=x, lse=x[0], g=x, recv_ptr=i))):
        with pytest.raises(TypeError, match="takes CUDA tensors"):
            f(**kw)
    with pytest.raises(TypeError):
        fc.head_norm_rotate()


def test_which_kernels_a_call_runs_on(fc):  # noqa: F811
    on = fc.node_attention_on_tcgen05
    bf16 = torch.bfloat16
    for vjp in (False, True):
        assert on(bf16, 4, 4, 64, 2, 600, 600, vjp) and on(torch.float16, 4, 1, 128, 1, 100, 100, vjp)
        assert not on(torch.float32, 4, 4, 64, 2, 600, 600, vjp)      # FP32 rows: strips
        assert not on(bf16, 4, 4, 64, 100, 600, 600, vjp)             # short structures
        assert not on(bf16, 4, 4, 64, 2, 600, 100, vjp)               # fewer than 64 senders
        assert not on(bf16, 4, 4, 64, 2, 0, 600, vjp) and not on(bf16, 4, 4, 64, 0, 600, 600, vjp)
        assert on(bf16, 1, 1, 8, 1, 2 ** 31 - 65, 2 ** 31 - 65, vjp)  # the ends of the copies' coordinates
        assert not on(bf16, 1, 1, 8, 1, 1000, 2 ** 31 - 64, vjp) and not on(bf16, 1, 1, 8, 1, 2 ** 31 - 64, 1000, vjp)
        for bad in ((4, 3, 64), (4, 4, 60), (4, 4, 136)):
            with pytest.raises(ValueError):
                on(bf16, *bad, 2, 600, 600, vjp)
    assert on(bf16, 65, 1, 64, 1, 600, 600) and not on(bf16, 65, 1, 64, 1, 600, 600, True)   # 65 heads to a key head
    with pytest.raises(TypeError):
        on(torch.float64, 4, 4, 64, 2, 600, 600)
