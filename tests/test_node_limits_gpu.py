"""The node operators at the ends of their ranges."""
import pytest
import torch

from parity import FWD_TOL, VJP_TOL
from test_nodes_gpu import BF16, close, fc  # noqa: F401

pytestmark = pytest.mark.gpu


def test_senders_to_the_last_of_31_bits(fc):  # noqa: F811
    """One receiver against 2^31 - 1 senders (34 GB of rows): the last two hold nearly all of the weight.  The count
    of their tiles of 64 does not fit 32 bits ahead of its division."""
    n, d = 2 ** 31 - 1, 8
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free device memory")
    k = torch.zeros(n, 1, d, dtype=BF16, device="cuda")
    k[-2:, 0, :2] = torch.tensor([[40.0, 1.0], [40.5, 0.0]], dtype=BF16, device="cuda")
    q = torch.zeros(1, 1, d, dtype=BF16, device="cuda")
    q[0, 0, 0] = 1.0
    g = torch.ones_like(q)
    ends = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, lse, o32 = fc.node_attention(q, k, k, *ends, scale=1.0, residual=True)
    t = torch.tensor([40.0, 40.5], dtype=torch.float64)
    z = torch.log(torch.exp(t).sum() + float(n - 2))
    p = torch.exp(t - z)
    rows = k[-2:, 0].double().cpu()
    ref = (p[:, None] * rows).sum(0)
    close(lse, z.reshape(1, 1), FWD_TOL * float(z))
    # the weights as two 16-bit terms
    close(o32, ref.reshape(1, 1, d), FWD_TOL * float(ref.abs().max()) + 2.0 ** -16 * ref.abs().reshape(1, 1, d))
    qb = fc.node_attention_vjp(q, k, k, o32, lse, g, *ends, scale=1.0, want=("q",))[0]
    dp = rows.sum(1)
    ds = p * (dp - ref.sum())     # and P (0 - sum of ref) for the rest, times keys of 0
    want = (ds[:, None] * rows).sum(0)
    # dS rounded to 16 bits: 2^-8 of |dS| |k|; delta, off by its 2^-16 of sum P |v| (41), moves dS by P of that; then one rounding
    bound = 2.0 ** -8 * ((ds.abs()[:, None] * rows.abs()).sum(0) + want.abs()) + 41 * 2.0 ** -16 * 1.1 * (p[:, None] * rows.abs()).sum(0)
    close(qb, want.reshape(1, 1, d), (bound + VJP_TOL * float(want.abs().max())).reshape(1, 1, d))


def test_scale_cap_and_eps_in_tensors_changed_in_place(fc):  # noqa: F811
    q = torch.randn(20, 2, 16, device="cuda")
    ptr = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    scale, cap, eps = torch.tensor(0.5), torch.tensor(4.0), torch.tensor(1e-6)
    for _ in range(3):
        a = fc.node_attention(q, q, q, ptr, scale=scale, cap=cap)
        b = fc.node_attention(q, q, q, ptr, scale=scale.item(), cap=cap.item())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert torch.equal(fc.head_norm_rotate(q, 1, eps=eps), fc.head_norm_rotate(q, 1, eps=eps.item()))
        scale.mul_(1.5)
        cap.mul_(0.5)
        eps.mul_(1e3)


def test_calls_by_name_alone(fc):  # noqa: F811
    x = torch.randn(20, 4, 16, device="cuda")
    q, k = x[:, :2], x[:, 2:]
    ptr = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    species = torch.arange(20, dtype=torch.int32, device="cuda") % 3
    table = torch.randn(3, 8, device="cuda")
    same = lambda a, b: all(torch.equal(u, v) for u, v in zip(a, b) if u is not None)  # noqa: E731
    assert torch.equal(fc.species_embed(table=table, species=species), fc.species_embed(species, table))
    g = torch.randn(20, 8, device="cuda")
    assert torch.equal(fc.species_embed_vjp(n_species=3, g=g, species=species), fc.species_embed_vjp(species, g, 3))
    y = fc.head_norm_rotate(heads_q=2, x=x, stream=torch.cuda.current_stream())
    assert torch.equal(y, fc.head_norm_rotate(x, 2))
    assert same(fc.head_norm_rotate_vjp(g=y, heads_q=2, x=x), fc.head_norm_rotate_vjp(x, y, 2))
    out = fc.node_attention(recv_ptr=ptr, v=k, k=k, q=q, residual=True)
    assert same(out, fc.node_attention(q, k, k, ptr, residual=True))
    a = (q, k, k, out[2], out[1], q, ptr)
    assert same(fc.node_attention_vjp(**dict(zip(("q", "k", "v", "out_f32", "lse", "g", "recv_ptr"), a))), fc.node_attention_vjp(*a))
