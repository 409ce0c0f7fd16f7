"""Refusals and workspace sizes of the node operators (include/flashcart_nodes.h): everything here is decided on
the host, before anything is enqueued."""
import ctypes as ct

import pytest
import torch

OK, ARG, ALIGN, WORKSPACE = 0, 1, 5, 7
P = ct.c_void_p(4096)        # never dereferenced
ODD = ct.c_void_p(4100)      # 4-byte aligned only
OFF = ct.c_void_p(4098)


@pytest.fixture(scope="module")
def fc():
    from cartesian_tensor_products_b200 import build
    build.build()
    from cartesian_tensor_products_b200 import flashcart
    return flashcart


def test_species_embed_refusals(fc):
    f = fc.lib().fc_species_embed
    call = lambda dt=0, n=5, v=3, lmax=0, c=8, s=1.0, sp=P, t=P, x=P: f(dt, n, v, lmax, c, s, sp, t, x, None)  # noqa: E731
    assert call(n=0) == OK
    assert call(dt=3) == ARG and call(dt=-1) == ARG and call(n=-1) == ARG and call(v=0) == ARG
    assert call(lmax=-1) == ARG and call(lmax=9) == ARG and call(c=0) == ARG and call(s=float("nan")) == ARG
    assert call(c=6) == ALIGN and call(dt=1, c=4) == ALIGN
    assert call(sp=None) == ARG and call(t=None) == ARG and call(x=None) == ARG
    assert call(t=ODD) == ALIGN and call(x=ODD) == ALIGN and call(sp=OFF) == ALIGN


def test_species_embed_vjp_refusals(fc):
    lib = fc.lib()
    size = lib.fc_species_embed_vjp_workspace_size(100, 10, 8)
    call = lambda dt=0, n=100, v=10, lmax=0, c=8, sp=P, g=P, b=P, ws=P, nb=size: lib.fc_species_embed_vjp(  # noqa: E731
        dt, n, v, lmax, c, 1.0, sp, g, b, ws, nb, None)
    assert call(nb=size - 1) == WORKSPACE and call(ws=None) == WORKSPACE and call(ws=ODD) == ALIGN
    assert call(b=None) == ARG and call(g=None) == ARG and call(sp=None) == ARG and call(v=0) == ARG
    assert call(b=ODD) == ALIGN and call(g=ODD) == ALIGN and call(c=2) == ALIGN
    assert lib.fc_species_embed_vjp_workspace_size(0, 10, 8) == 0
    assert lib.fc_species_embed_vjp_workspace_size(10, 0, 8) == 0
    # one pass of 8 bits up to 255 species (key 255 is "none"), two after
    one, two = (lib.fc_species_embed_vjp_workspace_size(1 << 20, v, 8) for v in (255, 256))
    assert two - one == 2 * 4 * (1 << 20)


def test_head_norm_refusals(fc):
    lib = fc.lib()

    def call(dt=0, hq=2, hk=1, d=16, r=8, eps=1e-6, n=4, x=P, ldx=48, gq=P, gk=P, pos=P, fr=P, y=P, ldy=48):
        desc = fc.HeadDesc(dt, hq, hk, d, r, eps)
        return lib.fc_head_norm_rotate(ct.byref(desc), n, x, ldx, gq, gk, pos, fr, y, ldy, None)
    assert call(n=0) == OK
    for bad in (dict(dt=5), dict(hq=0, hk=0), dict(hq=-1), dict(hq=1024, hk=1), dict(d=0), dict(d=136), dict(r=9), dict(r=-1),
                dict(eps=-1.0), dict(eps=float("inf")), dict(n=-1), dict(x=None), dict(y=None), dict(pos=None),
                dict(fr=None), dict(ldx=40), dict(ldy=40)):
        assert call(**bad) == ARG, bad
    for bad in (dict(d=12, r=4), dict(x=ODD), dict(y=ODD), dict(ldx=52), dict(ldy=49), dict(gq=OFF), dict(pos=OFF)):
        assert call(**bad) == ALIGN, bad
    assert lib.fc_head_norm_rotate(None, 4, P, 48, P, P, P, P, P, 48, None) == ARG


def test_head_norm_vjp_refusals(fc):
    lib = fc.lib()
    desc = fc.HeadDesc(0, 2, 1, 16, 8, 1e-6)
    size = lib.fc_head_norm_rotate_vjp_workspace_size(ct.byref(desc), 4)
    assert size > 0 and lib.fc_head_norm_rotate_vjp_workspace_size(ct.byref(desc), 0) == 0

    def call(n=4, x=P, ldx=48, g=P, ldg=48, xb=P, ldxb=48, gqb=P, gkb=P, pb=P, ws=P, nb=size):
        return lib.fc_head_norm_rotate_vjp(ct.byref(desc), n, x, ldx, g, ldg, P, P, P, P, xb, ldxb, gqb, gkb, pb, ws, nb, None)
    assert call(nb=size - 1) == WORKSPACE and call(ws=None) == WORKSPACE and call(ws=ODD) == ALIGN
    assert call(x=None) == ARG and call(g=None) == ARG and call(ldg=32) == ARG and call(ldxb=32) == ARG
    assert call(xb=ODD) == ALIGN and call(g=ODD) == ALIGN and call(pb=OFF) == ALIGN and call(ldxb=50) == ALIGN
    assert call(xb=None, gqb=None, gkb=None, pb=None, ws=None) == OK     # nothing asked for, nothing enqueued


def attn(fc, vjp=False, dt=0, h=4, kv=2, d=16, scale=0.25, cap=0.0, b=2, nr=10, ns=10, rp=P, sp=P, q=P, ldq=64, k=P, ldk=32,
         v=P, ldv=32, pr=P, ps=None, sl=P, mask=None, out=P, ldo=64, lse=P, o32=None, ws=P, nb=1 << 30, g=P, ldg=64, qb=P,
         kb=P, vb=P, prb=P, psb=None, slb=P):
    desc = fc.AttnDesc(dt, h, kv, d, scale, cap)
    head = (ct.byref(desc), b, nr, ns, rp, sp, q, ldq, k, ldk, v, ldv, pr, ps, sl, mask)
    if not vjp:
        return fc.lib().fc_node_attention(*head, out, ldo, lse, o32, ws, nb, None)
    return fc.lib().fc_node_attention_vjp(*head, P if o32 is None else o32, lse, g, ldg, qb, kb, vb, prb, psb, slb, ws, nb, None)


@pytest.mark.parametrize("vjp", [False, True])
def test_attention_refusals(fc, vjp):
    for bad in (dict(dt=3), dict(h=0), dict(kv=0), dict(h=3), dict(h=2, kv=4), dict(h=2048, kv=1), dict(d=0), dict(d=136),
                dict(scale=float("nan")), dict(cap=-1.0), dict(cap=float("inf")), dict(b=-1), dict(nr=-1), dict(ns=-1),
                dict(rp=None), dict(sp=None), dict(q=None), dict(k=None), dict(v=None), dict(ldq=56), dict(ldk=24),
                dict(ldv=24), dict(pr=None), dict(sl=None), dict(ns=11), dict(pr=None, sl=None, ps=P)):
        assert attn(fc, vjp, **bad) == ARG, bad
    for bad in (dict(d=12), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(ldq=68), dict(ldk=33), dict(ldv=36), dict(rp=OFF),
                dict(sp=OFF), dict(pr=OFF), dict(sl=OFF), dict(lse=OFF)):
        assert attn(fc, vjp, **bad) == ALIGN, bad
    if not vjp:
        assert attn(fc, nr=0) == OK
        assert attn(fc, out=None) == ARG and attn(fc, ldo=56) == ARG
        assert attn(fc, out=ODD) == ALIGN and attn(fc, o32=ODD) == ALIGN
        # few rows against many senders: the senders are split, which needs scratch
        desc = fc.AttnDesc(0, 4, 2, 16, 0.25, 0.0)
        need = fc.lib().fc_node_attention_workspace_size(ct.byref(desc), 1, 1, 100000)
        assert need > 0 and fc.lib().fc_node_attention_workspace_size(ct.byref(desc), 2, 10, 10) == 0
        assert attn(fc, b=1, nr=1, ns=100000, ps=P, nb=need - 1) == WORKSPACE
        assert attn(fc, b=1, nr=1, ns=100000, ps=P, ws=None) == WORKSPACE
        assert attn(fc, b=1, nr=1, ns=100000, ps=P, ws=ODD, nb=need) == ALIGN
    else:
        desc = fc.AttnDesc(0, 4, 2, 16, 0.25, 0.0)
        need = fc.lib().fc_node_attention_vjp_workspace_size(ct.byref(desc), 2, 10, 10)
        assert attn(fc, True, nb=need - 1) == WORKSPACE and attn(fc, True, ws=None) == WORKSPACE
        assert attn(fc, True, ws=ODD) == ALIGN
        assert attn(fc, True, g=None) == ARG and attn(fc, True, lse=None) == ARG and attn(fc, True, ldg=56) == ARG
        assert attn(fc, True, psb=P) == ARG                        # no pos_send: its sum is in pos_recv_bar
        assert attn(fc, True, pr=None, sl=None, prb=None) == ARG    # a slope gradient without slopes
        assert attn(fc, True, qb=ODD) == ALIGN and attn(fc, True, prb=OFF) == ALIGN and attn(fc, True, o32=ODD) == ALIGN


@pytest.mark.parametrize("vjp", [False, True])
def test_attention_refuses_factors_that_overflow(fc, vjp):
    for bad in (dict(cap=1e-38, scale=1e3), dict(cap=3e38), dict(scale=3e38), dict(scale=-3e38)):
        assert attn(fc, vjp, **bad) == ARG, bad


def test_python_sizes_fit_the_library(fc):
    fc._counts(0, 2 ** 31 - 1)
    for bad in (2 ** 31, 2 ** 32 + 5, -1):
        with pytest.raises(ValueError):
            fc._counts(1, bad)


def test_python_entries_refuse_cpu_tensors(fc):
    x = torch.zeros(4, 3, 8)
    i = torch.zeros(4, dtype=torch.int32)
    for f in (lambda: fc.species_embed(i, torch.zeros(3, 8)), lambda: fc.species_embed_vjp(i, torch.zeros(4, 8), 3),
              lambda: fc.head_norm_rotate(x, 2), lambda: fc.head_norm_rotate_vjp(x, x, 2),
              lambda: fc.node_attention(x, x, x, i), lambda: fc.node_attention_vjp(x, x, x, x, x, x, i)):
        with pytest.raises(TypeError):
            f()
