"""Species embedding, head norm with rotation and node attention against plain 64-bit forms.

Bounds.  One rounding to type t costs at most u(t) = eps(t)/2 of the value.  FP32 steps inside a kernel are held to
the library's own limits (1e-5 forward, 1e-4 gradients, of the largest entry); sums of m terms to m roundings of
the sum of magnitudes; 16-bit weights inside a product to u(t) of the sum of magnitudes they multiply."""
import math

import pytest
import torch

import node_ref as R
from parity import FWD_TOL, VJP_TOL

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def fc():
    from cartesian_tensor_products_b200 import build
    build.build()
    from cartesian_tensor_products_b200 import flashcart
    return flashcart


def gen(seed):
    return torch.Generator().manual_seed(seed)


def sub(dtype):
    """FP16 below 2^-14 has a fixed step of 2^-24 (smallest subnormal), so a rounding there costs up to 2^-25
    whatever the value: 2e-5, for one, lies up to 2^-25 = 3.0e-8 off, not 2^-11 2e-5 = 9.8e-9."""
    return 2.0 ** -25 if dtype == F16 else 0.0


def normal(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def dev(t):
    return None if t is None else t.cuda()


def close(got, ref, bound):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), "off by %.3g where %.3g is allowed (%d entries)" % (
        (got - ref).abs()[bad].max(), (bound * torch.ones_like(ref))[bad].max(), int(bad.sum()))


# ------------------------------------------------------------ species embedding

@pytest.mark.parametrize("n,v,c,lmax,dtype", [
    (1, 1, 4, 0, F32), (7, 3, 8, 2, BF16), (33, 5, 12, 3, F32), (1000, 100, 128, 3, F32), (513, 300, 72, 1, F16),
    (5, 70000, 8, 0, F16), (2, 3, 4096, 3, F32), (70001, 17, 8, 0, BF16)])
def test_species_embed(fc, n, v, c, lmax, dtype):
    g = gen(n)
    species = torch.randint(-1, v + 1, (n,), generator=g, dtype=torch.int32)     # -1 and v: no species
    table = normal(g, v, c, dtype=dtype)
    ref = R.embed(species, table, lmax, 0.7)
    scale = torch.tensor(0.7, dtype=F32).double()          # the product in FP32, then one rounding
    ref = ref / 0.7 * scale
    out = fc.species_embed(dev(species), dev(table), lmax=lmax, scale=0.7)
    close(out, ref, ref.abs() * (R.u(dtype) + (R.U32 if dtype != F32 else 0.0) * 1.01) + sub(dtype))
    one = fc.species_embed(dev(species), dev(table), lmax=lmax)
    assert torch.equal(one.double().cpu(), R.embed(species, table, lmax, 1.0))


@pytest.mark.parametrize("n,v,c,lmax,dtype,kind", [
    (1, 1, 4, 0, F32, "even"), (31, 3, 8, 1, BF16, "even"), (32, 3, 8, 0, F16, "one"), (33, 2, 12, 2, F32, "even"),
    (64, 4, 8, 0, F32, "blocks"), (1023, 100, 128, 1, F32, "even"), (1025, 255, 136, 0, BF16, "even"),
    (5000, 256, 8, 0, F32, "even"), (5000, 100, 260, 0, F32, "one"), (40000, 70000, 8, 0, F16, "even"),
    (100003, 9, 8, 0, F32, "skew"), (3000, 40, 8, 0, F32, "none"), (262144 + 5, 300, 4, 0, F32, "skew")])
def test_species_embed_vjp(fc, n, v, c, lmax, dtype, kind):
    g = gen(n + v)
    species = torch.randint(-1, v + 1, (n,), generator=g, dtype=torch.int32)
    if kind == "one":
        species[:] = v // 2
    elif kind == "skew":
        species = (torch.rand(n, generator=g) ** 6 * v).int()
    elif kind == "blocks":
        species = torch.arange(n, dtype=torch.int32) // 32
    elif kind == "none":
        species[::2] = -1
        species[1::2] = v
    gr = normal(g, n, (lmax + 1) ** 2 * c, dtype=dtype)
    ref, mag, count = R.embed_vjp(species, gr, v, lmax, 0.5)
    args = (dev(species), dev(gr), v)
    bar = fc.species_embed_vjp(*args, lmax=lmax, scale=0.5)
    # every addition rounds a partial sum, at most the sum of magnitudes
    close(bar, ref, (count[:, None] + 2) * R.U32 * mag)
    assert torch.equal(bar, fc.species_embed_vjp(*args, lmax=lmax, scale=0.5))


# ------------------------------------------------------------ head norm and rotation

NORM = [
    (1, 1, 0, 8, 0, F32), (1, 0, 1, 8, 4, BF16), (3, 2, 1, 16, 8, F32), (129, 8, 8, 16, 8, F32), (1000, 5, 3, 24, 5, F16),
    (77, 3, 3, 120, 59, BF16), (77, 3, 3, 120, 1, F32), (50, 16, 4, 64, 32, BF16), (301, 4, 1, 128, 64, F32),
    (33, 2, 2, 128, 62, F16), (65, 1, 7, 40, 12, F32), (4000, 8, 8, 32, 12, F32), (9, 600, 300, 8, 3, F32), (20, 2, 2, 96, 0, F16)]


def norm_case(n, hq, hk, d, r, dtype, far=50.0):
    g = gen(n * 7 + d)
    wide = normal(g, n, hq + hk + 2, d, dtype=dtype, scale=1.5)
    x = wide[:, 1: 1 + hq + hk]                            # a column block of a wider row
    gq, gk = 1 + normal(g, d, scale=0.3), 1 + normal(g, d, scale=0.3)
    pos = torch.rand((n, 3), generator=g) * far if r else None
    freq = normal(g, 3, r) if r else None
    return g, wide, x, gq, gk, pos, freq


@pytest.mark.parametrize("n,hq,hk,d,r,dtype", NORM)
def test_head_norm_rotate(fc, n, hq, hk, d, r, dtype):
    g, wide, x, gq, gk, pos, freq = norm_case(n, hq, hk, d, r, dtype)
    args = [None if t is None else t.double() for t in (gq, gk, pos, freq)]
    ref = R.norm(x.double(), hq, *args, 1e-6)
    plain = R.norm(x.double(), hq, *args[:2], None, None, 1e-6).abs()
    mag = plain.clone()
    if r:
        mag[..., :2 * r] = (plain[..., :r] + plain[..., r:2 * r]).repeat(1, 1, 2)
    xg = dev(wide)[:, 1: 1 + hq + hk]
    y = fc.head_norm_rotate(xg, hq, dev(gq), dev(gk), dev(pos), dev(freq))
    # mean square: d/2 roundings after the root; root, angle (2^-25 of half a turn) and products: under 16
    close(y, ref, R.u(dtype) * ref.abs() + (d / 2 + 16) * R.U32 * mag + sub(dtype))


def test_head_norm_far_positions_and_defaults(fc):
    """Positions 5e4 from the origin: the phase keeps its FP64 accuracy; no gamma means ones."""
    g, wide, x, _, _, pos, freq = norm_case(40, 3, 2, 32, 16, F32, far=5e4)
    ref = R.norm(x.double(), 3, None, None, pos.double(), freq.double(), 1e-6)
    y = fc.head_norm_rotate(x.cuda(), 3, pos=dev(pos), freq=dev(freq))
    close(y, ref, FWD_TOL * ref.abs().max())
    bars = fc.head_norm_rotate_vjp(x.cuda(), y, 3, pos=dev(pos), freq=dev(freq), want=("x",))
    assert bars[1] is None and bars[2] is None and bars[3] is None


@pytest.mark.parametrize("n,hq,hk,d,r,dtype", NORM)
def test_head_norm_rotate_vjp(fc, n, hq, hk, d, r, dtype):
    g, wide, x, gq, gk, pos, freq = norm_case(n, hq, hk, d, r, dtype)
    gy = normal(g, n, hq + hk, d, dtype=dtype)
    leaves = [None if t is None else t.double().requires_grad_(True) for t in (x, gq, gk, pos)]
    y = R.norm(leaves[0], hq, leaves[1], leaves[2], leaves[3], None if freq is None else freq.double(), 1e-6)
    bars = torch.autograd.grad(y, [t for t in leaves if t is not None], gy.double(), allow_unused=True)
    bars = [torch.zeros_like(l) if b is None else b for b, l in zip(bars, [t for t in leaves if t is not None])]
    xg = dev(wide)[:, 1: 1 + hq + hk]
    args = (xg, dev(gy), hq, dev(gq), dev(gk), dev(pos), dev(freq))
    got = fc.head_norm_rotate_vjp(*args)
    close(got[0], bars[0], R.u(dtype) * bars[0].abs() + VJP_TOL * bars[0].abs().max() + sub(dtype))
    for a, b in zip(got[1:3], bars[1:3]):
        close(a, b, VJP_TOL * b.abs().max())
    if r:
        close(got[3], bars[3], VJP_TOL * bars[3].abs().max())
    else:
        assert got[3] is None
    again = fc.head_norm_rotate_vjp(*args)
    assert all(torch.equal(a, b) for a, b in zip(got, again) if a is not None)


# ------------------------------------------------------------ node attention

def lens_ptr(lens, lead=0):
    return torch.tensor([lead] + [lead + sum(lens[: i + 1]) for i in range(len(lens))], dtype=torch.int32)


class Case:
    def __init__(self, recv, send, h, kv, d, dtype, cap=0.0, bias=True, hide=None, seed=0, lead=0, tail=0):
        """recv, send: lengths per structure (send None: self-attention); lead, tail: rows outside every structure."""
        g = gen(seed + h * d + sum(recv))
        self.h, self.kv, self.d, self.dtype, self.cap = h, kv, d, dtype, cap
        self.rp = lens_ptr(recv, lead)
        self.sp = self.rp if send is None else lens_ptr(send, lead)
        nr = int(self.rp[-1]) + tail
        ns = int(self.sp[-1]) + tail
        # queries, keys and values as column blocks of wider rows
        self.qw = normal(g, nr, h + 1, d, dtype=dtype)
        self.kw = normal(g, ns, 2 * kv + 1, d, dtype=dtype)
        self.g = normal(g, nr, h, d, dtype=dtype)
        self.pos = self.pos_send = self.slope = self.mask = None
        if bias:
            self.pos = torch.rand((nr, 3), generator=g) * 4
            self.pos_send = None if send is None else torch.rand((ns, 3), generator=g) * 4
            self.slope = torch.linspace(-0.1, 1.5, h)
        if hide is not None:
            self.mask = (torch.rand(ns, generator=g) >= hide).to(torch.uint8)
        self.scale = 1.3 * d ** -0.5

    def parts(self, qw, kw):
        return qw[:, 1:], kw[:, : self.kv], kw[:, self.kv: 2 * self.kv]

    def kwargs(self, move):
        return dict(pos=move(self.pos), pos_send=move(self.pos_send), slope=move(self.slope), scale=self.scale, cap=self.cap)

    def run(self, fc, vjp=True):
        q, k, v = self.parts(dev(self.qw), dev(self.kw))
        kw = dict(self.kwargs(dev), send_ptr=dev(self.sp), send_mask=dev(self.mask))
        out, lse, o32 = fc.node_attention(q, k, v, dev(self.rp), residual=True, **kw)
        if not vjp:
            return out, lse, o32
        return (out, lse, o32), fc.node_attention_vjp(q, k, v, o32, lse, dev(self.g), dev(self.rp), **kw)

    def reference(self):
        q, k, v = (t.double().requires_grad_(True) for t in self.parts(self.qw, self.kw))
        dbl = {n: (t.double().requires_grad_(True) if isinstance(t, torch.Tensor) else t)
               for n, t in self.kwargs(lambda t: t).items()}
        out, lse, w = R.attention(q, k, v, self.rp, self.sp, mask=self.mask, **dbl)
        names = ["q", "k", "v"] + [n for n in ("pos", "pos_send", "slope") if dbl[n] is not None]
        leaves = dict(q=q, k=k, v=v, **dbl)
        got = torch.autograd.grad(out, [leaves[n] for n in names], self.g.double(), allow_unused=True) if out.requires_grad \
            else [None] * len(names)
        bars = {n: torch.zeros_like(leaves[n]) if b is None else b for n, b in zip(names, got)}
        mags = R.attention_bounds(q.detach(), k.detach(), v.detach(), self.g.double(), w, self.dtype, self.scale)
        return out.detach(), lse, bars, mags

    def check(self, fc):
        ref, lse, bars, (mo, mq, mk, mv, row, q32, k32) = self.reference()
        (out, l, o32), got = self.run(fc)
        t = R.u(self.dtype) if self.dtype != F32 else 0.0
        big = lambda a: float(a.abs().max()) if a.numel() else 0.0  # noqa: E731
        low = sub(self.dtype)
        close(out, ref, R.u(self.dtype) * ref.abs() + t * mo + FWD_TOL * big(ref) + low)
        # the weights as two 16-bit terms: one rounding of what the first left
        close(o32, ref, t * t * mo + FWD_TOL * big(ref))
        fin = torch.isfinite(lse)
        assert torch.equal(torch.isfinite(l.cpu()), fin) and bool((l.cpu()[~fin] == -math.inf).all())
        close(l.cpu()[fin], lse[fin], FWD_TOL * max(1.0, big(lse[fin])))
        # an error t*t of delta moves every ds of the row by that share of P
        for a, b, m, w in ((got[0], bars["q"], mq, q32), (got[1], bars["k"], mk, k32), (got[2], bars["v"], mv, 0.0)):
            close(a, b, w + R.u(self.dtype) * b.abs() + (t + t * t) * m + VJP_TOL * big(b) + low + t * t * big(row) * self.scale)
        for a, n in zip(got[3:], ("pos", "pos_send", "slope")):
            if n not in bars:
                assert a is None
                continue
            far = 4 * 3 ** 0.5 if n == "slope" else 1.0    # the largest distance
            share = float(row.sum()) if n == "slope" else float(row.sum(1).max()) * 2 if n == "pos" else float(row.sum())
            close(a, bars[n], VJP_TOL * big(bars[n]) + t * t * share * 1.5 * far)
        if self.dtype != F32:     # without the residual the weights are one 16-bit term
            q, k, v = self.parts(dev(self.qw), dev(self.kw))
            one = fc.node_attention(q, k, v, dev(self.rp), send_ptr=dev(self.sp), send_mask=dev(self.mask), **self.kwargs(dev))
            close(one[0], ref, R.u(self.dtype) * ref.abs() + t * mo + FWD_TOL * big(ref) + low)
        assert fc.device_error() == 0
        again = self.run(fc)
        for a, b in zip([out, l, o32, *got], [*again[0], *again[1]]):
            assert (a is None and b is None) or torch.equal(a, b)


ATTN = {
    "one node": dict(recv=[1], send=None, h=1, kv=1, d=8, dtype=F32),
    "one node bf16": dict(recv=[1], send=None, h=2, kv=1, d=16, dtype=BF16),
    "lengths": dict(recv=[5, 0, 64, 1, 65, 130], send=None, h=4, kv=4, d=16, dtype=F32),
    "lengths bf16": dict(recv=[5, 0, 64, 1, 65, 130], send=None, h=4, kv=4, d=32, dtype=BF16, cap=3.0),
    "shared heads": dict(recv=[33, 90], send=None, h=6, kv=2, d=40, dtype=F32, cap=2.0),
    "shared heads f16": dict(recv=[33, 90], send=None, h=10, kv=2, d=64, dtype=F16, cap=5.0, hide=0.3),
    "one key head": dict(recv=[70, 3], send=None, h=7, kv=1, d=72, dtype=BF16),
    "wide f32": dict(recv=[100, 41], send=None, h=2, kv=2, d=128, dtype=F32, hide=0.2),
    "wide bf16": dict(recv=[100, 141], send=None, h=4, kv=2, d=128, dtype=BF16, cap=4.0),
    "wide f16": dict(recv=[129], send=None, h=2, kv=2, d=112, dtype=F16, bias=False),
    "no bias": dict(recv=[77, 20], send=None, h=3, kv=3, d=24, dtype=F32, bias=False),
    "apart": dict(recv=[3, 0, 70, 5], send=[100, 7, 0, 33], h=4, kv=2, d=48, dtype=F32, cap=3.0),
    "apart bf16": dict(recv=[3, 0, 70, 5], send=[100, 7, 0, 33], h=4, kv=2, d=64, dtype=BF16, hide=0.5),
    "outside rows": dict(recv=[20, 70], send=None, h=2, kv=2, d=32, dtype=F32, lead=5, tail=150),
    "all hidden": dict(recv=[9, 66], send=None, h=2, kv=1, d=16, dtype=F32, hide=1.1),
    "probe split": dict(recv=[1, 1], send=[3000, 2100], h=4, kv=2, d=64, dtype=F32, cap=3.0, hide=0.1),
    "probe split bf16": dict(recv=[2, 1, 1], send=[4000, 0, 1500], h=8, kv=2, d=128, dtype=BF16),
    "few rows": dict(recv=[3, 20, 0, 9], send=[130, 40, 5, 700], h=6, kv=3, d=40, dtype=F32, cap=9.0, hide=0.2),
    "few rows wide": dict(recv=[5, 1], send=[300, 65], h=8, kv=2, d=128, dtype=F32),
    "few rows f16": dict(recv=[7, 1, 2], send=[1, 129, 33], h=4, kv=1, d=16, dtype=F16, bias=False),
    "few rows, all hidden": dict(recv=[7, 1], send=[50, 129], h=4, kv=1, d=64, dtype=BF16, hide=1.1),
    "long": dict(recv=[1100], send=None, h=2, kv=1, d=64, dtype=F16, cap=3.0),
    "long f32": dict(recv=[1100], send=None, h=2, kv=2, d=64, dtype=F32),
    # enough blocks that the senders are not split: more tiles than a block has stages
    "many tiles": dict(recv=[1300], send=None, h=16, kv=16, d=32, dtype=BF16, cap=6.0),
    "many tiles wide": dict(recv=[900, 650], send=None, h=16, kv=8, d=128, dtype=F16, hide=0.1),
    "many tiles no bias": dict(recv=[1250], send=None, h=16, kv=16, d=64, dtype=BF16, bias=False),
    # groups of heads that do not divide a tile of 64 rows, masks, both sides apart
    "group of 3": dict(recv=[300, 131], send=None, h=6, kv=2, d=64, dtype=BF16, cap=8.0),
    "group of 5": dict(recv=[260], send=None, h=10, kv=2, d=96, dtype=F16, hide=0.2),
    "group of 40": dict(recv=[150], send=None, h=40, kv=1, d=48, dtype=BF16, bias=False, cap=5.0),
    "apart wide": dict(recv=[150, 0, 200], send=[400, 30, 300], h=2, kv=2, d=128, dtype=BF16, cap=9.0, hide=0.3),
    "few receivers": dict(recv=[130, 100], send=[1900, 900], h=2, kv=2, d=32, dtype=F16),
    "few senders": dict(recv=[1500, 900], send=[150, 140], h=4, kv=2, d=64, dtype=BF16, cap=9.0),
    "few senders f32": dict(recv=[1500, 900], send=[50, 70], h=4, kv=2, d=24, dtype=F32),
    "outside rows bf16": dict(recv=[200, 270], send=None, h=2, kv=2, d=64, dtype=BF16, lead=5, tail=350),
    "narrow, many tiles": dict(recv=[700, 400], send=None, h=4, kv=2, d=24, dtype=F16, cap=6.0, hide=0.1),
    "narrow apart": dict(recv=[400, 350], send=[90, 1500], h=3, kv=3, d=8, dtype=BF16),
    "many": dict(recv=[(7 * i) % 23 for i in range(300)], send=None, h=2, kv=2, d=16, dtype=F32),
}


@pytest.mark.parametrize("name", list(ATTN))
def test_attention(fc, name):
    Case(**ATTN[name]).check(fc)


def test_no_structures_is_all_empty(fc):
    q = torch.randn(70, 2, 16, device="cuda")
    ptr = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse, o32 = fc.node_attention(q, q, q, ptr, residual=True)
    assert not out.any() and bool((lse == -math.inf).all())
    bars = fc.node_attention_vjp(q, q, q, o32, lse, q, ptr)
    assert not any(bool(b.any()) for b in bars[:3])


def test_nan_stays_in_its_structure_and_behind_the_mask(fc):
    """NaN and infinities in one structure, and in hidden senders, reach no other row."""
    for dtype in (F32, BF16):
        c = Case([40, 30, 50], None, 4, 2, 32, dtype, cap=3.0, hide=0.2)
        c.mask[45] = 0
        clean, cbars = c.run(fc)
        hidden = int((c.mask[70:120] == 0).nonzero()[0]) + 70
        c.kw[hidden] = float("nan")
        c.kw[45] = float("inf")
        got, bars = c.run(fc)
        for a, b in zip([*clean, *cbars], [*got, *bars]):
            assert a is None or torch.equal(a, b)
        # a whole structure of NaN; the slope gradient sums over all structures
        c.qw[:40], c.kw[:40], c.pos[:40] = (float("nan"),) * 3
        got, bars = c.run(fc)
        for a, b in zip([*clean, *cbars[:4]], [*got, *bars[:4]]):
            assert torch.equal(a[40:], b[40:])


@pytest.mark.parametrize("d,group", [(64, 1), (128, 2)])
def test_nan_stays_in_its_structure_on_the_tensor_cores(fc, d, group):
    """The same at lengths that the tcgen05 kernels take; structures end inside their tiles of 64 and 128 rows."""
    c = Case([150, 130, 210], None, 4, 4 // group, d, BF16, cap=3.0, hide=0.2)
    c.mask[170] = 0
    clean, cbars = c.run(fc)
    hidden = int((c.mask[280:490] == 0).nonzero()[0]) + 280
    c.kw[hidden] = float("nan")
    c.kw[170] = float("inf")
    got, bars = c.run(fc)
    for a, b in zip([*clean, *cbars], [*got, *bars]):
        assert a is None or torch.equal(a, b)
    c.qw[:150], c.kw[:150], c.pos[:150] = (float("nan"),) * 3
    got, bars = c.run(fc)
    for a, b in zip([*clean, *cbars[:4]], [*got, *bars[:4]]):
        assert torch.equal(a[150:], b[150:])
    assert fc.device_error() == 0


@pytest.mark.parametrize("power", [-10, 10])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_score_factors_far_from_one(fc, power, d):
    """Queries and keys times 2^power and scale times 4^-power (exact in BF16) are the same scores, however large or
    small scale / cap is then; the bounds scale along."""
    c = Case([310], None, 2, 2, d, BF16, cap=3.0)
    c.qw *= 2.0 ** power
    c.kw[:, : c.kv] *= 2.0 ** power
    c.scale *= 4.0 ** -power
    c.check(fc)


def test_sizes_past_32_bits_are_refused(fc):
    """Counts that a 32-bit int cannot hold, from expanded tensors of one element: refused before any launch."""
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = torch.zeros(1, 1, 8, device="cuda")
    for n in (2 ** 31, 2 ** 32 + 5):
        with pytest.raises(ValueError):
            fc.species_embed(one.expand(n), torch.zeros(2, 8, device="cuda"))
        with pytest.raises(ValueError):
            fc.species_embed_vjp(one, torch.zeros(1, 8, device="cuda"), n)
        with pytest.raises(ValueError):
            fc.head_norm_rotate(rows.expand(n, 1, 8), 1)
        with pytest.raises(ValueError):
            fc.node_attention(rows, rows.expand(n, 1, 8), rows.expand(n, 1, 8), one, one)
        with pytest.raises(ValueError):
            fc.node_attention(rows, rows, rows, one.expand(n))
    with pytest.raises(ValueError):
        fc.species_embed_vjp(one, torch.zeros(1, 8, device="cuda"), 3, lmax=-1)


@pytest.mark.parametrize("dtype,d", [(F32, 32), (BF16, 64)])
def test_one_side_without_rows(fc, dtype, d):
    """No senders at all: zero rows, log-sum -infinity, zero gradients.  No receivers at all: the senders' gradients 0."""
    q, g = (torch.randn(150, 4, d, device="cuda").to(dtype) for _ in range(2))
    k = torch.empty(0, 2, d, dtype=dtype, device="cuda")
    pos, none, slope = torch.rand(150, 3, device="cuda"), torch.empty(0, 3, device="cuda"), torch.ones(4, device="cuda")
    ptr, zero = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 20, 150], [0, 0, 0]))
    out, lse, o32 = fc.node_attention(q, k, k, ptr, zero, pos, none, slope, residual=True)
    assert not out.any() and bool((lse == -math.inf).all())
    bars = fc.node_attention_vjp(q, k, k, o32, lse, g, ptr, zero, pos, none, slope)
    assert not any(bool(b.any()) for b in bars)
    k, q0 = q[:, :2], q[:0]
    out, lse, o32 = fc.node_attention(q0, k, k, zero, ptr, none, pos, slope, residual=True)
    assert out.shape == (0, 4, d) and lse.shape == (0, 4)
    bars = fc.node_attention_vjp(q0, k, k, o32, lse, q0, zero, ptr, none, pos, slope)
    assert not any(bool(b.any()) for b in bars)


@pytest.mark.parametrize("dtype", [F32, F16])
def test_many_structures_of_one_node(fc, dtype):
    """70,000 structures of one node: its weight is 1, so that the output is the value row and the log-sum the score."""
    n = 70000
    f = torch.randn(n, 3, 16, device="cuda").to(dtype)
    q, k, v = f[:, :1], f[:, 1:2], f[:, 2:]
    ptr = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    out, lse, o32 = fc.node_attention(q, k, v, ptr, residual=True)
    # FP32 values go in as two TF32 ones of 11 bits: a part of 2^-10 is left by the first, of that again by the second
    close(out, v.double().cpu(), (2.0 ** -20 if dtype == F32 else 0.0) * v.double().abs().cpu())
    ref = (q.double() * k.double()).sum(-1).cpu() / 4
    close(lse, ref, FWD_TOL * float(ref.abs().max()))
    qb, kb, vb = fc.node_attention_vjp(q, k, v, o32, lse, v, ptr)[:3]
    # P = exp2(t - log-sum) is 1 up to the rounding of both; in FP16 it is then rounded to 1 or a neighbour
    close(vb, v.double().cpu(), (2 * R.u(dtype) + VJP_TOL) * v.double().abs().cpu() + sub(dtype))


def test_offsets_past_32_bits(fc):
    """Rows 65,536 values apart, 4.6e9 in all: the same results as from packed copies."""
    n, ld = 70000, 65536
    wide = torch.empty(n, ld, dtype=BF16, device="cuda")
    col = ld - 3 * 2 * 64
    wide[:, col:] = torch.randn(n, 3 * 2 * 64, device="cuda").to(BF16)
    f = wide[:, col:].unflatten(1, (6, 64))
    q, k, v = f[:, :2], f[:, 2:4], f[:, 4:]
    packed = [t.contiguous() for t in (q, k, v)]
    pos, freq = torch.rand(n, 3, device="cuda") * 9, torch.rand(3, 32, device="cuda")
    assert torch.equal(fc.head_norm_rotate(f[:, :4], 2, pos=pos, freq=freq),
                       fc.head_norm_rotate(f[:, :4].contiguous(), 2, pos=pos, freq=freq))
    for lens in (350, 20):    # structures for the tensor cores, and short ones
        ptr = torch.arange(0, n + 1, lens, dtype=torch.int32, device="cuda")
        kw = dict(pos=pos, slope=torch.ones(2, device="cuda"))
        a, b = (fc.node_attention(*t, ptr, residual=True, **kw) for t in ((q, k, v), packed))
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        a, b = (fc.node_attention_vjp(*t, a[2], a[1], g, ptr, **kw) for t, g in (((q, k, v), v), (packed, packed[2])))
        assert all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)
    del wide, f, q, k, v
    # node features of 4.9e9 values
    species = torch.arange(n, dtype=torch.int32, device="cuda") % 5
    table = torch.randn(5, 4096, device="cuda").to(BF16)
    x = fc.species_embed(species, table, lmax=3)
    assert torch.equal(x[-7:, :4096], table[species[-7:].long()]) and not x[-7:, 4096:].any()
    bar = fc.species_embed_vjp(species, x, 5, lmax=3)
    # 14,000 equal values a species: 8 groups of 16 in a span (at most 16 + 8 roundings), 110 spans over 32 warps
    # (4 + 5): fewer than 64 roundings of 2^-24 on the way of any
    close(bar, table.double().cpu() * 14000, 2 ** -18 * table.double().abs().cpu() * 14000)


def test_coincident_nodes(fc):
    """Distance 0 between different nodes: no gradient, and no NaN."""
    c = Case([30], None, 2, 2, 16, F32)
    c.pos[10:20] = c.pos[0]
    c.check(fc)


def test_attention_gradients_against_differences(fc):
    """The gradients along random directions against central differences of the 64-bit forward."""
    c = Case([25, 14], None, 4, 2, 16, F32, cap=3.0, hide=0.1)
    _, bars = c.run(fc)
    q, k, v = (t.double() for t in c.parts(c.qw, c.kw))
    pos, slope, gy = c.pos.double(), c.slope.double(), c.g.double()
    f = lambda q, k, v, pos, slope: float((R.attention(  # noqa: E731
        q, k, v, c.rp, c.sp, pos=pos, slope=slope, mask=c.mask, scale=c.scale, cap=c.cap)[0] * gy).sum())
    at = [q, k, v, pos, slope]
    for i, bar in zip(range(5), (bars[0], bars[1], bars[2], bars[3], bars[5])):
        way = torch.randn(at[i].shape, generator=gen(i), dtype=torch.float64)
        h = 1e-5
        step = lambda s: f(*[a + s * way if j == i else a for j, a in enumerate(at)])  # noqa: E731
        want = (step(h) - step(-h)) / (2 * h)
        have = float((bar.double().cpu() * way).sum())
        # a difference of step h: h^2 third derivatives, and 2^-52 |f| / h
        assert abs(have - want) <= 2e-4 * max(1.0, float((bar.double().cpu().abs() * way.abs()).sum()) * 0.05), (i, have, want)


def test_head_norm_gradients_against_differences(fc):
    g, wide, x, gq, gk, pos, freq = norm_case(30, 3, 2, 16, 6, F32, far=5.0)
    gy = normal(g, 30, 5, 16)
    got = fc.head_norm_rotate_vjp(x.cuda(), dev(gy), 3, dev(gq), dev(gk), dev(pos), dev(freq))
    at = [t.double() for t in (x, gq, gk, pos)]
    f = lambda *a: float((R.norm(a[0], 3, a[1], a[2], a[3], freq.double(), 1e-6) * gy.double()).sum())  # noqa: E731
    for i in range(4):
        way = torch.randn(at[i].shape, generator=gen(i), dtype=torch.float64)
        h = 1e-5
        want = (f(*[a + h * way if j == i else a for j, a in enumerate(at)])
                - f(*[a - h * way if j == i else a for j, a in enumerate(at)])) / (2 * h)
        have = float((got[i].double().cpu() * way).sum())
        assert abs(have - want) <= 2e-4 * max(1.0, 0.05 * float((got[i].double().cpu().abs() * way.abs()).sum())), i


# ------------------------------------------------------------ how calls are made

def test_wants_streams_and_workspaces(fc):
    c = Case([80, 40], None, 4, 2, 32, BF16, cap=3.0)
    (out, lse, o32), bars = c.run(fc)
    q, k, v = c.parts(dev(c.qw), dev(c.kw))
    kw = c.kwargs(dev)
    rp, g = dev(c.rp), dev(c.g)
    for want in (("q",), ("k",), ("v", "pos"), ("slope",)):
        got = fc.node_attention_vjp(q, k, v, o32, lse, g, rp, want=want, **kw)
        names = ("q", "k", "v", "pos", "pos_send", "slope")
        for n, a, b in zip(names, got, bars):
            assert (torch.equal(a, b) if n in want else a is None), n
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fc.node_attention(q, k, v, rp, stream=side, **kw)
    side.synchronize()
    plain = fc.node_attention(q, k, v, rp, **kw)
    assert torch.equal(got[0], plain[0]) and plain[2] is None
    need = fc.lib().fc_node_attention_vjp_workspace_size(
        __import__("ctypes").byref(fc.AttnDesc(1, 4, 2, 32, c.scale, c.cap)), 2, 120, 120)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    got = fc.node_attention_vjp(q, k, v, o32, lse, g, rp, workspace=ws, **kw)
    assert torch.equal(got[0], bars[0])
    with pytest.raises(fc.FlashCartError):
        fc.node_attention_vjp(q, k, v, o32, lse, g, rp, workspace=ws[:-16], **kw)
    for bad in (dict(g=g[:, :2]), dict(lse=lse[:5]), dict(out_f32=None), dict(rp=rp.long())):
        a = dict(dict(out_f32=o32, lse=lse, g=g, rp=rp), **bad)
        with pytest.raises((ValueError, TypeError)):
            fc.node_attention_vjp(q, k, v, a["out_f32"], a["lse"], a["g"], a["rp"], **kw)
    with pytest.raises(ValueError):
        fc.node_attention(q.transpose(0, 1), k, v, rp, **kw)
    with pytest.raises(TypeError):
        fc.node_attention(q, k.half(), v, rp, **kw)


def test_waits_give_up_then_recover(fc):
    """The tensor-core attention kernels' bounded waits at a bound of 1 ns: the calls return, the error word is set,
    and with the default bound back the same calls give the same results."""
    c = Case([700], None, 4, 4, 64, BF16, cap=8.0)
    clean, cbars = c.run(fc)
    assert fc.device_error() == 0
    fc.set_wait_timeout(1)
    try:
        c.run(fc)
        torch.cuda.synchronize()
        flag = fc.device_error()
    finally:
        fc.set_wait_timeout(0)
    assert flag == 1
    assert fc.device_error() == 0          # the word was cleared by the read
    got, bars = c.run(fc)
    assert fc.device_error() == 0
    for a, b in zip([*clean, *cbars], [*got, *bars]):
        assert a is None or torch.equal(a, b)


def test_calls_on_two_streams_at_once(fc):
    """Two steps running beside each other, each with its own scratch."""
    cases = [Case([500, 300], None, 4, 2, 64, BF16, cap=8.0, seed=s) for s in (1, 2)]
    want = [c.run(fc) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(c.run(fc))
    torch.cuda.synchronize()
    for i, (g, w) in enumerate(zip(got, want * 3)):
        for a, b in zip([*g[0], *g[1]], [*w[0], *w[1]]):
            assert a is None or torch.equal(a, b), i


def test_rows_of_two_calls_in_one_capture_share_nothing(fc):
    """Two captured graphs, replayed in turn, each with the scratch of its own pool."""
    cases = [Case([260, 140], None, 4, 2, 32, F16, cap=8.0, seed=s) for s in (3, 4)]
    want = [c.run(fc) for c in cases]
    dev_in = []
    for c in cases:
        q, k, v = c.parts(dev(c.qw), dev(c.kw))
        dev_in.append((q, k, v, dev(c.rp), dev(c.g), dict(c.kwargs(dev), send_ptr=dev(c.sp))))
    graphs, outs = [], []
    torch.cuda.synchronize()
    for q, k, v, rp, g, kw in dev_in:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = fc.node_attention(q, k, v, rp, residual=True, **kw)
            outs.append((o, fc.node_attention_vjp(q, k, v, o[2], o[1], g, rp, **kw)))
        graphs.append(graph)
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (o, b), (wo, wb) in zip(outs, want):
        for x, y in zip([*o, *b], [*wo, *wb]):
            assert x is None or torch.equal(x, y)


def test_capture_and_replay(fc):
    """Every entry point inside one captured graph, replayed on new inputs."""
    c = Case([50, 30], None, 4, 2, 32, F32, cap=3.0)
    q, k, v = (t.clone() for t in c.parts(dev(c.qw), dev(c.kw)))
    kw, rp, g = c.kwargs(dev), dev(c.rp), dev(c.g)
    species = torch.randint(0, 300, (80,), dtype=torch.int32, device="cuda")
    freq = torch.randn(3, 16, device="cuda")

    def step():
        out, lse, o32 = fc.node_attention(q, k, v, rp, residual=True, **kw)
        bars = fc.node_attention_vjp(q, k, v, o32, lse, g, rp, **kw)
        y = fc.head_norm_rotate(q, 3, pos=kw["pos"], freq=freq)
        nb = fc.head_norm_rotate_vjp(q, g, 3, pos=kw["pos"], freq=freq)
        x = fc.species_embed(species, torch.ones(300, 8, device="cuda"), lmax=1)
        tb = fc.species_embed_vjp(species, g.reshape(80, -1), 300, lmax=1)
        return [t for t in (out, lse, *bars, y, *nb, x, tb) if t is not None]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        for t in (q, k, v, g):
            t.copy_(torch.randn_like(t))
        species.copy_(torch.randint(0, 300, (80,), dtype=torch.int32, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, step()):
            assert torch.equal(a, b)


def test_operators_together(fc):
    """Species table -> features -> projection -> norm and rotation -> attention -> energy, and the gradients of the
    energy down to the table, the norm weights, the slopes and the positions (forces) against automatic
    differentiation of the 64-bit forms."""
    g = gen(3)
    lens, C, H, D, Rp = [30, 1, 47], 32, 4, 16, 6
    rp = lens_ptr(lens)
    n = int(rp[-1])
    species = torch.randint(0, 5, (n,), generator=g, dtype=torch.int32)
    table, w = normal(g, 5, C), normal(g, C, 3 * H * D, scale=C ** -0.5)
    gq, gk = 1 + normal(g, D, scale=0.2), 1 + normal(g, D, scale=0.2)
    pos, freq, slope = torch.rand((n, 3), generator=g) * 5, normal(g, 3, Rp), torch.linspace(0.1, 1.0, H)
    go = normal(g, n, H, D)                               # the energy is <go, attention>

    dt = [t.double().requires_grad_(True) for t in (table, gq, gk, pos, slope)]
    x = dt[0][species.long()] * 1.5
    fused = (x @ w.double()).reshape(n, 3 * H, D)
    qk = R.norm(fused[:, : 2 * H], H, dt[1], dt[2], dt[3], freq.double(), 1e-6)
    out, _, _ = R.attention(qk[:, :H], qk[:, H:], fused[:, 2 * H:], rp, rp, pos=dt[3], slope=dt[4], cap=8.0)
    want = torch.autograd.grad((out * go.double()).sum(), dt)

    s, T, W, P, F = dev(species), dev(table), dev(w), dev(pos), dev(freq)
    x = fc.species_embed(s, T, lmax=1, scale=1.5)
    assert not x[:, C:].any()
    fused = (x[:, :C] @ W).reshape(n, 3 * H, D)
    hn = dict(gamma_q=dev(gq), gamma_k=dev(gk), pos=P, freq=F)
    qk = fc.head_norm_rotate(fused[:, : 2 * H], H, **hn)
    kw = dict(pos=P, slope=dev(slope), cap=8.0)
    q, k, v = qk[:, :H], qk[:, H:], fused[:, 2 * H:]
    got, lse, o32 = fc.node_attention(q, k, v, dev(rp), residual=True, **kw)
    qb, kb, vb, pb, _, sb = fc.node_attention_vjp(q, k, v, o32, lse, dev(go), dev(rp), **kw)
    xb, gqb, gkb, pb2 = fc.head_norm_rotate_vjp(fused[:, : 2 * H], torch.cat([qb, kb], 1), H, **hn)
    fb = torch.cat([xb, vb], 1).reshape(n, -1)
    gx = torch.zeros_like(x)
    gx[:, :C] = fb @ W.T
    tb = fc.species_embed_vjp(s, gx, 5, lmax=1, scale=1.5)
    close(got, out.detach(), FWD_TOL * out.abs().max().detach())
    for a, b in zip((tb, gqb, gkb, pb + pb2, sb), want):
        close(a, b, VJP_TOL * b.abs().max())
