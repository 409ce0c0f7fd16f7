"""Cases, plain forms and 64-bit definitions of the node operators: species embedding, head norm with position
rotation, and node attention, each with its gradient.

The plain forms are elementary torch operations in 32 bits (64 where angles of far positions or long sums need
them), rounded once at the end.  With `own` set, the same passes call the library."""
import math

import numpy as np
import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one 1000-atom crystal enters a rank-3 model: the rank-0 block of its node features, the rest zero
        dict(name="embed 1000 atoms", op="embed", n=1000, types=100, channels=128, lmax=3, scale=1.0, skew=2.0, dtype="f32"),
        # a large batch of structures, two ranks of features
        dict(name="embed 65537 atoms", op="embed", n=65537, types=100, channels=128, lmax=2, scale=0.5, skew=2.0, dtype="f32"),
        # training on a batch of organic structures: a few elements take nearly all atoms
        dict(name="embed grad few types", op="embed_vjp", n=100003, types=100, channels=128, lmax=2, scale=0.5, skew=4.0, dtype="f32"),
        # a large table of site types with wide rows
        dict(name="embed grad many types", op="embed_vjp", n=50001, types=32000, channels=512, lmax=0, scale=2.0, skew=1.0, dtype="bf16"),
        # queries and keys of one 1000-atom crystal
        dict(name="norm 1000 atoms", op="norm", n=1000, hq=8, hk=8, hv=0, dim=16, pairs=8, far=0.0, dtype="f32"),
        # queries and keys inside a fused projection of a large batch, shared key heads
        dict(name="norm 65536 atoms", op="norm", n=65536, hq=16, hk=4, hv=4, dim=64, pairs=32, far=5000.0, dtype="bf16"),
        # a training step at 4096 nodes, part of each head rotated
        dict(name="norm step 4096", op="norm_step", n=4096, hq=8, hk=8, hv=8, dim=32, pairs=12, far=100.0, dtype="f32"),
        # a training step of a large batch with wide heads
        dict(name="norm step 32769", op="norm_step", n=32769, hq=8, hk=2, hv=2, dim=128, pairs=64, far=1000.0, dtype="bf16"),
        # a training step on a batch of small molecules, FP32 as the rest of the model
        dict(name="attn step molecules", op="attn_step", structures=128, lo=9, hi=70, recv=0, hq=8, hk=8, dim=16, cap=0.0, bias=True, hide=0.0, dtype="f32"),
        # a few probe atoms, one per structure, against large fixed surroundings
        dict(name="attn probes", op="attn", structures=4, lo=5000, hi=9001, recv=1, hq=16, hk=4, dim=64, cap=0.0, bias=True, hide=0.1, dtype="bf16"),
        # one large periodic cell, capped scores
        dict(name="attn 16384 atoms", op="attn", structures=1, lo=16384, hi=16384, recv=0, hq=8, hk=8, dim=64, cap=20.0, bias=True, hide=0.0, dtype="bf16"),
        # a training step on large ragged structures, shared key heads, some senders hidden
        dict(name="attn step ragged", op="attn_step", structures=5, lo=700, hi=2300, recv=0, hq=8, hk=2, dim=128, cap=20.0, bias=True, hide=0.05, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_vjp", "norm", "norm_step", "attn", "attn", "attn_step", "attn_step"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op.startswith("embed"):
        # single atoms to large batches; a handful of elements to a large table of site types
        channels = 8 * _log(rng, 1, 128)
        lmax = rng.randint(0, 3)
        n = _log(rng, 1, min(131072, 2 ** 27 // ((lmax + 1) ** 2 * channels)))
        return dict(op=op, n=n, types=_log(rng, 1, 40000), channels=channels, lmax=lmax, scale=rng.choice([1.0, 0.5, 11.3]),
                    skew=rng.choice([1.0, 2.0, 4.0]), dtype=dtype)
    hk = rng.randint(1, 8)
    hq = hk * rng.choice([1, 1, 2, 3, 4])
    dim = 8 * rng.randint(1, 16)
    if op.startswith("norm"):
        n = _log(rng, 1, 2 ** 26 // ((hq + 2 * hk) * dim))
        return dict(op=op, n=n, hq=hq, hk=hk, hv=rng.choice([0, hk]), dim=dim, pairs=rng.randint(0, dim // 2),
                    far=rng.choice([0.0, 100.0, 5000.0]), dtype=dtype)
    # whole structures up to 4096 nodes, or 1 to 40 probe atoms each in surroundings of up to 8192
    recv = rng.choice([0, 0, 0, 1, rng.randint(2, 40)])
    structures = _log(rng, 1, 128)
    share = structures * hq * dim
    most = min(8192, 2 ** 25 // share) if recv else min(4096, math.isqrt(2 ** 35 // share))
    hi = _log(rng, 2, most)
    return dict(op=op, structures=structures, lo=rng.randint(1, hi), hi=hi, recv=recv, hq=hq, hk=hk, dim=dim, cap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                bias=rng.random() < 0.8, hide=rng.choice([0.0, 0.1, 0.5]), dtype=dtype)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _lengths(case):
    """Senders of each structure, between lo and hi: the same for every seed, as are all sizes."""
    r = np.random.Generator(np.random.PCG64([case["structures"], case["lo"], case["hi"]]))
    return [int(v) for v in r.integers(case["lo"], case["hi"] + 1, case["structures"])]


def _pointer(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g, t = _gen(seed), DTYPE[case["dtype"]]
    op = case["op"]
    if op.startswith("embed"):
        # elements are unevenly frequent: a power of a uniform variate, spread over the table by a permutation
        n, v, c = case["n"], case["types"], case["channels"]
        u = torch.rand(n, generator=g, device="cuda") ** case["skew"]
        order = torch.randperm(v, generator=g, device="cuda")
        st = dict(op=op, case=case, species=order[(u * v).long().clamp_(max=v - 1)].int())
        if op == "embed":
            st["table"] = _normal(g, (v, c), t)
        else:
            st["g"] = _normal(g, (n, (case["lmax"] + 1) ** 2 * c), t)
        return st
    if op.startswith("norm"):
        n, hq, hk, d, p = case["n"], case["hq"], case["hk"], case["dim"], case["pairs"]
        fused = _normal(g, (n, hq + hk + case["hv"], d), t, 1.5)
        st = dict(op=op, case=case, x=fused[:, : hq + hk],
                  gq=1 + _normal(g, (d,), scale=0.2), gk=1 + _normal(g, (d,), scale=0.2), pos=None, freq=None)
        if p:
            # coordinates in a 20 A box, far from the origin where a trajectory has drifted; wavelengths of 2 to 60 A
            st["pos"] = torch.rand((n, 3), generator=g, device="cuda") * 20 + case["far"]
            way = _normal(g, (3, p))
            wave = 2 * 30 ** torch.rand(p, generator=g, device="cuda")
            st["freq"] = way / way.norm(dim=0, keepdim=True) * (2 * math.pi / wave)
        if op == "norm_step":
            st["g"] = _normal(g, (n, hq + hk, d), t)
        return st
    lens = _lengths(case)
    recv = [case["recv"]] * len(lens) if case["recv"] else lens
    nr, ns, hq, hk, d = sum(recv), sum(lens), case["hq"], case["hk"], case["dim"]
    st = dict(op=op, case=case, recv_ptr=_pointer(recv), send_ptr=_pointer(lens), most=(max(recv), max(lens)),
              scale=d ** -0.5, slope=None, pos=None, pos_send=None, mask=None)
    if case["recv"]:
        st["q"] = _normal(g, (nr, hq, d), t)
        fused = _normal(g, (ns, 2 * hk, d), t)
        st["k"], st["v"] = fused[:, :hk], fused[:, hk:]
    else:
        # one fused projection, whose column blocks are the queries, keys and values
        fused = _normal(g, (nr, hq + 2 * hk, d), t)
        st["q"], st["k"], st["v"] = fused[:, :hq], fused[:, hq: hq + hk], fused[:, hq + hk:]
    if case["bias"]:
        # atoms at the density of organic matter (0.1 per cubic A); one slope per head
        side = torch.tensor([(v / 0.1) ** (1 / 3) for v in lens], device="cuda")
        at = lambda ls: torch.repeat_interleave(side, torch.tensor(ls, device="cuda"))[:, None]  # noqa: E731
        send = torch.rand((ns, 3), generator=g, device="cuda") * at(lens)
        st["pos"] = torch.rand((nr, 3), generator=g, device="cuda") * at(recv) if case["recv"] else send
        st["pos_send"] = send if case["recv"] else None
        st["slope"] = 2.0 ** -torch.linspace(0.0, 5.0, hq, device="cuda")
    if case["hide"]:
        st["mask"] = (torch.rand(ns, generator=g, device="cuda") >= case["hide"]).to(torch.uint8)
    if op == "attn_step":
        st["g"] = _normal(g, (nr, hq, d), t)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    from cartesian_tensor_products_b200 import flashcart as fc
    op, c = st["op"], st["case"]
    if op == "embed":
        return fc.species_embed(st["species"], st["table"], lmax=c["lmax"], scale=c["scale"])
    if op == "embed_vjp":
        return fc.species_embed_vjp(st["species"], st["g"], c["types"], lmax=c["lmax"], scale=c["scale"])
    if op.startswith("norm"):
        with_ = dict(gamma_q=st["gq"], gamma_k=st["gk"], pos=st["pos"], freq=st["freq"], eps=EPS)
        y = fc.head_norm_rotate(st["x"], c["hq"], **with_)
        if op == "norm":
            return y
        xb, gqb, gkb, pb = fc.head_norm_rotate_vjp(st["x"], st["g"], c["hq"], **with_)
        return dict(y=y, x=xb, gq=gqb, gk=gkb, **({"pos": pb} if st["pos"] is not None else {}))
    with_ = dict(send_ptr=st["send_ptr"], pos=st["pos"], pos_send=st["pos_send"], slope=st["slope"], send_mask=st["mask"],
                 scale=st["scale"], cap=c["cap"])
    if op == "attn":
        out, lse, _ = fc.node_attention(st["q"], st["k"], st["v"], st["recv_ptr"], **with_)
        return dict(out=out, lse=lse)
    out, lse, o32 = fc.node_attention(st["q"], st["k"], st["v"], st["recv_ptr"], residual=True, **with_)
    qb, kb, vb, pb, psb, sb = fc.node_attention_vjp(st["q"], st["k"], st["v"], o32, lse, st["g"], st["recv_ptr"], **with_)
    res = dict(out=out, lse=lse, q=qb, k=kb, v=vb)
    if st["pos"] is not None:
        res.update(pos=pb, slope=sb)
        if st["pos_send"] is not None:
            res["pos_send"] = psb
    return res


def _plain(st):
    op = st["op"]
    if op == "embed":
        return _plain_embed(st)
    if op == "embed_vjp":
        return _plain_embed_vjp(st)
    if op.startswith("norm"):
        return _plain_norm(st, op == "norm_step")
    return _plain_attn(st, op == "attn_step")


def _plain_embed(st):
    c, t = st["case"], st["table"]
    n, ch = c["n"], c["channels"]
    out = torch.zeros((n, (c["lmax"] + 1) ** 2 * ch), dtype=t.dtype, device=t.device)
    out[:, :ch] = (t[st["species"].long()].float() * c["scale"]).to(t.dtype)
    return out


def _plain_embed_vjp(st):
    c, g = st["case"], st["g"]
    # a frequent species sums tens of thousands of rows: 64 bits
    bar = torch.zeros((c["types"], c["channels"]), dtype=torch.float64, device=g.device)
    bar.index_add_(0, st["species"].long(), g[:, : c["channels"]].double())
    return (bar * c["scale"]).float()


def _plain_norm(st, step):
    c, x = st["case"], st["x"].float()
    hq, hk, d, p = c["hq"], c["hk"], c["dim"], c["pairs"]
    gam = torch.cat([st["gq"].expand(hq, d), st["gk"].expand(hk, d)])
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xn = x * r
    u = xn * gam
    if p:
        th = st["pos"].double() @ st["freq"].double()
        cs, sn = torch.cos(th).float()[:, None], torch.sin(th).float()[:, None]
        a, b = u[..., :p], u[..., p:2 * p]
        y = torch.cat([a * cs - b * sn, a * sn + b * cs, u[..., 2 * p:]], -1)
    else:
        y = u
    if not step:
        return y.to(st["x"].dtype)
    g = st["g"].float()
    ub, res = g, {}
    if p:
        ga, gb = g[..., :p], g[..., p:2 * p]
        ub = torch.cat([ga * cs + gb * sn, gb * cs - ga * sn, g[..., 2 * p:]], -1)
        thb = (gb * y[..., :p] - ga * y[..., p:2 * p]).sum(1)
        res["pos"] = (thb.double() @ st["freq"].double().T).float()
    gamb = (ub * xn).double().sum(0)
    w = ub * gam
    xb = r * (w - xn * (w * xn).mean(-1, keepdim=True))
    return dict(y=y.to(st["x"].dtype), x=xb.to(st["x"].dtype), gq=gamb[:hq].sum(0).float(), gk=gamb[hq:].sum(0).float(), **res)


def _plain_attn(st, step):
    c = st["case"]
    hq, hk, d, cap, t = c["hq"], c["hk"], c["dim"], c["cap"], st["q"].dtype
    dev, grp = st["q"].device, hq // hk
    # structures padded to the longest: rows [B, L] of the packed arrays, the rest masked
    at, live = [], []
    for ptr, most in ((st["recv_ptr"].long(), st["most"][0]), (st["send_ptr"].long(), st["most"][1])):
        i = torch.arange(most, device=dev)[None]
        ok = i < (ptr[1:] - ptr[:-1])[:, None]
        at.append(torch.where(ok, ptr[:-1, None] + i, 0))
        live.append(ok)
    (ir, js), (okr, oks) = at, live
    if st["mask"] is not None:
        oks = oks & (st["mask"][js] != 0)
    rows, cols = ir[live[0]], js[live[1]]
    q = st["q"][ir].float().transpose(1, 2)                                  # [B, hq, Lr, d]
    k = st["k"][js].float().transpose(1, 2).repeat_interleave(grp, 1)        # [B, hq, Ls, d]
    v = st["v"][js].float().transpose(1, 2).repeat_interleave(grp, 1)
    s = (q @ k.transpose(2, 3)) * st["scale"]
    th = torch.tanh(s / cap) if cap else None
    if cap:
        s = th * cap
    if st["pos"] is not None:
        ps = st["pos"] if st["pos_send"] is None else st["pos_send"]
        dx = st["pos"][ir][:, :, None] - ps[js][:, None]                     # [B, Lr, Ls, 3]
        dist = (dx * dx).sum(-1).sqrt()
        s = s - st["slope"][:, None, None] * dist[:, None]
    s = torch.where(oks[:, None, None], s, -math.inf)
    m = s.max(-1, keepdim=True).values
    e = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    del s
    z = e.sum(-1, keepdim=True)
    lse = (m + torch.log(z))[..., 0]
    pr = e / torch.where(z == 0, 1.0, z)
    del e
    o = pr @ v
    pack = lambda a, i, ok, n: a.transpose(1, 2)[ok].new_empty((n,) + a.transpose(1, 2).shape[2:]).index_copy_(0, i, a.transpose(1, 2)[ok])  # noqa: E731
    nr, ns = st["q"].shape[0], st["k"].shape[0]
    res = dict(out=pack(o, rows, okr, nr).to(t), lse=pack(lse[..., None], rows, okr, nr)[..., 0])
    if not step:
        return res
    g = torch.where(okr[..., None, None], st["g"][ir].float(), 0.0).transpose(1, 2)
    vb = pr.transpose(2, 3) @ g
    ds = pr * (g @ v.transpose(2, 3) - (g * o).sum(-1, keepdim=True))
    if st["pos"] is not None:
        w = ds * st["slope"][:, None, None]
        f = torch.where(dist > 0, w.sum(1) / torch.where(dist > 0, dist, 1.0), 0.0)[..., None] * dx   # [B, Lr, Ls, 3]
        del w
        res["slope"] = -(ds * dist[:, None]).double().sum((0, 2, 3)).float()
        br, bs = torch.zeros((nr, 3), device=dev), torch.zeros((ns, 3), device=dev)
        br.index_copy_(0, rows, -f.sum(2)[okr])
        bs.index_copy_(0, cols, f.sum(1)[live[1]])
        res.update(dict(pos=br + bs) if st["pos_send"] is None else dict(pos=br, pos_send=bs))
        del f
    if cap:
        ds = ds * (1 - th * th)
    ds = ds * st["scale"]
    shared = lambda a: a.unflatten(1, (hk, grp)).sum(2)  # noqa: E731
    res["q"] = pack(ds @ k, rows, okr, nr).to(t)
    res["k"] = pack(shared(ds.transpose(2, 3) @ q), cols, live[1], ns).to(t)
    res["v"] = pack(shared(vb), cols, live[1], ns).to(t)
    return {n: res[n] for n in ("out", "lse", "q", "k", "v", "pos", "slope", "pos_send") if n in res}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op.startswith("embed"):
        n, ch = case["n"], case["channels"]
        rows = min(n, case["types"])
        if op == "embed":
            return {"bytes": 4 * n + rows * ch * e + n * (case["lmax"] + 1) ** 2 * ch * e, "flops": n * ch}
        return {"bytes": 4 * n + n * ch * e + case["types"] * ch * 4, "flops": n * ch}
    if op.startswith("norm"):
        n, el = case["n"], case["n"] * (case["hq"] + case["hk"]) * case["dim"]
        small = (12 * n + 12 * case["pairs"] if case["pairs"] else 0) + 8 * case["dim"]
        if op == "norm":
            return {"bytes": 2 * el * e + small, "flops": 8 * el}
        return {"bytes": 4 * el * e + 2 * small, "flops": 24 * el}
    lens = _lengths(case)
    nr = case["recv"] * case["structures"] if case["recv"] else sum(lens)
    ns = sum(lens)
    pairs = sum((case["recv"] or v) * v for v in lens)
    qo, kv = nr * case["hq"] * case["dim"] * e, ns * case["hk"] * case["dim"] * e
    small = 4 * nr * case["hq"] + (12 * (nr + (ns if case["recv"] else 0)) if case["bias"] else 0) + (ns if case["hide"] else 0)
    mac = pairs * case["hq"] * case["dim"]
    if op == "attn":
        return {"bytes": int(2 * qo + 2 * kv + small), "flops": int(4 * mac)}
    # forward, and the five products of the gradient; q, k, v and the output's gradient read, the output and three gradients written
    return {"bytes": int(4 * qo + 4 * kv + 2 * small), "flops": int(14 * mac)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        rows = torch.index_select(st["table"].double() * case["scale"], 0, st["species"])
        return torch.nn.functional.pad(rows, (0, ((case["lmax"] + 1) ** 2 - 1) * case["channels"]))
    if op == "embed_vjp":
        order = torch.argsort(st["species"], stable=True)
        counts = torch.bincount(st["species"], minlength=case["types"])
        ends = torch.cumsum(counts, 0)
        c = case["channels"]
        sums = torch.cat([torch.zeros((1, c), dtype=torch.float64, device="cuda"), torch.cumsum(st["g"][order, :c].double(), 0)])
        return (sums[ends] - sums[ends - counts]) * case["scale"]
    with torch.enable_grad():
        return _exact_norm(st, case) if op.startswith("norm") else _exact_attn(st, case)


def _leaf(a):
    return None if a is None else a.detach().double().clone().requires_grad_(True)


def _exact_norm(st, case):
    """y of the definition, gradients by automatic differentiation; the rotation as a complex product."""
    x, gq, gk, pos = _leaf(st["x"]), _leaf(st["gq"]), _leaf(st["gk"]), _leaf(st["pos"])
    hq, p = case["hq"], case["pairs"]
    parts = []
    for part, gamma in ((x[:, :hq], gq), (x[:, hq:], gk)):
        u = part / torch.sqrt(part.pow(2).sum(-1, keepdim=True) / case["dim"] + EPS) * gamma
        if p:
            angle = sum(pos[:, a, None] * st["freq"].double()[a] for a in range(3))
            turn = torch.polar(torch.ones_like(angle), angle)[:, None]
            zz = torch.complex(u[..., :p], u[..., p:2 * p]) * turn
            u = torch.cat([zz.real, zz.imag, u[..., 2 * p:]], -1)
        parts.append(u)
    y = torch.cat(parts, 1)
    if case["op"] == "norm":
        return y.detach()
    leaves = [x, gq, gk] + ([pos] if p else [])
    bars = torch.autograd.grad(y, leaves, st["g"].double())
    return dict(y=y.detach(), x=bars[0], gq=bars[1], gk=bars[2], **({"pos": bars[3]} if p else {}))


def _exact_attn(st, case):
    """Structure by structure and head by head; gradients by automatic differentiation."""
    hq, grp, cap, step = case["hq"], case["hq"] // case["hk"], case["cap"], case["op"] == "attn_step"
    q, k, v, pos, pos_send, slope = (_leaf(st[n]) for n in ("q", "k", "v", "pos", "pos_send", "slope"))
    rp, sp = st["recv_ptr"].tolist(), st["send_ptr"].tolist()
    out, lse = torch.zeros_like(q).detach(), torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    names = ["q", "k", "v"] + ([] if pos is None else ["pos", "slope"]) + ([] if pos_send is None else ["pos_send"])
    leaves = dict(q=q, k=k, v=v, pos=pos, slope=slope, pos_send=pos_send)
    bars = {n: torch.zeros_like(leaves[n]).detach() for n in names}
    # all heads of a structure at once where they fit
    for b in range(case["structures"]):
        r, s = slice(rp[b], rp[b + 1]), slice(sp[b], sp[b + 1])
        n = (r.stop - r.start) * (s.stop - s.start)
        wide = max(grp, (hq if n * hq < 2 ** 27 else 1) // grp * grp)
        for h in range(0, hq, wide):
            hs, ks = slice(h, h + wide), slice(h // grp, (h + wide) // grp)
            if not step:
                with torch.no_grad():
                    out[r, hs], lse[r, hs] = _exact_block(st, q, k, v, pos, pos_send, slope, r, s, hs, ks, grp, cap)
                continue
            o, z = _exact_block(st, q, k, v, pos, pos_send, slope, r, s, hs, ks, grp, cap)
            out[r, hs], lse[r, hs] = o.detach(), z.detach()
            for name, bar in zip(names, torch.autograd.grad(o, [leaves[m] for m in names], st["g"][r, hs].double(), allow_unused=True)):
                if bar is not None:
                    bars[name] += bar
    if not step:
        return dict(out=out, lse=lse)
    return dict(out=out, lse=lse, **bars)


def _exact_block(st, q, k, v, pos, pos_send, slope, r, s, hs, ks, grp, cap):
    keys = k[s, ks].repeat_interleave(grp, dim=1)
    vals = v[s, ks].repeat_interleave(grp, dim=1)
    score = torch.einsum("ihd,jhd->hij", q[r, hs], keys) * st["scale"]
    if cap:
        score = cap * torch.tanh(score / cap)
    if pos is not None:
        other = pos if pos_send is None else pos_send
        sq = sum((pos[r, a, None] - other[None, s, a]) ** 2 for a in range(3))
        apart = sq > 0
        dist = torch.sqrt(torch.where(apart, sq, 1.0)) * apart
        score = score - slope[hs, None, None] * dist
    keep = torch.ones(s.stop - s.start, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"][s] != 0
    if not bool(keep.any()):
        return (q[r, hs] * 0.0, torch.full((r.stop - r.start, hs.stop - hs.start), -math.inf, dtype=torch.float64, device="cuda"))
    score = score.masked_fill(~keep, -math.inf)
    z = torch.logsumexp(score, -1)
    return torch.einsum("hij,jhd->ihd", torch.exp(score - z[..., None]), vals), z.T
