"""Plain 64-bit forms of the node operators (torch, CPU) that the tests compare with, and the bounds the
comparison uses.

u(t) = eps(t) / 2 is the largest relative error of one rounding to type t."""
import math

import torch

U32 = 2.0 ** -24


def u(dtype):
    return torch.finfo(dtype).eps / 2


def embed(species, table, lmax, scale):
    n, (v, c) = species.shape[0], table.shape
    x = torch.zeros((n, (lmax + 1) ** 2 * c), dtype=torch.float64)
    ok = (species >= 0) & (species < v)
    x[ok, :c] = table.double()[species[ok].long()] * scale
    return x


def embed_vjp(species, g, v, lmax, scale):
    """table_bar, and for the bound the sum of magnitudes and the count per species."""
    c = g.shape[1] // (lmax + 1) ** 2
    bar, mag = torch.zeros((v, c), dtype=torch.float64), torch.zeros((v, c), dtype=torch.float64)
    ok = (species >= 0) & (species < v)
    s, r = species[ok].long(), g[ok, :c].double()
    bar.index_add_(0, s, r)
    mag.index_add_(0, s, r.abs())
    return bar * scale, mag * abs(scale), torch.bincount(s, minlength=v)


def norm(x, hq, gq, gk, pos, freq, eps):
    """y, with autograd through double leaves."""
    n, h, d = x.shape
    one = torch.ones(d, dtype=torch.float64)
    gam = torch.cat([(one if gq is None else gq).expand(hq, d), (one if gk is None else gk).expand(h - hq, d)])
    un = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gam
    if freq is None or freq.shape[1] == 0:
        return un
    r = freq.shape[1]
    th = (pos @ freq)[:, None]
    a, b = un[..., :r], un[..., r:2 * r]
    return torch.cat([a * torch.cos(th) - b * torch.sin(th), a * torch.sin(th) + b * torch.cos(th), un[..., 2 * r:]], -1)


def attention(q, k, v, rp, sp, pos=None, pos_send=None, slope=None, mask=None, scale=None, cap=0.0):
    """(out, lse, P per structure); rows outside every structure, and rows without senders, are 0 and -inf."""
    nr, h, d = q.shape
    grp = h // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, lse = torch.zeros_like(q), torch.full((nr, h), -math.inf, dtype=torch.float64)
    weights = []
    other = pos if pos_send is None else pos_send
    for b in range(len(rp) - 1):
        r = slice(int(rp[b]), int(rp[b + 1]))
        js = torch.arange(int(sp[b]), int(sp[b + 1]))
        if mask is not None:
            js = js[mask[js] != 0]
        weights.append(None)
        if r.stop == r.start or len(js) == 0:
            continue
        t = torch.einsum("ihd,jhd->hij", q[r], k[js].repeat_interleave(grp, 1)) * scale
        if cap:
            t = cap * torch.tanh(t / cap)
        if pos is not None:
            d2 = ((pos[r, None] - other[None, js]) ** 2).sum(-1)
            dist = torch.sqrt(torch.where(d2 > 0, d2, 1.0)) * (d2 > 0)
            t = t - slope[:, None, None] * dist
        z = torch.logsumexp(t, -1)
        p = torch.exp(t - z[..., None])
        out = out.index_add(0, torch.arange(r.start, r.stop), torch.einsum("hij,jhd->ihd", p, v[js].repeat_interleave(grp, 1)))
        lse[r] = z.detach().T
        weights[-1] = (r, js, p.detach())
    return out, lse, weights


def attention_bounds(q, k, v, g, weights, dtype, scale, slope=None, cap=0.0):
    """Sums of magnitudes behind every output, which each rounding of a 16-bit weight is relative to:
    out: sum P |v|; v_bar: sum P |g|; q_bar, k_bar: sum |ds| |k|, |q| (plus 2^-25 per FP16 term below its normal
    range); pos, slope: what an error of delta, (u sum P |dP|) u, moves.
    Last, for FP32: dP and delta are inner products of d terms whose difference may vanish (one sender: it is 0),
    so what they lose is relative to w = P (S_ij + sum_j P S_ij), S_ij = sum_d |g_d v_d|.  A product through the
    tensor core takes d/8 steps of three TF32 terms, each step truncating at 2^-23 of a sum of at most S, and the
    split leaves 3 2^-22 of it: under (d/2 + 16) 2^-23 S in all.  With that factor: scale sum w |k|, scale sum w |q|."""
    nr, h, d = q.shape
    kv = k.shape[1]
    grp = h // kv
    o, qb, kb, vb, q32, k32 = (torch.zeros_like(t) for t in (q, q, k, v, q, k))
    row = torch.zeros((nr, h), dtype=torch.float64)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    for w in weights:
        if w is None:
            continue
        r, js, p = w
        kk, vv = k[js].repeat_interleave(grp, 1), v[js].repeat_interleave(grp, 1)
        o[r] = torch.einsum("hij,jhd->ihd", p, vv.abs())
        dp = torch.einsum("ihd,jhd->hij", g[r], vv)
        ds = (p * (dp - (p * dp).sum(-1, keepdim=True))).abs() + tiny
        qb[r] = scale * torch.einsum("hij,jhd->ihd", ds, kk.abs())
        fold = lambda a: a.unflatten(1, (kv, grp)).sum(2)  # noqa: E731
        kb[js] = fold(scale * torch.einsum("hij,ihd->jhd", ds, q[r].abs()))
        vb[js] = fold(torch.einsum("hij,ihd->jhd", p + tiny, g[r].abs()))
        row[r] = (p * dp.abs()).sum(-1).T
        sij = torch.einsum("ihd,jhd->hij", g[r].abs(), vv.abs())
        w = p * (sij + (p * sij).sum(-1, keepdim=True)) * (d / 2 + 16) * 2.0 ** -23 * scale
        q32[r] = torch.einsum("hij,jhd->ihd", w, kk.abs())
        k32[js] = fold(torch.einsum("hij,ihd->jhd", w, q[r].abs()))
    return o, qb, kb, vb, row, q32, k32
