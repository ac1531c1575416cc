"""Plain 64-bit forms of the operators beside the mixer, from their definitions (torch, float64, no
code shared with the library): attention over a window or a paged cache, its gradients, the block
norms and theirs. Each also returns how far fp32 arithmetic, and roundings of relative size `u` in the
places the library documents, may move each value: first-order bounds, summed over every term."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24


def attend(q, k, v, at, window, sinks, scale, do=None, u=0.0, uo=0.0):
    """Rows q [n,H,D] at places `at` [n] over k, v [L,Hkv,D]; window 0 = no limit. u: relative rounding of
    the softmax weights and of ds before their products; uo: of the outputs.

    Returns a dict of (value, bound) pairs: o, lse, and with `do` dq, dk, dv."""
    q, k, v = q.double(), k.double(), v.double()
    n, H, D = q.shape
    held = k.shape[0]
    if held == 0:  # a key that nothing sees stands in for none
        k, v = k.new_zeros(1, *k.shape[1:]), v.new_zeros(1, *v.shape[1:])
    L, Hkv = k.shape[0], k.shape[1]
    G = H // Hkv
    j = torch.arange(L, device=q.device)
    dist = at[:, None] - j[None, :]
    seen = (dist >= 0) & (j[None, :] < held)
    if window:
        seen = seen & ((dist < window) | (j[None, :] < sinks))
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.einsum("nhd,lhd->hnl", q, kk) * scale
    es = torch.einsum("nhd,lhd->hnl", q.abs(), kk.abs()) * scale * (D + 4) * U32
    s = s.masked_fill(~seen, float("-inf"))
    lse = torch.logsumexp(s, 2)                                    # [H, n]; -inf where nothing is seen
    empty = lse == float("-inf")
    ref = lse.masked_fill(empty, 0.0)
    p = torch.exp(s - ref[..., None]).masked_fill(~seen, 0.0)
    # a weight moves by its score's error, the normaliser's (a mean of such errors), the rounding of the
    # two exponents in fp32, and a few operations; ex2 and lg2 are good to about 2^-21
    mag = s.masked_fill(~seen, 0.0).abs().amax(2) + ref.abs()
    worst = es.masked_fill(~seen, 0.0).amax(2)
    rp = es + worst[..., None] + (4 * mag[..., None] + L + 64) * U32 + 2.0 ** -20
    o = torch.einsum("hnl,lhd->nhd", p, vv)
    # rounded weights move o by sum eta p v over the plain sum of weights, by sum eta p (v - o) over their own
    eo = torch.einsum("hnl,lhd->nhd", p * (rp + u + (L + 8) * U32), vv.abs()) + (u + uo + 2 * U32) * o.abs()
    out = {"o": (o, eo), "lse": (lse.T, (worst + (8 * mag + 64) * U32 + 2.0 ** -20).T)}
    if do is None:
        return out
    do = do.double()
    dp = torch.einsum("nhd,lhd->hnl", do, vv)
    delta = (do * o).sum(2).T[..., None]
    ds = p * (dp - delta)
    edp = torch.einsum("nhd,lhd->hnl", do.abs(), vv.abs()) * (D + 4) * U32
    edelta = ((do.abs() * (eo + (D + 4) * U32 * o.abs())).sum(2).T)[..., None]
    eds = p * (edp + edelta) + ds.abs() * (rp + u + 8 * U32)
    terms = (n * G + L + 8) * U32

    def shared(x):  # sum over the query heads of a group
        return x.view(L, Hkv, G, D).sum(2)

    dq = torch.einsum("hnl,lhd->nhd", ds, kk) * scale
    edq = torch.einsum("hnl,lhd->nhd", eds + terms * ds.abs(), kk.abs()) * scale + (uo + 2 * U32) * dq.abs()
    dk = shared(torch.einsum("hnl,nhd->lhd", ds, q)) * scale
    edk = shared(torch.einsum("hnl,nhd->lhd", eds + terms * ds.abs(), q.abs())) * scale + (uo + 2 * U32) * dk.abs()
    dv = shared(torch.einsum("hnl,nhd->lhd", p, do))
    edv = shared(torch.einsum("hnl,nhd->lhd", p * (rp + u + terms), do.abs())) + (uo + 2 * U32) * dv.abs()
    out.update(dq=(dq, edq), dk=(dk, edk), dv=(dv, edv))
    return out


def window(q, k, v, window, sinks, scale, do=None, u=0.0, uo=0.0):
    """Window attention of q [B,T,H,D], k, v [B,T,Hkv,D]; outputs stacked over the batch."""
    at = torch.arange(q.shape[1], device=q.device)
    each = [attend(q[b], k[b], v[b], at, window, sinks, scale, None if do is None else do[b], u, uo)
            for b in range(q.shape[0])]
    return {n: tuple(torch.stack([e[n][i] for e in each]) for i in (0, 1)) for n in each[0]} if each else {}


def block_norm(y, gate, res, w_post, w_pre, act, scale, eps, dh=None, dx=None):
    """h, x and, with dh or dx, the gradients dy, dgate, dresidual, dw_post, dw_pre."""
    y, r, w1 = y.double(), res.double(), w_post.double()
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    r1 = (mean(y * y) + eps) ** -0.5
    n = y * r1 * w1
    if gate is None:
        a, slope = torch.ones_like(r), torch.zeros_like(r)
    else:
        g = gate.double()
        sg = torch.sigmoid(g)
        a, slope = (g * sg, sg + g * sg * (1 - sg)) if act == "silu" else (sg, sg * (1 - sg))
    h = r + scale * n * a
    r2 = (mean(h * h) + eps) ** -0.5
    out = {"h": h}
    if w_pre is not None:
        out["x"] = h * r2 * w_pre.double()
    if dh is None and dx is None:
        return out
    dH = torch.zeros_like(h) if dh is None else dh.double()
    if dx is not None:
        e = dx.double() * w_pre.double()
        dH = dH + r2 * e - h * r2 ** 3 * mean(e * h)
        out["dw_pre"] = (dx.double() * h * r2).flatten(0, -2).sum(0)
    du = scale * dH
    f = du * a * w1
    out["dresidual"] = dH
    out["dy"] = r1 * f - y * r1 ** 3 * mean(f * y)
    out["dw_post"] = (du * a * y * r1).flatten(0, -2).sum(0)
    if gate is not None:
        out["dgate"] = du * n * slope
    return out
