"""Measured cases of the operators that a hybrid stack needs beside the RSM mixer.

Three families: attention over a sliding window whose first tokens stay visible (prompts, and training
with its gradients), attention of new tokens over a paged key/value cache (chunks and single tokens,
with the write of their keys and values), and the norms around a block fused with its output gate and
residual scale. `run` computes each in plain torch operations, or, with `own` set, through librsm.
"""
import math
import random

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
NEG = float("-inf")


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # One layer's window attention on the pages' small training shape (4 x 128 tokens, 4 heads of 64):
        # the call is over in microseconds and its latency counts.
        dict(name="window small", op="window", B=4, T=128, H=4, Hkv=4, D=64, W=64, S=4, dtype="bf16", train=False),
        # A long prompt (32,768 tokens, 16 heads of 128) through a window of one training length.
        dict(name="window long prompt", op="window", B=1, T=32768, H=16, Hkv=4, D=128, W=2048, S=4, dtype="bf16", train=False),
        # A training step of a window layer at the mid-size shape (8 x 2048 tokens, 8 heads of 128).
        dict(name="window train", op="window", B=8, T=2048, H=8, Hkv=8, D=128, W=512, S=4, dtype="bf16", train=True),
        # Training with a length, a window and a group size that fill no tile, and heads of 80.
        dict(name="window train ragged", op="window", B=3, T=1537, H=6, Hkv=2, D=80, W=200, S=1, dtype="bf16", train=True),
        # Training in fp32, as the library's CUDA-core path is used to check a run.
        dict(name="window train fp32", op="window", B=2, T=777, H=4, Hkv=2, D=64, W=128, S=8, dtype="f32", train=True),
        # One user's generation step over a short cache.
        dict(name="paged one token", op="paged", B=1, new=1, ragged=False, H=16, Hkv=4, D=128, page=16, most=1000, W=0, S=0, dtype="bf16"),
        # A generation step of 256 sequences around 2048 tokens long.
        dict(name="paged step of 256", op="paged", B=256, new=1, ragged=False, H=16, Hkv=4, D=128, page=64, most=4096, W=0, S=0, dtype="bf16"),
        # Four prompts going in by chunks of 512 over caches of up to 32,768 tokens.
        dict(name="paged long chunk", op="paged", B=4, new=512, ragged=False, H=16, Hkv=4, D=128, page=64, most=32768, W=0, S=0, dtype="bf16"),
        # Prompts and single tokens mixed in one fp32 call, with a window and pages that end inside a tile.
        dict(name="paged mixed fp32", op="paged", B=9, new=130, ragged=True, H=8, Hkv=2, D=64, page=24, most=1500, W=256, S=4, dtype="f32"),
        # The norms of a generation step of 256 sequences.
        dict(name="norm step", op="norm", rows=256, d=2048, y="bf16", dtype="bf16", act="silu", train=False),
        # The norms behind the mixer's fp32 output on a long prompt.
        dict(name="norm prompt", op="norm", rows=32768, d=2048, y="f32", dtype="bf16", act="silu", train=False),
        # A training step of the norms at the mid-size shape.
        dict(name="norm train", op="norm", rows=16384, d=1024, y="bf16", dtype="bf16", act="sigmoid", train=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("window", "window", "paged", "paged", "norm"))
    if op == "window":
        train = rng.random() < 0.6
        dtype = rng.choice(("bf16", "bf16", "f32"))
        Hkv = rng.choice((1, 2, 3, 4, 8))
        H = Hkv * rng.choice((1, 2, 3, 4))
        D = rng.choice((64, 128, 128, 8 * rng.randint(2, 16)))
        room = (1 << 15) if dtype == "f32" else (1 << 17) if train else (1 << 19)
        # (training starts at two tokens and two keys: over one key the gradients of q and k are zero throughout)
        T = _log(rng, 2 if train else 1, 2048 if dtype == "f32" else 8192)
        B = rng.randint(1, max(1, min(8, room // (T * H))))
        W = _log(rng, 2 if train else 1, 700 if train else 2048)
        return dict(op="window", B=B, T=T, H=H, Hkv=Hkv, D=D, W=W, S=rng.choice((0, 1, 4, 4, 37)), dtype=dtype, train=train)
    if op == "paged":
        dtype = rng.choice(("bf16", "bf16", "f32"))
        Hkv = rng.choice((1, 2, 4, 8))
        H = Hkv * rng.choice((1, 2, 4, 5))
        D = rng.choice((64, 128, 128, 8 * rng.randint(2, 16)))
        new = rng.choice((1, 1, _log(rng, 2, 512)))
        most = _log(rng, new + 1, 2000 if dtype == "f32" else 16384)
        B = max(1, min(_log(rng, 1, 128), (1 << 20) // (most * Hkv), (1 << 28) // (most * new * H)))
        page = rng.choice((8, 16, 16, 24, 32, 64, 128, 256))
        W = rng.choice((0, 0, _log(rng, 16, 2048)))
        return dict(op="paged", B=B, new=new, ragged=new > 1 and rng.random() < 0.7, H=H, Hkv=Hkv, D=D, page=page,
                    most=most, W=W, S=rng.choice((0, 4)) if W else 0, dtype=dtype)
    d = 4 * _log(rng, 16, 1024)
    y, dtype = rng.choice((("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")))
    return dict(op="norm", rows=_log(rng, 1, min(32768, (1 << 24) // d)), d=d, y=y, dtype=dtype,
                act=rng.choice(("silu", "sigmoid")), train=rng.random() < 0.5)


def _type(name):
    return BF16 if name == "bf16" else F32


def _new_counts(c):
    """The new tokens of each sequence: all `new`, or mixed lengths (none, one, many) that the case's sizes fix."""
    if not c["ragged"]:
        return [c["new"]] * c["B"]
    r = random.Random(1000 * c["B"] + c["new"])
    n = [r.choice((0, 1, 1, r.randint(1, c["new"]), c["new"])) for _ in range(c["B"])]
    n[0] = c["new"]
    return n


def _lengths(c, seed):
    """Tokens in each sequence's cache, the new ones included: half of `most` to `most`, and never fewer than are new."""
    r = random.Random(seed)
    return [max(n, r.randint((c["most"] + 1) // 2, c["most"])) for n in _new_counts(c)]


# --------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, dtype=F32, times=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * times).to(dtype)

    if c["op"] == "window":
        t = _type(c["dtype"])
        # queries of standard deviation 2: scores spread over several units, as trained heads' do
        s = dict(q=rand(c["B"], c["T"], c["H"], c["D"], dtype=t, times=2.0), k=rand(c["B"], c["T"], c["Hkv"], c["D"], dtype=t),
                 v=rand(c["B"], c["T"], c["Hkv"], c["D"], dtype=t))
        if c["train"]:
            s["do"] = rand(c["B"], c["T"], c["H"], c["D"], dtype=t)
            for n in "qkv":
                s[n].requires_grad_(True)
        return dict(case=dict(c), **s)
    if c["op"] == "paged":
        t = _type(c["dtype"])
        n, lens = _new_counts(c), _lengths(c, seed)
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        width = -(-c["most"] // c["page"])
        pages = c["B"] * width
        dev = dict(device="cuda")
        return dict(case=dict(c), n=n, total=cu[-1], max_q=max(n),
                    q=rand(cu[-1], c["H"], c["D"], dtype=t, times=2.0), k=rand(cu[-1], c["Hkv"], c["D"], dtype=t),
                    v=rand(cu[-1], c["Hkv"], c["D"], dtype=t),
                    k_cache=rand(pages, c["page"], c["Hkv"], c["D"], dtype=t), v_cache=rand(pages, c["page"], c["Hkv"], c["D"], dtype=t),
                    table=torch.randperm(pages, generator=g, **dev).to(torch.int32).view(c["B"], width),
                    cu_q=torch.tensor(cu, dtype=torch.int32, **dev), kv_len=torch.tensor(lens, dtype=torch.int32, **dev))
    t, ty = _type(c["dtype"]), _type(c["y"])
    s = dict(y=rand(c["rows"], c["d"], dtype=ty, times=0.3), gate=rand(c["rows"], c["d"], dtype=t), res=rand(c["rows"], c["d"], dtype=t),
             w_post=1 + rand(c["d"], times=0.1), w_pre=1 + rand(c["d"], times=0.1), alpha=0.7, eps=1e-6)
    if c["train"]:
        s["dh"], s["dx"] = rand(c["rows"], c["d"], dtype=t), rand(c["rows"], c["d"], dtype=t)
        for n in ("y", "gate", "res", "w_post", "w_pre"):
            s[n].requires_grad_(True)
    return dict(case=dict(c), **s)


# ---------------------------------------------------------------------------------- plain forms
def _softmax(s, seen):
    """Softmax over the last axis of the places that are seen; a row that sees nothing gets zeros."""
    s = s.masked_fill(~seen, NEG)
    m = s.amax(-1, keepdim=True)
    p = (s - m.masked_fill(m == NEG, 0.0)).exp()
    z = p.sum(-1, keepdim=True)
    return p / z.masked_fill(z == 0, 1.0)


def _window_plain(q, k, v, W, S):
    """The window in blocks of C queries: a block sees its own C keys, the C before them, and the first S."""
    B, T, H, D = q.shape
    Hkv, G = k.shape[2], q.shape[2] // k.shape[2]
    S = min(S, T)
    C = max(1, min(W, T))
    if C < 64:  # short windows: blocks of at least 64 keep the products large
        C = min(64, T)
    n = -(-T // C)
    pad = n * C - T

    def blocks(x):  # [B, T, h, D] -> [B, h, n, C, D] in fp32
        x = torch.cat([x.float(), x.new_zeros(B, pad, x.shape[2], D, dtype=F32)], 1) if pad else x.float()
        return x.view(B, n, C, x.shape[2], D).permute(0, 3, 1, 2, 4)

    qb = blocks(q).reshape(B, Hkv, G, n, C, D)

    def keys(x):  # [B, Hkv, n, S + 2C, D]: the sinks, the block before, the block itself
        xb = blocks(x)
        before = torch.cat([torch.zeros_like(xb[:, :, :1]), xb[:, :, :-1]], 2)
        first = x[:, :S].float().permute(0, 2, 1, 3)[:, :, None].expand(B, Hkv, n, S, D)
        return torch.cat([first, before, xb], 3)

    kb, vb = keys(k), keys(v)
    at = torch.arange(n, device=q.device)[:, None] * C
    i = (at + torch.arange(C, device=q.device))[:, :, None]                    # the queries' places [n, C, 1]
    j = (at + torch.arange(-C, C, device=q.device))[:, None, :]                # the band's keys [n, 1, 2C]
    band = (j >= S) & (j <= i) & (i - j < W)
    first = torch.arange(S, device=q.device)[None, None, :] <= i               # the sinks' keys [n, C, S]
    seen = torch.cat([first, band], 2)
    p = _softmax(qb @ kb[:, :, None].transpose(-1, -2) * (1.0 / math.sqrt(D)), seen)
    o = p @ vb[:, :, None]
    return o.reshape(B, H, n * C, D)[:, :, :T].permute(0, 2, 1, 3).to(q.dtype)


def _paged_plain(s):
    c = s["case"]
    H, Hkv, D, page = c["H"], c["Hkv"], c["D"], c["page"]
    G, B, N, mq = H // Hkv, c["B"], s["total"], s["max_q"]
    cu, lens = s["cu_q"].long(), s["kv_len"].long()
    tok = torch.arange(N, device="cuda")
    b = (tok[:, None] >= cu[None, 1:]).sum(1)                     # the sequence of each new token
    i = tok - cu[b]                                               # its place among them
    pos = lens[b] - (cu[b + 1] - cu[b]) + i                       # its place in the sequence
    row = s["table"].long()[b, pos // page] * page + pos % page
    s["k_cache"].view(-1, Hkv, D)[row] = s["k"]
    s["v_cache"].view(-1, Hkv, D)[row] = s["v"]
    L = s["table"].shape[1] * page
    kk = s["k_cache"][s["table"].long()].float().view(B, L, Hkv, D).permute(0, 2, 3, 1)
    vv = s["v_cache"][s["table"].long()].float().view(B, L, Hkv, D).permute(0, 2, 1, 3)
    qq = torch.zeros(B, mq, H, D, device="cuda")
    qq[b, i] = s["q"].float()
    qq = qq.view(B, mq, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, mq * G, D)
    at = (lens - (cu[1:] - cu[:-1]))[:, None, None] + torch.arange(mq, device="cuda")[None, :, None]
    j = torch.arange(L, device="cuda")[None, None, :]
    seen = (j <= at) & (j < lens[:, None, None])
    if c["W"]:
        seen = seen & ((at - j < c["W"]) | (j < c["S"]))
    seen = seen[:, None, :, None, :].expand(B, 1, mq, G, L).reshape(B, 1, mq * G, L)
    o = _softmax(qq @ kk * (1.0 / math.sqrt(D)), seen) @ vv
    o = o.view(B, Hkv, mq, G, D).permute(0, 2, 1, 3, 4).reshape(B, mq, H, D)
    return dict(o=o[b, i].to(s["q"].dtype), k_cache=s["k_cache"], v_cache=s["v_cache"])


def _norm_plain(y, gate, res, w_post, w_pre, act, alpha, eps):
    yf, g, r = y.float(), gate.float(), res.float()
    n = yf * (yf.square().mean(-1, keepdim=True) + eps).rsqrt() * w_post
    sig = 1.0 / (1.0 + (-g).exp())
    h = r + alpha * n * (g * sig if act == "silu" else sig)
    x = h * (h.square().mean(-1, keepdim=True) + eps).rsqrt() * w_pre
    return h.to(res.dtype), x.to(res.dtype)


# ------------------------------------------------------------------------------------- one pass
def run(state):
    s = state
    c = s["case"]
    if own:
        import sparse_routed_slot_b200 as rsm
    if c["op"] == "window":
        q, k, v = s["q"], s["k"], s["v"]
        if not c["train"]:
            return rsm.window_forward(q, k, v, c["W"], c["S"])["o"] if own else _window_plain(q, k, v, c["W"], c["S"])
        o = rsm.WindowFunction.apply(q, k, v, c["W"], c["S"]) if own else _window_plain(q, k, v, c["W"], c["S"])
        dq, dk, dv = torch.autograd.grad(o, (q, k, v), s["do"])
        return dict(o=o, dq=dq, dk=dk, dv=dv)
    if c["op"] == "paged":
        if not own:
            return _paged_plain(s)
        rsm.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu_q"], s["kv_len"])
        r = rsm.paged_forward(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu_q"], s["kv_len"], s["max_q"],
                              window=c["W"], sinks=c["S"])
        return dict(o=r["o"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    a = (s["y"], s["gate"], s["res"], s["w_post"], s["w_pre"])
    if not c["train"]:
        if own:
            r = rsm.block_norm_forward(*a, act=c["act"], scale=s["alpha"], eps=s["eps"])
            return dict(h=r["h"], x=r["x"])
        h, x = _norm_plain(*a, c["act"], s["alpha"], s["eps"])
        return dict(h=h, x=x)
    h, x = (rsm.BlockNormFunction.apply if own else _norm_plain)(*a, c["act"], s["alpha"], s["eps"])
    dy, dg, dr, dpost, dpre = torch.autograd.grad((h, x), a, (s["dh"], s["dx"]))
    return dict(h=h, x=x, dy=dy, dgate=dg, dres=dr, dw_post=dpost, dw_pre=dpre)


# ------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "norm":
        e, ey = (2 if c["dtype"] == "bf16" else 4), (2 if c["y"] == "bf16" else 4)
        n = c["rows"] * c["d"]
        b = n * (ey + 4 * e) + 8 * c["d"]                     # y, gate, residual in; h, x out
        if c["train"]:
            b += n * (2 * e + ey + 2 * e) + 8 * c["d"]        # dh, dx in; dy, dgate, dres and the weights' gradients out
        return dict(bytes=b, flops=n * (14 + (30 if c["train"] else 0)))
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "window":
        B, T, H, Hkv, D, W, S = (c[n] for n in ("B", "T", "H", "Hkv", "D", "W", "S"))
        w = min(W, T)
        pairs = w * (w + 1) // 2 + (T - w) * w                # keys of the window
        if T > w and S:                                       # sinks behind it: min(S, t + 1 - W) at token t
            m = T - w
            s = min(S, m)
            pairs += s * (s + 1) // 2 + (m - s) * S
        b = e * B * T * D * (2 * H + 2 * Hkv)
        if c["train"]:
            b += e * B * T * D * (2 * H + 2 * Hkv)            # dO in; dq, dk, dv out
        return dict(bytes=b, flops=B * H * pairs * D * (14 if c["train"] else 4))
    n, lens = _new_counts(c), _lengths(c, 1)
    pairs, rows = 0, 0
    for x, L in zip(n, lens):
        if not x:
            continue
        lo = L - x                                            # the first new token's place
        if c["W"]:
            seen = [min(p + 1, c["W"]) + max(0, min(c["S"], p + 1 - c["W"])) for p in range(lo, L)]
            pairs += sum(seen)
            rows += min(L, L - max(0, lo - c["W"] + 1) + c["S"])
        else:
            pairs += x * lo + x * (x + 1) // 2
            rows += L
    N = sum(n)
    b = e * c["D"] * (2 * N * c["H"] + 2 * rows * c["Hkv"] + 2 * N * c["Hkv"])
    return dict(bytes=b, flops=4 * c["D"] * c["H"] * pairs)


# ----------------------------------------------------------------------------- the definitions
def _attend64(q, k, v, at, W, S, do=None):
    """Attention of the rows q [n, D], at places `at`, over keys and values [L, D], all of one head and in 64 bits:
    o, and with `do` the rows' gradients."""
    L, D = k.shape
    dist = at[:, None] - torch.arange(L, device=q.device)[None, :]
    seen = dist >= 0
    if W:
        seen &= (dist < W) | (torch.arange(L, device=q.device)[None, :] < S)
    logits = torch.einsum("nd,ld->nl", q, k) / math.sqrt(D)
    logits = torch.where(seen, logits, torch.full_like(logits, NEG))
    lse = torch.logsumexp(logits, 1, keepdim=True)
    p = torch.where(seen, torch.exp(logits - lse), torch.zeros_like(logits))
    o = torch.einsum("nl,ld->nd", p, v)
    if do is None:
        return o, None, None, None
    dp = torch.einsum("nd,ld->nl", do, v)
    ds = p * (dp - (do * o).sum(1, keepdim=True)) / math.sqrt(D)
    return o, ds @ k, ds.T @ q, p.T @ do


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    with torch.no_grad():
        if c["op"] == "window":
            q, k, v = (s[n].detach().double() for n in "qkv")
            do = s["do"].double() if c["train"] else None
            G, W, S, T = c["H"] // c["Hkv"], c["W"], c["S"], c["T"]
            o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
            step = max(256, min(T, 2048))
            for b in range(c["B"]):
                for h in range(c["H"]):
                    for t0 in range(0, T, step):
                        t1 = min(T, t0 + step)
                        lo = max(0, t0 - W + 1)
                        S0 = min(S, lo)  # sinks in front of the band's first key
                        kv = h // G
                        kk, vv = (torch.cat([x[b, :S0, kv], x[b, lo:t1, kv]]) for x in (k, v))
                        # places counted from the band's first key: the S0 sinks take the places below S0
                        at = torch.arange(t0, t1, device="cuda") - lo + S0
                        a = _attend64(q[b, t0:t1, h], kk, vv, at, W, S if S > lo else S0, do[b, t0:t1, h] if c["train"] else None)
                        o[b, t0:t1, h] = a[0]
                        if c["train"]:
                            dq[b, t0:t1, h] = a[1]
                            for d, x in ((dk, a[2]), (dv, a[3])):
                                d[b, :S0, kv] += x[:S0]
                                d[b, lo:t1, kv] += x[S0:]
            return dict(o=o, dq=dq, dk=dk, dv=dv) if c["train"] else o
        if c["op"] == "paged":
            n, lens, page = s["n"], _lengths(c, seed), c["page"]
            G = c["H"] // c["Hkv"]
            o = torch.zeros(s["total"], c["H"], c["D"], dtype=torch.float64, device="cuda")
            kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
            at = 0
            for b, (x, L) in enumerate(zip(n, lens)):
                if not x:
                    continue
                places = torch.arange(L, device="cuda")
                pg, off = s["table"][b].long()[places // page], places % page
                kc[pg[L - x:], off[L - x:]] = s["k"][at:at + x]
                vc[pg[L - x:], off[L - x:]] = s["v"][at:at + x]
                kk, vv = kc[pg, off].double(), vc[pg, off].double()
                for h in range(c["Hkv"]):
                    rows = s["q"][at:at + x, h * G:(h + 1) * G].double().reshape(x * G, c["D"])
                    where = torch.arange(L - x, L, device="cuda").repeat_interleave(G)
                    a = _attend64(rows, kk[:, h], vv[:, h], where, c["W"], c["S"])
                    o[at:at + x, h * G:(h + 1) * G] = a[0].view(x, G, c["D"])
                at += x
            return dict(o=o, k_cache=kc.float(), v_cache=vc.float())
        y, g, r, w1, w2 = (s[n].detach().double() for n in ("y", "gate", "res", "w_post", "w_pre"))
        al, d = s["alpha"], c["d"]
        r1 = 1 / torch.sqrt((y * y).sum(1, keepdim=True) / d + s["eps"])
        sig = torch.sigmoid(g)
        act = g * sig if c["act"] == "silu" else sig
        slope = sig * (1 + g * (1 - sig)) if c["act"] == "silu" else sig * (1 - sig)
        n = y * r1 * w1
        h = r + al * n * act
        r2 = 1 / torch.sqrt((h * h).sum(1, keepdim=True) / d + s["eps"])
        x = h * r2 * w2
        if not c["train"]:
            return dict(h=h, x=x)
        dh, dx = s["dh"].double(), s["dx"].double()
        e = dx * w2
        dH = dh + r2 * e - h * r2 ** 3 * (e * h).sum(1, keepdim=True) / d
        du = al * dH
        f = du * act * w1
        dy = r1 * f - y * r1 ** 3 * (f * y).sum(1, keepdim=True) / d
        return dict(h=h, x=x, dy=dy, dgate=du * n * slope, dres=dH, dw_post=(du * act * y * r1).sum(0), dw_pre=(dx * h * r2).sum(0))
