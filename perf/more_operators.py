"""Cases and plain forms of the operators of a block's dense half: the gated
feed-forward of a shared expert or a dense layer (forward, and its backward),
and dropout on the way back into the residual stream (inside the fused norms,
gate and residual, forward and backward).

With ``own`` false ``run`` evaluates the formulas with elementary torch
operations in 32 bits, rounded once at the end; with ``own`` true it calls the
package.  ``exact`` evaluates them in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6     # under the root of the mean square


def _moe():
    import dropless_moe_expert_gb300
    return dropless_moe_expert_gb300


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # decode of one sequence through a shared expert of the width of one routed expert: latency and weights
        dict(name="ffn one token", op="ffn", T=1, d=7168, f=2048, act="silu"),
        # decode of an odd batch through a small one
        dict(name="ffn small batch", op="ffn", T=37, d=2048, f=768, act="gelu_tanh"),
        # a chunk of a prompt beside decoding ones, sizes that fill no tile
        dict(name="ffn ragged", op="ffn", T=1003, d=2056, f=1368, act="gelu"),
        # prefill or a training batch through a wide dense layer
        dict(name="ffn wide batch", op="ffn", T=4096, d=4096, f=14336, act="silu"),
        # training, a short last batch with sizes that fill no tile
        dict(name="ffn backward ragged", op="ffn_backward", T=777, d=1032, f=2056, act="gelu"),
        # training of a shared expert
        dict(name="ffn backward shared", op="ffn_backward", T=4096, d=7168, f=2048, act="silu"),
        # training of a wide dense layer
        dict(name="ffn backward wide", op="ffn_backward", T=4096, d=4096, f=14336, act="silu"),
        # a short batch, the residual sum alone: latency
        dict(name="dropout sum short", op="norm", T=129, d=1024, residual="bf16", post=False, pre=False,
             gate="none", scale=1.0, p=0.1),
        # a training batch: post-norm, gate, dropout, residual and the next pre-norm, the stream in 16 bits
        dict(name="dropout norms batch", op="norm", T=8192, d=4096, residual="bf16", post=True, pre=True,
             gate="channel", scale=1.0, p=0.1),
        # a wide model, a ragged batch, the stream in 32 bits
        dict(name="dropout norms wide ragged", op="norm", T=4093, d=7168, residual="fp32", post=False, pre=True,
             gate="token", scale=1.0, p=0.25),
        # the training batch's backward
        dict(name="dropout backward batch", op="norm_backward", T=8192, d=4096, residual="bf16", post=True, pre=True,
             gate="channel", scale=1.0, p=0.1),
        # the wide one's
        dict(name="dropout backward wide", op="norm_backward", T=4093, d=7168, residual="fp32", post=False, pre=True,
             gate="token", scale=1.0, p=0.25),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_backward", "norm", "norm_backward"])
    if op in ("ffn", "ffn_backward"):
        d, f = 8 * _log_int(rng, 8, 1024), 8 * _log_int(rng, 8, 2048)
        most = min(8192, 4096 * 4096 * 14336 // (d * f))
        return dict(op=op, T=_log_int(rng, 1, most), d=d, f=f, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]))
    d = 64 * _log_int(rng, 1, 128)
    return dict(op=op, T=_log_int(rng, 1, min(16384, 33554432 // d)), d=d, residual=rng.choice(["bf16", "fp32"]),
                post=rng.random() < 0.5, pre=rng.random() < 0.7, gate=rng.choice(["none", "channel", "token"]),
                scale=rng.choice([1.0, 0.5, 0.70710678]), p=rng.choice([0.05, 0.1, 0.2, 0.5]))


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case=case)
    T, d = case["T"], case["d"]
    if case["op"] in ("ffn", "ffn_backward"):
        f = case["f"]
        # rows after a norm, weights as they are initialised
        s["x"] = normal(T, d).to(BF16)
        s["W1"] = (normal(2 * f, d) / math.sqrt(d)).to(BF16)    # gate rows, then up rows
        s["W2"] = (normal(d, f) / math.sqrt(f)).to(BF16)
        if case["op"] == "ffn_backward":
            s["a"] = (s["x"].float() @ s["W1"].float().T).to(BF16)   # the pre-activations that the forward kept
            s["dy"] = normal(T, d).to(BF16)
        if own:
            moe = _moe()
            if case["op"] == "ffn":
                s["ffn"] = moe.GatedFFN(s["W1"], s["W2"], case["act"], T_max=T)
                s["out"] = torch.empty(T, d, dtype=BF16, device="cuda")
            else:
                s["out"] = moe.GatedFFNGrads.empty(T, d, f)
        return s
    res = F32 if case["residual"] == "fp32" else BF16
    s["r"] = (3.0 * normal(T, d)).to(res)
    s["y"] = (0.2 * normal(T, d)).to(BF16)
    s["gp"] = 1.0 + 0.2 * normal(d) if case["post"] else None
    s["gq"] = 1.0 + 0.2 * normal(d) if case["pre"] else None
    s["gate"] = {"none": lambda: None, "channel": lambda: 0.3 + 0.1 * normal(d),
                 "token": lambda: torch.sigmoid(normal(T, 1))}[case["gate"]]()
    # the generator's state: a run's seed, and the number of this call in it
    s["rng"] = torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), generator=g, device="cuda")
    if case["op"] == "norm_backward":
        # what the forward left: its output stream and the two rows of factors
        r2, _, rp, rq = _norm(case, s, F32)
        s["r2"], s["rp"], s["rq"] = r2.to(res), rp, rq
        s["dr2"], s["dn"] = normal(T, d).to(res), normal(T, d).to(BF16) if case["pre"] else None
        del s["r"]
    if own:
        moe = _moe()
        if case["op"] == "norm":
            s["out"] = moe.NormResidual.empty(T, d, res, post=case["post"], pre=case["pre"], rng=True)
        else:
            s["out"] = moe.NormResidualGrads.empty(T, d, res, post=case["post"], pre=case["pre"], gate=case["gate"])
    return s


# ------------------------------------------------------------------ plain forms
def _act(name, g):
    """The activation and its derivative."""
    if name == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g / math.sqrt(2.0)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    # silu, or gelu with its tanh: g times the logistic function of z(g), as (1 + tanh(z / 2)) / 2 is that
    c = 2.0 * math.sqrt(2.0 / math.pi)
    z = g if name == "silu" else c * (g + 0.044715 * g * g * g)
    dz = 1.0 if name == "silu" else c * (1.0 + 3 * 0.044715 * g * g)
    s = 1.0 / (1.0 + torch.exp(-z))
    return g * s, s + g * s * (1.0 - s) * dz


def _ffn(case, st):
    f = case["f"]
    a = st["x"].float() @ st["W1"].float().T
    return (_act(case["act"], a[:, :f])[0] * a[:, f:]) @ st["W2"].float().T


def _ffn_backward(case, st):
    f, dy, x = case["f"], st["dy"].float(), st["x"].float()
    g, u = st["a"][:, :f].float(), st["a"][:, f:].float()
    act, slope = _act(case["act"], g)
    dh = dy @ st["W2"].float()
    da = torch.cat([dh * u * slope, dh * act], dim=1)
    return dict(dx=da @ st["W1"].float(), dW1=da.T @ x, dW2=dy.T @ (act * u))


_LOW = 0xFFFFFFFF


def _philox(rng, blocks):
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, SC 2011): [blocks, 4] words in int64, for the key rng[0] and the
    counters (block, rng[1]).  Products of 32-bit words wrap in int64; both their halves are what they are unsigned."""
    i = torch.arange(blocks, device=rng.device)
    key = [rng[0] & _LOW, rng[0] >> 32 & _LOW]
    c = [i & _LOW, i >> 32, (rng[1] & _LOW).expand(blocks), (rng[1] >> 32 & _LOW).expand(blocks)]
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32 & _LOW) ^ c[1] ^ key[0], q & _LOW, (p >> 32 & _LOW) ^ c[3] ^ key[1], p & _LOW]
        key = [key[0] + 0x9E3779B9 & _LOW, key[1] + 0xBB67AE85 & _LOW]
    return torch.stack(c, dim=1)


def _mask(case, rng, kind):
    """The factor of each element: 0, or one over the share that is kept.  An element has one 16-bit draw: the
    (i % 8)-th of block i / 8, low halves first; p counts in steps of 2^-16."""
    T, d = case["T"], case["d"]
    w = _philox(rng, T * d // 8)
    draws = torch.stack([w & 0xFFFF, w >> 16], dim=2).view(T, d)
    drop = round(case["p"] * 65536)
    return (draws >= drop).to(kind) * (65536 / (65536 - drop))


def _norm(case, st, kind):
    """r' and n before any rounding, and the two rows of factors."""
    u, rp, rq, n = st["y"].to(kind), None, None, None
    if case["post"]:
        rp = 1.0 / torch.sqrt((u * u).mean(dim=1) + EPS)
        u = u * rp[:, None] * st["gp"].to(kind)
    if st["gate"] is not None:
        u = u * st["gate"].to(kind)
    r2 = case["scale"] * st["r"].to(kind) + u * _mask(case, st["rng"], kind)
    if case["pre"]:
        rq = 1.0 / torch.sqrt((r2 * r2).mean(dim=1) + EPS)
        n = r2 * rq[:, None] * st["gq"].to(kind)
    return r2, n, rp, rq


def _norm_backward(case, st, kind):
    r2, D, y = st["r2"].to(kind), st["dr2"].to(kind), st["y"].to(kind)
    out = {}
    if case["pre"]:
        rq, dn = st["rq"].to(kind)[:, None], st["dn"].to(kind)
        h = dn * st["gq"].to(kind)
        out["dgamma_pre"] = (dn * r2 * rq).sum(dim=0)
        D = D + rq * (h - r2 * rq * rq * (h * r2).mean(dim=1, keepdim=True))
    out["dr"] = case["scale"] * D
    k = D * _mask(case, st["rng"], kind)    # the gradient of what the dropout takes
    v = u = y
    if case["post"]:
        rp = st["rp"].to(kind)[:, None]
        v = y * rp
        u = v * st["gp"].to(kind)
    if st["gate"] is not None:
        out["dgate"] = (u * k).sum(dim=0) if case["gate"] == "channel" else (u * k).sum(dim=1, keepdim=True)
        k = k * st["gate"].to(kind)
    if case["post"]:
        out["dgamma_post"] = (k * v).sum(dim=0)
        k = k * st["gp"].to(kind)
        k = rp * (k - y * rp * rp * (k * y).mean(dim=1, keepdim=True))
    out["dy"] = k
    return out


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        return _run_own(case, op, st)
    if op == "ffn":
        return _ffn(case, st).to(BF16)
    if op == "ffn_backward":
        return {k: v.to(BF16) for k, v in _ffn_backward(case, st).items()}
    if op == "norm":
        r2, n, rp, rq = _norm(case, st, F32)
        return dict(r=r2.to(st["r"].dtype), n=None if n is None else n.to(BF16), rstd_post=rp, rstd_pre=rq)
    out = _norm_backward(case, st, F32)
    return dict(out, dr=out["dr"].to(st["r2"].dtype), dy=out["dy"].to(BF16))


def _run_own(case, op, st):
    if op == "ffn":
        return st["ffn"](st["x"], out=st["out"])
    moe = _moe()
    if op == "ffn_backward":
        g = moe.gated_ffn_backward(st["x"], st["a"], st["dy"], st["W1"], st["W2"], case["act"], out=st["out"])
        return dict(dx=g.dx, dW1=g.dW1, dW2=g.dW2)
    if op == "norm":
        o = moe.norm_residual(st["r"], st["y"], gamma_post=st["gp"], gate=st["gate"], gamma_pre=st["gq"],
                              res_scale=case["scale"], eps=EPS, dropout=case["p"], rng=st["rng"], out=st["out"])
        return dict(r=o.r, n=o.n, rstd_post=o.rstd_post, rstd_pre=o.rstd_pre)
    g = moe.norm_residual_backward(st["r2"], st["dr2"], st["dn"], st["y"], gamma_post=st["gp"], gate=st["gate"],
                                   gamma_pre=st["gq"], res_scale=case["scale"], rstd_post=st["rp"],
                                   rstd_pre=st["rq"], dropout=case["p"], rng=st["rng"], out=st["out"])
    return {k: v for k, v in dict(dr=g.dr, dy=g.dy, dgamma_pre=g.dgamma_pre, dgamma_post=g.dgamma_post,
                                  dgate=g.dgate).items() if v is not None}


# ------------------------------------------------------------------ 64 bits
def _exact_act(name, g):
    if name == "relu":
        return torch.clamp(g, min=0.0)
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "gelu":
        return g * torch.special.ndtr(g)
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))


def _exact_kept(case, rng):
    """The elements that stay, from the generator's definition on unsigned words, on the host."""
    seed, call = (int(v) & (1 << 64) - 1 for v in rng.tolist())
    n = case["T"] * case["d"]
    word = np.uint64(_LOW)
    ctr = np.arange((n + 7) // 8, dtype=np.uint64)
    a, b = ctr & word, ctr >> np.uint64(32)
    c, e = (np.full_like(ctr, v) for v in (call & _LOW, call >> 32))
    for k in range(10):
        k0, k1 = ((v + k * step) & _LOW for v, step in ((seed & _LOW, 0x9E3779B9), (seed >> 32, 0xBB67AE85)))
        lo, hi = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)
        a, b, c, e = (hi >> np.uint64(32)) ^ b ^ np.uint64(k0), hi & word, \
            (lo >> np.uint64(32)) ^ e ^ np.uint64(k1), lo & word
    words = np.stack([a, b, c, e], axis=1).astype("<u4")
    draws = words.view("<u2").reshape(-1)[:n].reshape(case["T"], case["d"])
    return torch.from_numpy(draws.astype(np.int32) >= round(case["p"] * 65536)).cuda()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "ffn":
        a = st["x"].double() @ st["W1"].double().T
        g, u = a.split(case["f"], dim=1)
        return (_exact_act(case["act"], g) * u) @ st["W2"].double().T
    if op == "ffn_backward":
        # by the definition of the forward, the pre-activations and the second weights being its inputs
        a, dy = st["a"].double().requires_grad_(True), st["dy"].double()
        g, u = a.split(case["f"], dim=1)
        h = _exact_act(case["act"], g) * u
        da, = torch.autograd.grad(h, a, dy @ st["W2"].double())
        return dict(dx=torch.einsum("tk,kd->td", da, st["W1"].double()),
                    dW1=torch.einsum("tk,td->kd", da, st["x"].double()), dW2=torch.einsum("td,tf->df", dy, h.detach()))
    kept = _exact_kept(case, st["rng"])
    share = 1.0 - round(case["p"] * 65536) / 65536
    y = st["y"].double()
    gp, gq, gate = (None if st[k] is None else st[k].double() for k in ("gp", "gq", "gate"))
    if op == "norm":
        z, rp, rq, n = y, None, None, None
        if gp is not None:
            rp = (y.square().mean(1) + EPS).rsqrt()
            z = y * rp.unsqueeze(1) * gp
        if gate is not None:
            z = z * gate
        r = case["scale"] * st["r"].double() + torch.where(kept, z / share, 0.0)
        if gq is not None:
            rq = (r.square().mean(1) + EPS).rsqrt()
            n = r * rq.unsqueeze(1) * gq
        return dict(r=r, n=n, rstd_post=rp, rstd_pre=rq)
    # the rows' factors are inputs; with x = r' and m = mean, the Jacobian of x -> x * f(x) * weight
    x, D, out, d = st["r2"].double(), st["dr2"].double(), {}, case["d"]
    if gq is not None:
        f, dn = st["rq"].double().unsqueeze(1), st["dn"].double()
        out["dgamma_pre"] = torch.einsum("td,td->d", dn, x * f)
        D = D + f * dn * gq - x * f ** 3 * (torch.einsum("td,td,d->t", dn, x, gq) / d).unsqueeze(1)
    out["dr"] = D * case["scale"]
    D = torch.where(kept, D / share, 0.0)
    f = st["rp"].double().unsqueeze(1) if gp is not None else None
    z = y if gp is None else y * f
    weight = 1.0 if gp is None else gp
    if gate is not None:
        out["dgate"] = torch.einsum("td,td->d", z * weight, D) if case["gate"] == "channel" else \
            torch.einsum("td,td->t", z * weight, D).unsqueeze(1)
        D = D * gate
    if gp is not None:
        out["dgamma_post"] = torch.einsum("td,td->d", D, z)
        D = f * D * gp - y * f ** 3 * (torch.einsum("td,td,d->t", D, y, gp) / d).unsqueeze(1)
    out["dy"] = D
    return out


# ------------------------------------------------------------------ work
def work(case):
    T, d = case["T"], case["d"]
    if case["op"] == "ffn":
        f = case["f"]
        return dict(bytes=2 * (3 * d * f + 2 * T * d), flops=6 * T * d * f)
    if case["op"] == "ffn_backward":
        f = case["f"]
        return dict(bytes=2 * (6 * d * f + 3 * T * d + 2 * T * f), flops=12 * T * d * f)
    R = 4 if case["residual"] == "fp32" else 2
    rows = case["post"] + case["pre"] + (case["gate"] == "token")
    cols = case["post"] + case["pre"] + (case["gate"] == "channel")
    # a block of eight elements takes about 60 operations of the generator
    if case["op"] == "norm":
        return dict(bytes=T * d * (2 * R + 2 + 2 * case["pre"]) + 4 * T * rows + 4 * d * cols, flops=18 * T * d)
    through = 2 * R + (R + 2 if case["pre"] else 0) + 4
    return dict(bytes=T * d * through + 4 * T * (rows + (case["gate"] == "token")) + 8 * d * cols, flops=32 * T * d)
