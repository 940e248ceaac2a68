"""Cases and plain forms of the operators around the MoE layer: scored routing
(forward, and the gradient of the logits), the fused norms, gate and residual
between two layers (forward and backward), and the global gradient norm with
clipping.

With ``own`` false ``run`` evaluates the formulas with elementary torch
operations in 32 bits, rounded once at the end; with ``own`` true it calls the
package.  ``exact`` evaluates them in 64 bits.
"""
import math

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
EPS_NORM = 1e-6     # under the root of the mean square
EPS_SUM = 1e-20     # beside the sum of the chosen scores
EPS_CLIP = 1e-6     # beside the gradient norm


def _moe():
    import dropless_moe_expert_gb300
    return dropless_moe_expert_gb300


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # decode of one sequence through a layer of 256 routed experts in 8 groups: latency alone
        dict(name="route one token", op="route", T=1, E=256, K=8, score="sigmoid", groups=8, keep=4, group_top=2,
             bias=True, renorm=True, scale=2.5),
        # the same router over a prefill or a micro-batch
        dict(name="route sigmoid groups", op="route", T=4096, E=256, K=8, score="sigmoid", groups=8, keep=4,
             group_top=2, bias=True, renorm=True, scale=2.5),
        # a long batch, few experts, softmax scores as they are
        dict(name="route softmax long", op="route", T=32768, E=64, K=6, score="softmax", groups=1, keep=1, group_top=1,
             bias=True, renorm=False, scale=1.0),
        # training: the logits' gradient, K entries of each row are not zero
        dict(name="route backward sigmoid", op="route_backward", T=4096, E=256, K=8, score="sigmoid", groups=8, keep=4,
             group_top=2, bias=True, renorm=True, scale=2.5),
        # training: a dense gradient, a batch that fills no tile
        dict(name="route backward softmax", op="route_backward", T=16381, E=128, K=8, score="softmax", groups=1,
             keep=1, group_top=1, bias=False, renorm=False, scale=1.0),
        # decode: post-norm, gate, residual and the next pre-norm of one token, the residual in 32 bits
        dict(name="norm one token", op="norm", T=1, d=7168, residual="fp32", post=True, pre=True, y=True,
             gate="channel", scale=1.0),
        # a training batch with the residual in 16 bits
        dict(name="norm batch", op="norm", T=8192, d=4096, residual="bf16", post=True, pre=True, y=True,
             gate="channel", scale=0.5),
        # its backward
        dict(name="norm backward batch", op="norm_backward", T=8192, d=4096, residual="bf16", post=True, pre=True,
             y=True, gate="channel", scale=0.5),
        # a wide model, a ragged batch, the residual in 32 bits, a gate for each token
        dict(name="norm backward wide ragged", op="norm_backward", T=4093, d=7168, residual="fp32", post=True,
             pre=True, y=True, gate="token", scale=1.0),
        # the many small gradients of a model (norms, gates, biases, routers): odd sizes, packed without padding
        dict(name="clip many small", op="clip", tensors=301, smallest=1, largest=60000, dtype="mixed",
             max_norm=1.0),
        # the gradients of a layer of 128 experts, d = 2048, f = 768, in 32 bits, with its router and norms
        dict(name="clip expert layer", op="clip", tensors=6, E=128, d=2048, f=768, dtype="fp32", max_norm=1.0),
        # the gradients of a stack of dense weights, in 16 bits
        dict(name="clip dense weights", op="clip", tensors=40, smallest=2048, largest=16777216, dtype="bf16",
             max_norm=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "norm", "norm_backward", "clip"])
    if op in ("route", "route_backward"):
        groups, size = rng.choice([(1, 8), (1, 37), (1, 60), (1, 64), (1, 100), (1, 128), (1, 256), (4, 16), (8, 32),
                                   (8, 20), (5, 12), (16, 16), (3, 21)])
        E = groups * size
        keep = rng.randint(1, groups)
        K = rng.randint(1, min(16, keep * size))
        return dict(op=op, T=_log_int(rng, 1, 32768), E=E, K=K, score=rng.choice(["sigmoid", "softmax"]),
                    groups=groups, keep=keep, group_top=rng.choice([1, 2]), bias=rng.random() < 0.7,
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))
    if op in ("norm", "norm_backward"):
        d = 64 * _log_int(rng, 1, 128)
        form = rng.choice(["both", "both", "pre", "post", "add"])
        y = form != "pre"
        return dict(op=op, T=_log_int(rng, 1, min(16384, 33554432 // d)), d=d, residual=rng.choice(["bf16", "fp32"]),
                    post=y and form != "add", pre=form != "post", y=y,
                    gate=rng.choice(["none", "channel", "token"]) if y else "none",
                    scale=rng.choice([1.0, 0.5, 0.70710678]) if y else 1.0)
    tensors = _log_int(rng, 1, 400)
    return dict(op=op, tensors=tensors, smallest=1, largest=_log_int(rng, 1000, 200_000_000 // tensors),
                dtype=rng.choice(["fp32", "bf16", "mixed"]), max_norm=rng.choice([1.0, 0.1, 1e6]))


# ------------------------------------------------------------------ inputs
def _sizes(case):
    """Element counts of the gradients: spread over the logarithm between the
    smallest and the largest, in a fixed scrambled order; or those of one layer."""
    if "E" in case:
        E, d, f = case["E"], case["d"], case["f"]
        return [E * 2 * f * d, E * d * f, d * E, E, d, d]   # dW1, dW2, dWr, dbias, two norms
    n, lo, hi = case["tensors"], case["smallest"], case["largest"]
    at = [((i * 7919) % n) / max(1, n - 1) for i in range(n)]
    return [int(round(math.exp(math.log(lo) + a * (math.log(hi) - math.log(lo))))) for a in at]


def _kinds(case):
    n = case["tensors"]
    return [F32 if case["dtype"] == "fp32" or (case["dtype"] == "mixed" and i % 3) else BF16 for i in range(n)]


def _cut(flat, sizes):
    return list(torch.split(flat, sizes)) if sizes else []


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case=case)
    op = case["op"]
    if op in ("route", "route_backward"):
        T, E, K = case["T"], case["E"], case["K"]
        # scores of a trained router: tokens differ, and some experts are more popular than others
        s["logits"] = normal(T, E) + 0.5 * normal(E)
        s["bias"] = 0.05 * normal(E) if case["bias"] else None
        if op == "route_backward":
            s["idx"] = _choose(case, s["logits"], s["bias"])[1].to(I32)
            s["dw"] = normal(T, K)
        if own:
            moe = _moe()
            s["rule"] = moe.RouteRule(score=case["score"], n_group=case["groups"], topk_group=case["keep"],
                                      group_top=case["group_top"], renorm=case["renorm"], scale=case["scale"])
            if op == "route":
                s["buffers"] = moe.RouteBuffers(T, E, K)
            else:
                s["out"] = torch.empty(T, E, device="cuda")
    elif op in ("norm", "norm_backward"):
        T, d = case["T"], case["d"]
        res = F32 if case["residual"] == "fp32" else BF16
        s["r"] = (3.0 * normal(T, d)).to(res)
        s["y"] = (0.2 * normal(T, d)).to(BF16) if case["y"] else None
        s["gp"] = 1.0 + 0.2 * normal(d) if case["post"] else None
        s["gq"] = 1.0 + 0.2 * normal(d) if case["pre"] else None
        s["gate"] = {"none": lambda: None, "channel": lambda: 0.3 + 0.1 * normal(d),
                     "token": lambda: torch.sigmoid(normal(T, 1))}[case["gate"]]()
        if op == "norm_backward":
            # what the forward left: its output stream and the two rows of factors
            r2, _, rp, rq = _norm(case, s, F32)
            s["r2"], s["rp"], s["rq"] = r2.to(res), rp, rq
            s["dr2"], s["dn"] = normal(T, d).to(res), normal(T, d).to(BF16) if case["pre"] else None
            del s["r"]
        if own:
            make = _moe().NormResidual.empty if op == "norm" else _moe().NormResidualGrads.empty
            s["out"] = make(T, d, res, y=case["y"], post=case["post"], pre=case["pre"], **(
                {} if op == "norm" else dict(gate=case["gate"])))
    else:
        sizes, kinds = _sizes(case), _kinds(case)
        of = {k: [n for n, q in zip(sizes, kinds) if q is k] for k in (F32, BF16)}
        flat = {k: (1e-3 * normal(sum(v))).to(k) for k, v in of.items() if v}
        cut = {k: iter(_cut(flat[k], of[k])) for k in flat}
        s["grads"] = [next(cut[k]) for k in kinds]
        s["kinds"] = kinds
        if own:
            # the clipped gradients go beside the raw ones, so that a pass can be repeated
            s["flat"] = {k: torch.empty_like(f) for k, f in flat.items()}
            cut = {k: iter(_cut(s["flat"][k], of[k])) for k in flat}
            s["clipper"] = _moe().GradClipper(s["grads"], outs=[next(cut[k]) for k in kinds])
    return s


# ------------------------------------------------------------------ plain forms
def _half(z):
    m = z.shape[1] // 2
    return z[:, :m] + z[:, m:]


def _scores(case, logits):
    """Scores of all experts.  The softmax's sum is folded by halves (E padded
    to 256 with zeros), so its 32-bit value has one definition."""
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    z = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
    pad = torch.zeros(z.shape[0], 256 - z.shape[1], dtype=z.dtype, device=z.device)
    return z / _half(_half(_half(_half(_half(_half(_half(_half(torch.cat([z, pad], dim=1)))))))))


def _choose(case, logits, bias):
    """Scores and the chosen experts (descending, the lowest index on ties)."""
    T, E, G = logits.shape[0], case["E"], case["groups"]
    s = _scores(case, logits)
    c = s if bias is None else s + bias
    if G > 1:
        inside = c.view(T, G, E // G).sort(dim=2, descending=True, stable=True).values
        score = inside[:, :, 0] if case["group_top"] == 1 or E == G else inside[:, :, 0] + inside[:, :, 1]
        kept = score.sort(dim=1, descending=True, stable=True).indices[:, :case["keep"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=c.device).scatter_(1, kept, True)
        c = torch.where(open_.repeat_interleave(E // G, dim=1), c, torch.full_like(c, -math.inf))
    return s, c.sort(dim=1, descending=True, stable=True).indices[:, :case["K"]]


def _weights(case, chosen):
    if case["renorm"]:
        return case["scale"] * chosen / (chosen.sum(dim=1, keepdim=True) + EPS_SUM)
    return case["scale"] * chosen


def _route(case, st):
    s, idx = _choose(case, st["logits"], st["bias"])
    w = _weights(case, s.gather(1, idx))
    T, K, E = case["T"], case["K"], case["E"]
    flat = idx.reshape(-1)
    counts = torch.zeros(E, dtype=torch.int64, device=flat.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    order = flat.sort(stable=True).indices
    row_of = torch.empty_like(order).scatter_(0, order, torch.arange(T * K, device=order.device))
    return dict(topk_idx=idx.to(I32), topk_w=w, counts=counts.to(I32), offsets=offsets.to(I32),
                row_of=row_of.view(T, K).to(I32), src_tok=(order // K).to(I32))


def _route_backward(case, logits, idx, dw):
    idx = idx.long()
    s = _scores(case, logits)
    a = case["scale"]
    t = s.gather(1, idx)
    if case["renorm"]:
        total = t.sum(dim=1, keepdim=True) + EPS_SUM
        ds = a * (dw - (dw * (t / total)).sum(dim=1, keepdim=True)) / total
    else:
        ds = a * dw
    zero = torch.zeros_like(s)
    if case["score"] == "sigmoid":
        return zero.scatter_(1, idx, ds * t / (1.0 + torch.exp(logits.gather(1, idx))))
    return s * (zero.scatter_(1, idx, ds) - (t * ds).sum(dim=1, keepdim=True))


def _norm(case, st, kind):
    """r' and n before any rounding, and the two rows of factors."""
    r2, rp, rq, n = st["r"].to(kind), None, None, None
    if case["y"]:
        u = st["y"].to(kind)
        if case["post"]:
            rp = 1.0 / torch.sqrt((u * u).mean(dim=1) + EPS_NORM)
            u = u * rp[:, None] * st["gp"].to(kind)
        if st["gate"] is not None:
            u = u * st["gate"].to(kind)
        r2 = case["scale"] * r2 + u
    if case["pre"]:
        rq = 1.0 / torch.sqrt((r2 * r2).mean(dim=1) + EPS_NORM)
        n = r2 * rq[:, None] * st["gq"].to(kind)
    return r2, n, rp, rq


def _norm_backward(case, st, kind):
    r2, D = st["r2"].to(kind), st["dr2"].to(kind)
    out = {}
    if case["pre"]:
        rq, dn = st["rq"].to(kind)[:, None], st["dn"].to(kind)
        h = dn * st["gq"].to(kind)
        out["dgamma_pre"] = (dn * r2 * rq).sum(dim=0)
        D = D + rq * (h - r2 * rq * rq * (h * r2).mean(dim=1, keepdim=True))
    out["dr"] = case["scale"] * D
    if case["y"]:
        y = st["y"].to(kind)
        v = y                       # the normalised output, before its weight
        k = D                       # the gradient of what the gate multiplies
        u = y
        if case["post"]:
            rp = st["rp"].to(kind)[:, None]
            v = y * rp
            u = v * st["gp"].to(kind)
        if st["gate"] is not None:
            out["dgate"] = (u * D).sum(dim=0) if case["gate"] == "channel" else (u * D).sum(dim=1, keepdim=True)
            k = D * st["gate"].to(kind)
        if case["post"]:
            out["dgamma_post"] = (k * v).sum(dim=0)
            k = k * st["gp"].to(kind)
            k = rp * (k - y * rp * rp * (k * y).mean(dim=1, keepdim=True))
        out["dy"] = k
    return out


def _clip(case, st, kind):
    total = torch.stack([(x.to(kind) * x.to(kind)).sum() for x in st["grads"]]).sum()
    norm = torch.sqrt(total)
    c = torch.clamp(case["max_norm"] / (norm + EPS_CLIP), max=1.0)
    return norm, [x.to(kind) * c for x in st["grads"]]


def _flat(outs, kinds):
    """The clipped gradients of each type, packed as the inputs are."""
    return {str(k).split(".")[1]: torch.cat([o for o, q in zip(outs, kinds) if q is k]).to(k)
            for k in (F32, BF16) if k in kinds}


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        return _run_own(case, op, st)
    if op == "route":
        return _route(case, st)
    if op == "route_backward":
        return _route_backward(case, st["logits"], st["idx"], st["dw"])
    if op == "norm":
        r2, n, rp, rq = _norm(case, st, F32)
        return dict(r=r2.to(st["r"].dtype), n=None if n is None else n.to(BF16), rstd_post=rp, rstd_pre=rq)
    if op == "norm_backward":
        out = _norm_backward(case, st, F32)
        out["dr"] = out["dr"].to(st["r2"].dtype)
        if case["y"]:
            out["dy"] = out["dy"].to(BF16)
        return out
    norm, outs = _clip(case, st, F32)
    return dict(norm=norm.reshape(1), **_flat(outs, st["kinds"]))


def _run_own(case, op, st):
    moe = _moe()
    if op == "route":
        r = moe.route_scored(st["logits"], case["K"], st["rule"], sel_bias=st["bias"], buffers=st["buffers"])
        return dict(topk_idx=r.topk_idx, topk_w=r.topk_w, counts=r.counts, offsets=r.offsets, row_of=r.row_of,
                    src_tok=r.src_tok)
    if op == "route_backward":
        return moe.route_scored_backward(st["logits"], st["idx"], st["dw"], st["rule"], out=st["out"])
    if op == "norm":
        o = moe.norm_residual(st["r"], st["y"], gamma_post=st["gp"], gate=st["gate"], gamma_pre=st["gq"],
                              res_scale=case["scale"], eps=EPS_NORM, out=st["out"])
        return dict(r=o.r, n=o.n, rstd_post=o.rstd_post, rstd_pre=o.rstd_pre)
    if op == "norm_backward":
        g = moe.norm_residual_backward(st["r2"], st["dr2"], st["dn"], st["y"], gamma_post=st["gp"], gate=st["gate"],
                                       gamma_pre=st["gq"], res_scale=case["scale"], rstd_post=st["rp"],
                                       rstd_pre=st["rq"], out=st["out"])
        return {k: v for k, v in dict(dr=g.dr, dy=g.dy, dgamma_pre=g.dgamma_pre, dgamma_post=g.dgamma_post,
                                      dgate=g.dgate).items() if v is not None}
    norm = st["clipper"](case["max_norm"])
    return dict(norm=norm, **{str(k).split(".")[1]: f for k, f in st["flat"].items()})


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_backward"):
        T, E, K, G = case["T"], case["E"], case["K"], case["groups"]
        l = st["logits"].double()
        s = torch.softmax(l, dim=1) if case["score"] == "softmax" else torch.sigmoid(l)
        if op == "route_backward":
            # the choice is an input; the gradient of sum(dw * w) by its definition
            idx = st["idx"].long()
            l = l.requires_grad_(True)
            s = torch.softmax(l, dim=1) if case["score"] == "softmax" else torch.sigmoid(l)
            t = torch.gather(s, 1, idx)
            w = t / (t.sum(1, keepdim=True) + EPS_SUM) if case["renorm"] else t
            return torch.autograd.grad((case["scale"] * w * st["dw"].double()).sum(), l)[0]
        # the ranking is of scores as they are held, in 32 bits; an entry that is taken is lowered below all
        c = (s if st["bias"] is None else s + st["bias"].double()).float().double()
        if G > 1:
            per = c.view(T, G, E // G)
            score = per.topk(min(case["group_top"], E // G), dim=2).values.sum(2)
            last = score.topk(case["keep"], dim=1).values[:, -1:]
            c = torch.where((score >= last).repeat_interleave(E // G, dim=1), c, -math.inf)
        lowest_first = torch.argsort(-c, dim=1, stable=True)[:, :K]
        t = torch.gather(s, 1, lowest_first)
        w = case["scale"] * (t / (t.sum(1, keepdim=True) + EPS_SUM) if case["renorm"] else t)
        return dict(topk_idx=None, topk_w=w, counts=None, offsets=None, row_of=None, src_tok=None)
    if op in ("norm", "norm_backward"):
        y = st["y"].double() if case["y"] else None
        gp = st["gp"].double() if case["post"] else None
        gq = st["gq"].double() if case["pre"] else None
        gate = st["gate"].double() if st["gate"] is not None else None
        if op == "norm":
            r, rp, rq, n = st["r"].double(), None, None, None
            if y is not None:
                z = y
                if gp is not None:
                    rp = (y.square().mean(1) + EPS_NORM).rsqrt()
                    z = y * rp.unsqueeze(1) * gp
                r = case["scale"] * r + (z if gate is None else z * gate)
            if gq is not None:
                rq = (r.square().mean(1) + EPS_NORM).rsqrt()
                n = r * rq.unsqueeze(1) * gq
            return dict(r=r, n=n, rstd_post=rp, rstd_pre=rq)
        # the rows' factors are inputs; with x = r' and m = mean, the Jacobian of x -> x * f(x) * weight
        x, D, out = st["r2"].double(), st["dr2"].double(), {}
        d = case["d"]
        if gq is not None:
            f, dn = st["rq"].double().unsqueeze(1), st["dn"].double()
            out["dgamma_pre"] = torch.einsum("td,td->d", dn, x * f)
            D = D + f * dn * gq - x * f ** 3 * (torch.einsum("td,td,d->t", dn, x, gq) / d).unsqueeze(1)
        out["dr"] = D * case["scale"]
        if y is not None:
            f = st["rp"].double().unsqueeze(1) if gp is not None else None
            z = y if gp is None else y * f
            weight = 1.0 if gp is None else gp
            if gate is not None:
                out["dgate"] = torch.einsum("td,td->d", z * weight, D) if case["gate"] == "channel" else \
                    torch.einsum("td,td->t", z * weight, D).unsqueeze(1)
            e = D if gate is None else D * gate
            if gp is not None:
                out["dgamma_post"] = torch.einsum("td,td->d", e, z)
                e = f * e * gp - y * f ** 3 * (torch.einsum("td,td,d->t", e, y, gp) / d).unsqueeze(1)
            out["dy"] = e
        return out
    total = math.fsum(float(torch.linalg.vector_norm(x, dtype=F64)) ** 2 for x in st["grads"])
    norm = math.sqrt(total)
    out = dict(norm=torch.tensor([norm], dtype=F64))
    c = min(1.0, case["max_norm"] / (norm + EPS_CLIP))
    for k in (F32, BF16):
        if k in st["kinds"]:
            out[str(k).split(".")[1]] = torch.cat([x for x, q in zip(st["grads"], st["kinds"]) if q is k]).double() * c
    return out


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "route":
        T, E, K = case["T"], case["E"], case["K"]
        # a score is about 6 operations an expert (negate, exp, add, divide, bias, compare)
        return dict(bytes=4 * T * E + 4 * E * case["bias"] + 16 * T * K + 4 * (2 * E + 1), flops=6 * T * E)
    if op == "route_backward":
        T, E, K = case["T"], case["E"], case["K"]
        dense = case["score"] == "softmax"
        return dict(bytes=4 * T * E + 8 * T * K + (4 * T * E if dense else 4 * T * K),
                    flops=8 * T * E if dense else 12 * T * K)
    if op in ("norm", "norm_backward"):
        T, d = case["T"], case["d"]
        R = 4 if case["residual"] == "fp32" else 2
        rows = case["post"] + case["pre"] + (case["gate"] == "token")
        cols = case["post"] + case["pre"] + (case["gate"] == "channel")
        if op == "norm":
            through = R + (2 + R if case["y"] else 0) + 2 * case["pre"]
            return dict(bytes=T * d * through + 4 * T * rows + 4 * d * cols, flops=10 * T * d)
        through = 2 * R + (R + 2 if case["pre"] else 0) + (4 if case["y"] else 0)
        return dict(bytes=T * d * through + 4 * T * (rows + (case["gate"] == "token")) + 8 * d * cols, flops=24 * T * d)
    sizes, kinds = _sizes(case), _kinds(case)
    n = sum(v * (4 if k is F32 else 2) for v, k in zip(sizes, kinds))
    return dict(bytes=2 * n + 4, flops=3 * sum(sizes))
