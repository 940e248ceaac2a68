"""The MXFP8 steps behind routing by scores."""
import pytest
import torch

import dropless_moe_expert_gb300 as moe
from workloads import Shape, make_tokens, make_weights

from _bounds import check_within
from _helpers import to_np

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24


@pytest.mark.parametrize("s", [Shape(T=300, d=256, E=64, K=8, f=128), Shape(T=517, d=256, E=16, K=4, f=512, bias="normal_0.5")],
                         ids=str)
def test_mxfp8_steps_behind_scored_routing(s):
    """Renormalised softmax scores are the softmax over the chosen logits: the same experts in the same order, so the
    grouped products have the same bits, and the gate weights differ by roundings (24 + K + 2 D of them for logits
    that spread over D).  Then another rule, whose output is its weights' sum of those rows."""
    w = make_weights(s, seed=3, device="cpu")
    x = make_tokens(s, seed=4, device="cpu").cuda()
    W1q, W1s = moe.mxfp8_quantize(w.W1.cuda())
    W2q, W2s = moe.mxfp8_quantize(w.W2.cuda())
    logits = moe.router_logits(x, w.Wr.cuda(), w.bias.cuda())

    def steps(r):
        xq, sfa = moe.permute_mxfp8(x, r)
        h, sfh = moe.grouped_gemm1_swiglu_mxfp8(xq, sfa, r.offsets, W1q, W1s)
        y_perm = moe.grouped_gemm2_mxfp8(h, sfh, r.offsets, W2q, W2s)
        return y_perm, moe.unpermute(y_perm, r.row_of, r.topk_w)

    own, scored = moe.route(logits, s.K), moe.route_scored(logits, s.K, moe.RouteRule("softmax"))
    for k in ("topk_idx", "counts", "offsets", "row_of", "src_tok"):
        assert torch.equal(getattr(own, k), getattr(scored, k)), k
    D = float((logits.max(dim=1).values - logits.min(dim=1).values).max())
    n = 24 + s.K + 2 * D
    check_within(scored.topk_w, to_np(own.topk_w).astype("float64"), 2 * n * ULP * to_np(own.topk_w))
    y_perm, y = steps(scored)
    assert torch.equal(y_perm, steps(own)[0])

    def check(r, y_perm, y):
        rows = to_np(y_perm).astype("float64")[to_np(r.row_of)]
        terms = rows * to_np(r.topk_w).astype("float64")[..., None]
        check_within(y, terms.sum(axis=1), (s.K + 1) * ULP * abs(terms).sum(axis=1) + 1e-37)

    check(scored, y_perm, y)
    other = moe.route_scored(logits, s.K, moe.RouteRule("sigmoid", 4, 3, 2, True, 2.5),
                             sel_bias=0.1 * torch.randn(s.E, generator=torch.Generator().manual_seed(5)).cuda())
    check(other, *steps(other))
