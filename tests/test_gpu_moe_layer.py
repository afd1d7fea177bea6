"""The example layer (8-bit rows and experts through the whole path) and its
training step against a 64-bit computation of the same layer.

The 64-bit layer rounds to 8 bits where the layer does.  Its rounding differs
only where a value lies within fp32 error of a rounding boundary: at most one
in a thousand values, each off by at most 2^-3 of itself, which moves the
result by at most 2^-3 * sqrt(1e-3) = 0.004 of its norm; bf16 roundings add
2^-8 at each of three places (y, z, out): 0.016 in all."""
import os
import sys

import pytest
import torch

import _ops_ref as R

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def rows8(y):
    """y rounded to 8-bit rows, as what they stand for."""
    s = R.spread((R.block_max(y).clamp_min(2.0 ** -100) / 448), y.shape[1])
    return (y / s).clamp(-448, 448).to(torch.float8_e4m3fn).double() * s


def matrices(q, s):
    m = q.double() * R.spread(R.spread(s.double(), q.shape[-1]).transpose(-1, -2), q.shape[-2]).transpose(-1, -2)
    return m


def layer64(layer, x, residual):
    y, h, _ = R.norm(x, layer.norm, residual)
    logits = (y.to(torch.bfloat16) @ layer.gate)
    r = R.route(logits, layer.topk)
    a = rows8(y)
    w13, w2 = matrices(layer.w13, layer.s13), matrices(layer.w2, layer.s2)
    out = torch.zeros_like(a)
    for e in range(w13.shape[0]):
        t, k = (r["idx"] == e).nonzero(as_tuple=True)
        if len(t):
            gate, up = a[t] @ w13[e, 0].t(), a[t] @ w13[e, 1].t()
            out.index_add_(0, t, r["weights"][t, k, None] * (rows8(gate * torch.sigmoid(gate) * up) @ w2[e].t()))
    return out, h, r


@pytest.mark.parametrize("ranks,tpr,hidden,experts,topk,inter", [
    (4, 16, 256, 16, 2, 128), (1, 33, 272, 4, 3, 144), (8, 25, 1024, 64, 8, 256), (2, 300, 512, 8, 4, 384),
    (32, 4, 256, 32, 4, 128)])
def test_layer(ranks, tpr, hidden, experts, topk, inter):
    from moe_layer import MoeLayer
    layer = MoeLayer(ranks, tpr, hidden, experts, topk, inter)
    g = torch.Generator(device="cuda").manual_seed(hidden + tpr)
    x, res = (torch.randn(ranks * tpr, hidden, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    out, stream = layer(x, res)
    want, h, r = layer64(layer, x, res)
    assert layer.send.device_status() == 0 and layer.back.device_status() == 0
    assert ((out.double() - want).norm() / want.norm()).item() < 0.016
    assert ((stream.double() - h).norm() / h.norm()).item() < 2.0 ** -8
    layer.close()


def test_layer_with_tokens_that_reach_nobody():
    """Rows without picks come back as zeros (expert layout and sum see no row of theirs)."""
    import combine_ep_layout_04_gb300 as ep
    from moe_layer import MoeLayer
    layer = MoeLayer(4, 8, 256, 16, 2, 128)
    x = torch.randn(32, 256, device="cuda").to(torch.bfloat16)
    n = ep.rms_norm(x, layer.norm, fp8=True, with_bf16=True)
    mask = torch.arange(32, device="cuda") % 3 != 0
    r = ep.route(n.bf16 @ layer.gate, 2, num_ranks=4, token_mask=mask)
    lay = layer.send.layout(r.topk_idx)
    recv = layer.send.dispatch(n.out.packed, lay)
    xl = layer.send.expert_layout(r.topk_idx, r.topk_weights, lay)
    out = layer.back.combine(layer.experts(ep.Fp8Rows.from_packed(recv, 256), lay, xl), r.rank_weights, r.topk_idx,
                             lay)
    assert (out[~mask] == 0).all() and (out[mask].float().abs().sum(1) > 0).all()
    assert layer.send.device_status() == 0 and layer.back.device_status() == 0
    layer.close()


def test_train_step():
    from moe_layer import MoeLayer
    layer = MoeLayer(4, 32, 256, 16, 2, 128)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, res, dy = (torch.randn(128, 256, device="cuda", generator=g).to(torch.bfloat16) for _ in range(3))
    dw = torch.randn(128, 2, device="cuda", generator=g)
    dx, dnorm, dgate, loss = layer.train_step(x, res, lambda r: dw, dy, 0.01)
    # the same by torch's autograd in 64 bits, with the picks and counts held
    xv, wv, gv = (t.double().requires_grad_() for t in (x, layer.norm, layer.gate))
    h = xv + res.double()
    y = h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * wv
    logits = y @ gv
    with torch.no_grad():
        n = (y.to(torch.bfloat16) @ layer.gate)
        fixed = R.route(n, 2, True, None, 0.01)
    p = torch.softmax(logits, 1)
    weights = torch.softmax(logits.gather(1, fixed["idx"]), 1)
    balance = (fixed["slope"] * p.sum(0)).sum()
    ((weights * dw).sum() + balance + (y * dy.double()).sum()).backward()
    # bf16 logits, rows and sums of them: a few roundings of 2^-8 in series
    for got, want in ((dx, xv.grad), (dnorm, wv.grad), (dgate, gv.grad), (loss, balance.detach())):
        assert ((got.double() - want).norm() / want.norm()).item() < 0.03
    layer.close()
