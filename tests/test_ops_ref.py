"""The operators' 64-bit forms (CPU): their gradients against central
differences of their forward forms, and the corner rows they define."""
import pytest
import torch

import _ops_ref as R


def differences(f, x, eps=1e-6):
    """Central differences of the scalar f at x."""
    g = torch.zeros_like(x)
    flat, gf = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + eps
        hi = f()
        flat[i] = keep - eps
        lo = f()
        flat[i] = keep
        gf[i] = (hi - lo) / (2 * eps)
    return g


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def test_norm_gradient_against_differences():
    x, res, w = rnd(1, 3, 8), rnd(2, 3, 8), rnd(3, 8)
    dout, dres = rnd(4, 3, 8), rnd(5, 3, 8)

    def loss():
        y, h, _ = R.norm(x, w, res, 1e-6)
        return ((y * dout).sum() + (h * dres).sum()).item()

    _, h, r = R.norm(x, w, res, 1e-6)
    dx, dw = R.norm_grad(dout, h, w, r, dres)
    # differences of step 1e-6 in 64 bits are good to about 1e-9 of values of size one
    assert (differences(loss, x) - dx).abs().max() < 1e-7
    assert (differences(loss, res) - dx).abs().max() < 1e-7
    assert (differences(loss, w) - dw).abs().max() < 1e-7


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(renorm):
    T, E, K = 5, 7, 3
    logits = rnd(6, T, E) * 2
    logits[1, 4] = float("-inf")
    mask = torch.tensor([True, True, False, True, True])
    dw = rnd(7, T, K)
    fixed = R.route(logits, K, renorm, mask, 0.3)

    def loss():
        r = R.route(logits, K, renorm, mask, 0.3)
        assert torch.equal(r["idx"], fixed["idx"])            # the picks stay the same
        # f (the counts) is a constant of the loss, so the slope is too
        return ((r["weights"] * dw).sum() + 0.7 * (fixed["slope"] * r["p"].sum(0)).sum()).item()

    want = R.route_grad(fixed, renorm, dw, 0.7)
    got = differences(loss, logits)
    got[~torch.isfinite(logits)] = 0.0
    assert (got - want).abs().max() < 1e-7
    assert (want[2] == 0).all() and want[1, 4] == 0


def test_route_corner_rows():
    ninf, nan = float("-inf"), float("nan")
    logits = torch.tensor([[1.0, 1.0, 2.0], [ninf, ninf, ninf], [ninf, 3.0, ninf], [nan, 1.0, 0.0], [nan, nan, nan]])
    r = R.route(logits, 2, True, None, 1.0)
    assert r["idx"].tolist() == [[2, 0], [-1, -1], [1, -1], [1, 2], [-1, -1]]
    assert r["weights"][1].tolist() == [0, 0] and r["weights"][2].tolist() == [1, 0]
    assert (r["p"][1] == 0).all() and r["p"][3].isnan().all() and r["p"][4].isnan().all()
    masked = R.route(logits, 2, True, torch.tensor([True, True, True, False, False]), 1.0)
    assert masked["loss"].isfinite() and (masked["p"][3:] == 0).all()
