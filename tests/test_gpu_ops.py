"""The operators of include/ep_ops.h on the GPU against their 64-bit forms.

Tolerances, fixed by the arithmetic: a bf16 output is rounded once, so it is
within 2^-8 of its value (half a unit in the last of 8 significant bits), an
e4m3 one within 2^-4 of it or half a step (2^-10) of the subnormal range;
before that the kernels work in fp32, where a sum of n terms is off by at most
n * 2^-24 of the sum of their magnitudes.  The tensor cores may truncate where
an fp32 add rounds, so their sums get 2^-23 a term."""
import pytest
import torch

import _ops_ref as R

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
HALF_BF, HALF_F8, SUB_F8 = 2.0 ** -8, 2.0 ** -4, 2.0 ** -10
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ep():
    import combine_ep_layout_04_gb300 as ep
    return ep


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


def near(got, want, bound):
    """got within `bound` of want everywhere; NaN and infinities alike."""
    got, want = got.double(), want.double()
    fine = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()])
    off = (got - want).abs()[fine] - bound.expand_as(want)[fine]
    assert off.numel() == 0 or off.max().item() <= 0, off.max().item()


def near_rows8(rows, want, rel):
    """8-bit rows stand for `want` (whose own error is at most rel of it)."""
    width = want.shape[1]
    most = R.block_max(want).clamp_min(2.0 ** -100)
    near(rows.scales, most / 448, most / 448 * (rel + 4 * U))
    s = R.spread(rows.scales.double(), width)
    near(rows.values.double() * s, want, want.abs() * (HALF_F8 * 1.01 + 2 * rel) + s.abs() * SUB_F8 * 1.01)


# ------------------------------------------------------------------ the norm
NORM_SHAPES = [(1, 8), (1, 7168), (2, 24), (7, 136), (129, 256), (5, 520), (33, 1000), (64, 1024), (3, 1032),
               (130, 2048), (17, 4104), (66, 7168), (2, 32768)]


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("wtype", [BF, torch.float32])
def test_norm(ep, T, H, residual, wtype):
    g = gen(T * 131 + H)
    x, w = rnd(g, T, H, dtype=BF), (1 + 0.2 * rnd(g, H)).to(wtype)
    res = (rnd(g, T, H) * 3).to(BF) if residual else None
    y, h, r = R.norm(x, w, res)
    # r: a sum of H squares, halved by the root, and a few single operations
    rel = (40 + H ** 0.5) * U
    n = ep.rms_norm(x, w, residual=res, save_rstd=True)
    near(n.out, y, y.abs() * (HALF_BF + rel))
    near(n.rstd, r, r * rel)
    n8 = ep.rms_norm(x, w, residual=res, fp8=True)
    near_rows8(n8.out, y, rel)
    if residual:
        near(n.residual, h, h.abs() * (HALF_BF + U))
        assert torch.equal(n8.residual, n.residual)
    else:
        assert n.residual is None and n8.residual is None


def test_norm_strided_rows_and_in_place(ep):
    g = gen(3)
    buf = rnd(g, 9, 3 * 264, dtype=BF)
    x, res = buf[:, :264], buf[:, 264:528]
    w = rnd(g, 264)
    y, h, _ = R.norm(x, w, res)
    keep = buf[:, 528:].clone()
    out = torch.zeros(9, 512, dtype=BF, device="cuda")
    n = ep.rms_norm(x, w, residual=res, residual_out=res, out=out[:, 8:272])
    near(res, h, h.abs() * (HALF_BF + U))
    near(out[:, 8:272], y, y.abs() * (HALF_BF + 60 * U))
    assert n.residual is res and (out[:, :8] == 0).all() and (out[:, 272:] == 0).all()
    assert torch.equal(buf[:, 528:], keep)


def test_norm_rows_with_infinities_zeros_and_extremes(ep):
    H = 384
    x = torch.ones(6, H, dtype=BF, device="cuda")
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 1e-30           # squares underflow: the row is scaled by 1 / sqrt(eps)
    x[5, 130] = 1e18
    w = torch.ones(H, device="cuda")
    n = ep.rms_norm(x, w, fp8=True)
    y, _, _ = R.norm(x, w)
    assert n.out.values[2].float().isnan().all() and n.out.scales[2].isnan().all()
    assert n.out.scales[3, 0].isnan() and (n.out.values[3, 128:].float() == 0).all()
    for row in (0, 1, 4, 5):
        near_rows8(ep.Fp8Rows(n.out.values[row:row + 1], n.out.scales[row:row + 1]), y[row:row + 1], 1e-5)


@pytest.mark.parametrize("T,H", NORM_SHAPES + [(1700, 136), (1300, 2048)])
@pytest.mark.parametrize("dres", [True, False])
def test_norm_backward(ep, T, H, dres):
    g = gen(T * 7 + H)
    h, dout, w = rnd(g, T, H, dtype=BF), rnd(g, T, H, dtype=BF), (1 + 0.2 * rnd(g, H)).to(BF)
    dr = rnd(g, T, H, dtype=BF) if dres else None
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    dx, dw = ep.rms_norm_backward(dout, h, w, rstd, dresidual=dr)
    want, wantw = R.norm_grad(dout, h, w, rstd, dr)
    du = (dout.double() * w.double()).abs()
    u = (h.double() * rstd.double()[:, None]).abs()
    size = rstd.double()[:, None] * (du + u * (du * u).mean(-1, keepdim=True)) + (0 if dr is None else dr.abs())
    near(dx, want, want.abs() * HALF_BF + size * (40 + H ** 0.5) * U)
    # a team adds at most a few rows, the teams' sums are added in chains of at most 64
    near(dw, wantw, (dout.double().abs() * u).sum(0) * 80 * U + 1e-30)
    again = ep.rms_norm_backward(dout, h, w, rstd, dresidual=dr, dx=dr if dres else dout)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_norm_of_nothing(ep):
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    assert ep.rms_norm(x, w, fp8=True).out.values.shape == (0, 64)
    dx, dw = ep.rms_norm_backward(x, x, w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and (dw == 0).all()


# ---------------------------------------------------------------- the router
ROUTE_SHAPES = [(1, 1, 1), (5, 2, 2), (64, 16, 2), (33, 31, 5), (9, 33, 1), (700, 64, 6), (300, 100, 32),
                (257, 256, 8), (40, 500, 7), (12, 1000, 8), (6, 1025, 3), (3, 4096, 32)]


def check_route(ep, logits, K, renorm, mask, coef, ranks=None):
    got = ep.route(logits, K, renormalize=renorm, token_mask=mask, balance_coef=coef, num_ranks=ranks)
    want = R.route(logits, K, renorm, mask, coef)
    assert torch.equal(got.topk_idx.long(), want["idx"])
    # the exponent's argument is off by a unit of its own size, the sum by its terms
    top = torch.where(logits.isfinite(), logits.double(), 0.0).abs().amax(1, keepdim=True)
    rel = (24 + 4 * top + logits.shape[1] / 32) * U
    near(got.topk_weights, want["weights"], want["weights"] * rel + 1e-37)
    if coef is not None:
        assert torch.equal(got.expert_count.long(), want["count"])
        near(got.slope, want["slope"], want["slope"] * 8 * U)
        near(got.lse, want["lse"], want["lse"].abs() * 4 * U + rel[:, 0])
        # the sum over tokens goes by warp, block and block again
        near(got.balance_loss, want["loss"], want["loss"].abs() * (rel.max() + 100 * U))
    return got, want


@pytest.mark.parametrize("T,E,K", ROUTE_SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("masked", [False, True])
def test_route_and_gradient(ep, T, E, K, dtype, renorm, masked):
    g = gen(T * 17 + E + K)
    logits = (rnd(g, T, E) * 3).to(dtype)
    mask = None
    if masked:
        logits[torch.rand(T, E, device="cuda", generator=g) < 0.2] = R.NEG
        logits[torch.rand(T, device="cuda", generator=g) < 0.1] = R.NEG
        logits[torch.rand(T, device="cuda", generator=g) < 0.1] = torch.finfo(dtype).min
        mask = torch.rand(T, device="cuda", generator=g) < 0.8
        logits[~mask & (torch.rand(T, device="cuda", generator=g) < 0.5)] = float("nan")
        logits[~mask & (torch.rand(T, device="cuda", generator=g) < 0.5), 0] = float("inf")
    check_route(ep, logits, K, renorm, mask, None)
    got, want = check_route(ep, logits, K, renorm, mask, 0.5)
    dw, dl = rnd(g, T, K), torch.tensor(0.7, device="cuda")
    dw[want["idx"] < 0] = float("nan")              # no pick: not used
    d = ep.route_backward(logits, got, dw, dl)
    ref = R.route_grad(want, renorm, dw, dl.double())
    assert d.dtype == dtype
    p, at = want["p"], want["idx"].clamp_min(0)
    dwa = torch.where(want["idx"] >= 0, dw.double().abs(), 0.0)
    gabs = (want["slope"] * 0.7).expand_as(p)
    if renorm:
        w = want["weights"]
        size = p * (gabs + (p * gabs).sum(1, keepdim=True)) + torch.zeros_like(p).scatter_add_(
            1, at, w * (dwa + (w * dwa).sum(1, keepdim=True)))
    else:
        gabs = gabs.scatter_add(1, at, dwa)
        size = p * (gabs + (p * gabs).sum(1, keepdim=True))
    top = torch.where(want["lse"].isfinite(), want["lse"], 0.0).abs().clamp_max(40)[:, None]
    rel = (40 + 8 * (top + 20) + E / 32) * U        # p's argument l - lse, and lse's own error
    near(d, ref, ref.abs() * (HALF_BF if dtype == BF else 0) + size * rel + 1e-37)
    # no loss: only the picks' part
    d0 = ep.route_backward(logits, got, dw)
    ref0 = R.route_grad(want, renorm, dw, 0.0)
    near(d0, ref0, ref0.abs() * (HALF_BF if dtype == BF else 0) + size * rel + 1e-37)
    inplace = logits.clone()
    assert torch.equal(ep.route_backward(inplace, got, dw, dl, dlogits=inplace), d)


def test_route_ties_and_signed_zeros(ep):
    g = gen(11)
    logits = torch.randint(-1, 2, (400, 96), device="cuda", generator=g).float()
    logits[torch.rand(400, 96, device="cuda", generator=g) < 0.3] = -0.0
    check_route(ep, logits, 9, True, None, 1.0)
    check_route(ep, logits.to(BF), 9, False, None, 1.0)


def test_route_rows_with_nan(ep):
    g = gen(12)
    logits = rnd(g, 40, 48)
    logits[3, 7] = float("nan")
    logits[4] = float("nan")
    logits[5, 1] = float("inf")
    for renorm in (True, False):
        got = ep.route(logits, 4, renormalize=renorm)
        want = R.route(logits, 4, renorm)
        assert torch.equal(got.topk_idx.long(), want["idx"])
        rest = [i for i in range(40) if i not in (3, 4, 5)]
        near(got.topk_weights[rest], want["weights"][rest], want["weights"][rest] * 1e-5)
        assert (got.topk_weights[4] == 0).all() and got.topk_weights[5, 0].isnan()
        assert got.topk_weights[3].isnan().all() == (not renorm)
    assert ep.route(logits, 4, balance_coef=1.0).balance_loss.isnan()


@pytest.mark.parametrize("ranks", [1, 4, 32])
def test_route_rank_weights(ep, ranks):
    g = gen(13)
    logits = rnd(g, 200, 64)
    logits[torch.rand(200, 64, device="cuda", generator=g) < 0.9] = R.NEG
    got = ep.route(logits, 8, num_ranks=ranks)
    idx = got.topk_idx.cpu().tolist()
    want = [[float(e >= 0 and e // (64 // ranks) not in [f // (64 // ranks) for f in row[:k] if f >= 0])
             for k, e in enumerate(row)] for row in idx]
    assert got.rank_weights.cpu().tolist() == want


def test_route_strided_logits(ep):
    g = gen(14)
    wide = rnd(g, 50, 200)
    part = wide[:, 3:70]
    got, want = check_route(ep, part, 5, True, None, 1.0)
    into = torch.zeros(50, 201, device="cuda")
    d = ep.route_backward(part, got, torch.ones(50, 5, device="cuda"), dlogits=into[:, 1:68])
    assert torch.equal(d, ep.route_backward(part.contiguous(), got, torch.ones(50, 5, device="cuda")))
    assert (into[:, 0] == 0).all() and (into[:, 68:] == 0).all()


def test_route_of_nothing(ep):
    r = ep.route(torch.empty(0, 16, device="cuda"), 2, balance_coef=1.0)
    assert r.topk_idx.shape == (0, 2) and (r.expert_count == 0).all() and r.balance_loss.item() == 0
    assert ep.route_backward(torch.empty(0, 16, device="cuda"), r, torch.empty(0, 2, device="cuda")).shape == (0, 16)


def test_route_is_the_same_every_time(ep):
    g = gen(15)
    logits = rnd(g, 30011, 256)
    a, b = (ep.route(logits, 8, balance_coef=1.0) for _ in range(2))
    assert torch.equal(a.balance_loss, b.balance_loss) and torch.equal(a.slope, b.slope)


# -------------------------------------------------------------- the products
def rows8(g, ep, M, K):
    a = ep.Fp8Rows.empty(M, K)
    a.values.copy_(rnd(g, M, K) * 100)
    a.scales.copy_(torch.rand(M, a.scales.shape[1], device="cuda", generator=g) / 100)
    return a


def weights8(g, *shape):
    s = (*shape[:-2], -(-shape[-2] // 128), -(-shape[-1] // 128))
    return (rnd(g, *shape) * 50).to(F8), torch.rand(*s, device="cuda", generator=g) / 100 + 1e-3


def places(counts, gaps=None):
    off, at = [], 0
    for i, n in enumerate(counts):
        at += gaps[i] if gaps else 0
        off.append(at)
        at += n
    i32 = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(off, **i32), torch.tensor(counts, **i32), at


def check_product(ep, a, w, s, off, count, rows=None, **kw):
    got = ep.expert_product(a, w, s, off, count, rows=rows, **kw)
    y, S = R.product(a.values, a.scales, w, s, off, count, rows)
    K = a.values.shape[1]
    err = S * (min(K, 128) + -(-K // 128) + 4) * 2.0 ** -23
    live = ~(y[:, 0] if w.dim() == 3 else y[:, 0, 0]).isnan()
    if w.dim() == 3:
        near(got[live], y[live], (y.abs() * HALF_BF + err)[live] + 1e-38)
    else:
        gate, up = y[live][:, 0], y[live][:, 1]
        h = gate * torch.sigmoid(gate) * up
        eh = 1.1 * up.abs() * err[live][:, 0] + (gate * torch.sigmoid(gate)).abs() * err[live][:, 1] + h.abs() * 16 * U
        most, em = R.block_max(h).clamp_min(2.0 ** -100), R.block_max(eh)
        near(got.scales[live], most / 448, em / 448 + most * 4 * U)
        sc = R.spread(got.scales[live].double(), h.shape[1])
        near(got.values[live].double() * sc, h, h.abs() * HALF_F8 * 1.01 + sc * SUB_F8 * 1.01 + 2 * eh)
    return got


@pytest.mark.parametrize("counts", [[1], [0, 3, 0], [128], [129, 1, 64, 0, 127, 300], [37, 256]])
@pytest.mark.parametrize("N,K", [(8, 16), (128, 128), (136, 144), (264, 400), (512, 1024)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("gather", [False, True])
def test_product(ep, counts, N, K, gated, gather):
    g = gen(sum(counts) + N + K + gated)
    off, count, M = places(counts)
    w, s = weights8(g, *((len(counts), 2, N, K) if gated else (len(counts), N, K)))
    if gather:
        a = rows8(g, ep, max(1, M // 2), K)
        rows = torch.randint(a.values.shape[0], (M,), device="cuda", generator=g, dtype=torch.int32)
        check_product(ep, a, w, s, off, count, rows)
    else:
        check_product(ep, rows8(g, ep, M, K), w, s, off, count)


@pytest.mark.parametrize("counts", [[129], [300, 0, 400, 1], [513, 130], [256, 257]])
@pytest.mark.parametrize("N,K", [(8, 16), (72, 272), (136, 144), (264, 400), (512, 1024)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("gather", [False, True])
def test_product_many_places_to_an_expert(ep, counts, N, K, gated, gather):
    test_product(ep, counts, N, K, gated, gather)


@pytest.mark.parametrize("counts", [[130] + [0] * 9, [0, 65, 1, 33, 0, 0, 0, 0, 64, 0, 2, 32], [3] * 20, [16]])
@pytest.mark.parametrize("N,K", [(8, 16), (136, 144), (264, 400), (512, 1024)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("gather", [False, True])
def test_product_few_places_to_an_expert(ep, counts, N, K, gated, gather):
    test_product(ep, counts, N, K, gated, gather)


@pytest.mark.parametrize("gated", [False, True])
def test_product_long_rows_many_experts(ep, gated):
    g = gen(31)
    counts = [(i * 7) % 40 for i in range(40)]
    off, count, M = places(counts)
    w, s = weights8(g, *((40, 2, 256, 2048) if gated else (40, 256, 2048)))
    check_product(ep, rows8(g, ep, M, 2048), w, s, off, count)
    off, count, M = places([700, 5])
    w, s = weights8(g, *((2, 2, 128, 7168) if gated else (2, 128, 7168)))
    check_product(ep, rows8(g, ep, M, 7168), w, s, off, count)


@pytest.mark.parametrize("gated", [False, True])
def test_product_leaves_other_places_alone(ep, gated):
    g = gen(32)
    off, count, end = places([5, 0, 130], [3, 2, 7])
    M = end + 4
    a = rows8(g, ep, M, 256)
    w, s = weights8(g, *((3, 2, 136, 256) if gated else (3, 136, 256)))
    if gated:
        out = ep.Fp8Rows.empty(M, 136)
        out.packed.zero_()
        out.values.copy_(torch.full((M, 136), 7.0, device="cuda"))
        out.scales.fill_(5.0)
    else:
        out = torch.full((M, 136), 7.0, dtype=BF, device="cuda")
    got = check_product(ep, a, w, s, off, count, out=out)
    assert got is out
    live = torch.zeros(M, dtype=torch.bool, device="cuda")
    for o, n in zip(off.tolist(), count.tolist()):
        live[o:o + n] = True
    if gated:
        assert (out.values[~live].float() == 7).all() and (out.scales[~live] == 5).all()
    else:
        assert (out[~live] == 7).all()


def test_product_strided_rows_and_outputs(ep):
    g = gen(33)
    off, count, M = places([200])
    base = torch.zeros(M, 512, dtype=torch.uint8, device="cuda")
    a = ep.Fp8Rows(base.view(F8)[:, 32:288], torch.rand(M, 9, device="cuda", generator=g)[:, 3:5])
    a.values.copy_(rnd(g, M, 256) * 30)
    w, s = weights8(g, 1, 72, 256)
    out = torch.zeros(M, 200, dtype=BF, device="cuda")
    check_product(ep, a, w, s, off, count, out=out[:, 8:80])
    assert (out[:, :8] == 0).all() and (out[:, 80:] == 0).all()


def test_product_rows_and_places_out_of_range(ep):
    g = gen(34)
    a = rows8(g, ep, 50, 128)
    w, s = weights8(g, 2, 64, 128)
    rows = torch.randint(50, (90,), device="cuda", generator=g, dtype=torch.int32)
    off, count, _ = places([40, 50])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.expert_product(a, w, s, off, count, rows=rows, status=status)
    assert status.item() == 0
    rows[3], rows[60] = -1, 50
    check_product(ep, a, w, s, off, count, rows, status=status)       # such rows count as zeros
    assert status.item() == 1
    status.zero_()
    rows.clamp_(0, 49)
    count[1] = 51                                                     # past the places: the expert is skipped
    check_product(ep, a, w, s, off, count, rows, status=status)
    assert status.item() == 1
    count[1], off[1] = 10, -4
    check_product(ep, a, w, s, off, count, rows)


def test_product_nan_and_infinity_stay_in_their_rows(ep):
    g = gen(35)
    off, count, M = places([9])
    a = rows8(g, ep, M, 256)
    w, s = weights8(g, 1, 64, 256)
    clean = ep.expert_product(a, w, s, off, count)
    a.values.view(torch.uint8)[4, 17] = 0x7F          # NaN
    a.scales[6, 1] = float("inf")
    got = ep.expert_product(a, w, s, off, count)
    assert got[4].isnan().all() and not got[6].isfinite().any()
    rest = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(got[rest], clean[rest])


def test_product_of_nothing(ep):
    g = gen(36)
    w, s = weights8(g, 2, 64, 128)
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert ep.expert_product(ep.Fp8Rows.empty(0, 128), w, s, z, z).shape == (0, 64)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert ep.expert_product(rows8(g, ep, 5, 128), w, s, z, z, rows=none).shape == (0, 64)


# ------------------------------------------------------------- the picks' sum
def receive_view(ep, R_, Tpr, E, K, g, zipf=False, drop=0.0):
    T = R_ * Tpr
    logits = rnd(g, T, E)
    if zipf:
        logits -= 2 * torch.log(torch.arange(1, E + 1, device="cuda"))
    if drop:
        logits[torch.rand(T, E, device="cuda", generator=g) < drop] = R.NEG
    r = ep.route(logits, K, num_ranks=R_)
    layer = ep.EpLayer(R_, Tpr, 64, E, K)
    lay = layer.layout(r.topk_idx)
    xl = layer.expert_layout(r.topk_idx, r.topk_weights, lay)
    assert layer.device_status() == 0
    return layer, r, lay, xl


@pytest.mark.parametrize("R_,Tpr,E,K", [(1, 1, 1, 1), (1, 30, 8, 3), (4, 16, 16, 2), (8, 9, 64, 8), (32, 3, 64, 32),
                                        (64, 2, 64, 5)])
@pytest.mark.parametrize("H", [8, 136, 1024, 2056, 7168])
def test_pick_sum(ep, R_, Tpr, E, K, H):
    g = gen(R_ + Tpr + H)
    layer, r, lay, xl = receive_view(ep, R_, Tpr, E, K, g, zipf=Tpr % 2 == 1, drop=0.5 if Tpr == 16 else 0.0)
    M = int(xl.expert_count.sum())
    y = rnd(g, xl.expert_rows.shape[0], H, dtype=BF)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ep.pick_sum(y, xl.recv_topk_idx, xl.recv_topk_weights, lay.recv_base, lay.expert_off, xl.expert_count,
                      xl.expert_rows, status=status)
    want, S = R.pick_sum(y, xl.recv_topk_idx, xl.recv_topk_weights, lay.recv_base, lay.expert_off, xl.expert_count,
                         xl.expert_rows)
    near(got, want, want.abs() * HALF_BF + S * (K + 1) * U)
    assert status.item() == 0 and M <= y.shape[0]
    layer.close()


def test_pick_sum_skips_what_it_does_not_find(ep):
    g = gen(41)
    layer, r, lay, xl = receive_view(ep, 4, 8, 16, 3, g)
    y = rnd(g, xl.expert_rows.shape[0], 64, dtype=BF)
    args = [xl.recv_topk_weights, lay.recv_base, lay.expert_off, xl.expert_count, xl.expert_rows]
    idx = xl.recv_topk_idx.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    row, k = [int(v) for v in (idx >= 0).nonzero()[5]]
    idx[row, k] = 4                                  # a rank has 4 experts
    got = ep.pick_sum(y, idx, *args, status=status)
    idx[row, k] = -1
    assert status.item() == 1 and torch.equal(got, ep.pick_sum(y, idx, *args))
    idx[:] = -1                                      # rows without picks
    assert (ep.pick_sum(y, idx, *args) == 0).all()
    layer.close()


def test_pick_sum_strided(ep):
    g = gen(42)
    layer, r, lay, xl = receive_view(ep, 4, 8, 16, 3, g)
    wide = rnd(g, xl.expert_rows.shape[0], 200, dtype=BF)
    args = [xl.recv_topk_idx, xl.recv_topk_weights, lay.recv_base, lay.expert_off, xl.expert_count, xl.expert_rows]
    out = torch.zeros(lay.n_recv, 120, dtype=BF, device="cuda")
    ep.pick_sum(wide[:, 8:80], *args, out=out[:, 16:88])
    assert torch.equal(out[:, 16:88], ep.pick_sum(wide[:, 8:80].contiguous(), *args))
    assert (out[:, :16] == 0).all() and (out[:, 88:] == 0).all()
    layer.close()


# ------------------------------------------------------------------- refusals
def test_refusals(ep):
    d = dict(device="cuda")
    x, w = torch.zeros(4, 64, dtype=BF, **d), torch.ones(64, **d)
    rstd = torch.ones(4, **d)
    i32 = torch.zeros(2, dtype=torch.int32, **d)
    a = ep.Fp8Rows(torch.zeros(4, 128, dtype=F8, **d), torch.ones(4, 1, **d))
    m, s = torch.zeros(2, 64, 128, dtype=F8, **d), torch.ones(2, 1, 1, **d)
    logits = torch.zeros(4, 8, **d)
    plain = ep.route(logits, 2)
    bad = [
        (TypeError, lambda: ep.rms_norm(x.float(), w)),
        (TypeError, lambda: ep.rms_norm([1.0], w)),
        (TypeError, lambda: ep.rms_norm(x, w.double())),
        (TypeError, lambda: ep.rms_norm(x, w, fp8=True, out=x)),
        (ValueError, lambda: ep.rms_norm(x.cpu(), w)),
        (ValueError, lambda: ep.rms_norm(x, w.cpu())),
        (ValueError, lambda: ep.rms_norm(x, w[:32])),
        (ValueError, lambda: ep.rms_norm(x[:, :60], w[:60])),
        (ValueError, lambda: ep.rms_norm(x[:, 4:36], w[:32])),
        (ValueError, lambda: ep.rms_norm(x.t().contiguous().t(), w)),
        (ValueError, lambda: ep.rms_norm(x, w, residual=x[:3])),
        (ValueError, lambda: ep.rms_norm(x, w, residual_out=x)),
        (ValueError, lambda: ep.rms_norm(x, w, eps=-1.0)),
        (ValueError, lambda: ep.rms_norm(x, w, eps=float("nan"))),
        (ValueError, lambda: ep.rms_norm_backward(x, x, w, rstd[:3])),
        (TypeError, lambda: ep.rms_norm_backward(x, x.float(), w, rstd)),
        (TypeError, lambda: ep.route(logits.double(), 2)),
        (ValueError, lambda: ep.route(logits, 0)),
        (ValueError, lambda: ep.route(logits, 9)),
        (ValueError, lambda: ep.route(torch.zeros(1, 64, **d), 33)),
        (ValueError, lambda: ep.route(torch.zeros(1, 4097, **d), 2)),
        (ValueError, lambda: ep.route(logits, 2, num_ranks=3)),
        (TypeError, lambda: ep.route(logits, 2, token_mask=torch.ones(4, **d))),
        (ValueError, lambda: ep.route(logits, 2, token_mask=torch.ones(3, dtype=torch.bool, **d))),
        (ValueError, lambda: ep.route_backward(logits, plain, torch.zeros(4, 2, **d))),
        (TypeError, lambda: ep.route_backward(logits, None, torch.zeros(4, 2, **d))),
        (TypeError, lambda: ep.expert_product(m, m, s, i32, i32)),
        (TypeError, lambda: ep.expert_product(a, m.float(), s, i32, i32)),
        (ValueError, lambda: ep.expert_product(a, m[0], s, i32, i32)),
        (ValueError, lambda: ep.expert_product(a, m[:, :, :64], s, i32, i32)),
        (ValueError, lambda: ep.expert_product(a, m, s[:1], i32, i32)),
        (ValueError, lambda: ep.expert_product(a, m, s, i32[:1], i32)),
        (TypeError, lambda: ep.expert_product(a, m, s, i32.long(), i32)),
        (TypeError, lambda: ep.expert_product(a, m, s, i32, i32, out=a)),
        (ValueError, lambda: ep.expert_product(ep.Fp8Rows(a.values[:, :120], a.scales), m[:, :, :120].contiguous(),
                                               s, i32, i32)),
        (TypeError, lambda: ep.pick_sum(x.float(), i32[None], rstd[None, :2], i32, i32, i32, i32)),
        (ValueError, lambda: ep.pick_sum(x, i32[None], rstd[None, :2], i32, i32, i32, i32)),
        (ValueError, lambda: ep.Fp8Rows.empty(4, 100)),
        (ValueError, lambda: ep.Fp8Rows.from_packed(x, 64)),
        (ValueError, lambda: a.packed),
    ]
    for i, (exc, f) in enumerate(bad):
        with pytest.raises(exc):
            f()
            pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()


def test_on_another_stream(ep):
    """Work goes to the current stream: an input made there is not waited for elsewhere."""
    g = gen(51)
    side = torch.cuda.Stream()
    logits, w = rnd(g, 4096, 256), torch.ones(4096, device="cuda")
    x = rnd(g, 4096, 4096, dtype=BF)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            x = x @ x * 0.01                          # keeps the side stream busy
        x = x.clamp(-4, 4)
        n = ep.rms_norm(x, w)
        r = ep.route(logits + x[:, :256].float(), 8)
    side.synchronize()
    y, _, _ = R.norm(x, w)
    near(n.out, y, y.abs() * (HALF_BF + 120 * U))
    assert torch.equal(r.topk_idx.long(), R.route(logits + x[:, :256].float(), 8)["idx"])


def test_in_a_graph(ep):
    """Every call can be captured and replayed on new inputs."""
    g = gen(52)
    x, w, logits = rnd(g, 64, 256, dtype=BF), torch.ones(256, device="cuda"), rnd(g, 64, 16)
    m, s = weights8(g, 2, 2, 128, 256)
    off, count, _ = places([30, 34])

    def step():
        n = ep.rms_norm(x, w, residual=x, fp8=True, save_rstd=True)
        r = ep.route(logits, 2, balance_coef=1.0)
        d = ep.route_backward(logits, r, r.topk_weights, r.balance_loss)
        dx, dw = ep.rms_norm_backward(x, n.residual, w, n.rstd)
        h = ep.expert_product(n.out, m, s, off, count)
        return [n.residual, r.topk_idx, r.balance_loss, d, dx, dw, h.values.float(), h.scales]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.copy_(rnd(g, 64, 256))
    logits.copy_(rnd(g, 64, 16))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, step()):
        assert torch.equal(a, b)


def test_norm_in_8_bits_and_bf16_at_once(ep):
    g = gen(61)
    x, res, w = rnd(g, 40, 520, dtype=BF), rnd(g, 40, 520, dtype=BF), rnd(g, 520)
    both = ep.rms_norm(x, w, residual=res, fp8=True, with_bf16=True)
    eight, plain = ep.rms_norm(x, w, residual=res, fp8=True), ep.rms_norm(x, w, residual=res)
    assert torch.equal(both.bf16, plain.out)
    assert torch.equal(both.out.values.float(), eight.out.values.float())
    assert torch.equal(both.out.scales, eight.out.scales) and plain.bf16 is None
    with pytest.raises(ValueError):
        ep.rms_norm(x, w, with_bf16=True)


def test_packed_rows_travel_as_one_piece(ep):
    """A packed row's bytes are its values, then its scales, on the widths a dispatch takes."""
    g = gen(62)
    for width in (8, 136, 256, 1000, 7168):
        a = ep.Fp8Rows.empty(5, width)
        assert a.packed.shape == (5, ep.Fp8Rows.packed_width(width)) and a.packed.shape[1] % 8 == 0
        a.packed.zero_()
        a.values.copy_(rnd(g, 5, width))
        a.scales.copy_(rnd(g, *a.scales.shape))
        b = ep.Fp8Rows.from_packed(a.packed.clone(), width)
        assert torch.equal(b.values.float(), a.values.float()) and torch.equal(b.scales, a.scales)
        assert torch.equal(b.float(), a.float())


# ------------------------------------------------- rows that lie far apart
def test_norm_offsets_past_32_bits(ep):
    """Rows 2^27 bytes apart: the last ones lie beyond 2^32 bytes."""
    g = gen(71)
    far = torch.empty(36, 1 << 26, dtype=BF, device="cuda")
    x = far[:, :264]
    x.copy_(rnd(g, 36, 264))
    w = rnd(g, 264)
    y, h, r = R.norm(x, w)
    near(ep.rms_norm(x, w).out, y, y.abs() * (HALF_BF + 60 * U))
    n = ep.rms_norm(x.contiguous(), w, out=far[:, 512:776], save_rstd=True)
    assert torch.equal(n.out, ep.rms_norm(x, w).out)
    dx, dw = ep.rms_norm_backward(x, x, w, n.rstd, dx=far[:, 1024:1288])
    dx2, dw2 = ep.rms_norm_backward(x.contiguous(), x.contiguous(), w, n.rstd)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_product_offsets_past_32_bits(ep, gather, gated):
    g = gen(72)
    far = torch.empty(36, 1 << 27, dtype=torch.uint8, device="cuda").view(F8)
    a = ep.Fp8Rows(far[:, :256], far.view(torch.float32)[:, 256:258])
    a.values.copy_(rnd(g, 36, 256) * 50)
    a.scales.copy_(torch.rand(36, 2, device="cuda", generator=g))
    w, s = weights8(g, *((2, 2, 72, 256) if gated else (2, 72, 256)))
    off, count, M = places([17, 19])
    rows = torch.arange(35, -1, -1, dtype=torch.int32, device="cuda") if gather else None
    out = ep.Fp8Rows(far[:, 4096:4168], far.view(torch.float32)[:, 2048:2049]) if gated else \
        far.view(BF)[:, 4096:4168]
    check_product(ep, a, w, s, off, count, rows, out=out)


def test_pick_sum_and_route_offsets_past_32_bits(ep):
    g = gen(73)
    far = torch.empty(48, 1 << 26, dtype=BF, device="cuda")
    layer, r, lay, xl = receive_view(ep, 2, 8, 8, 3, g)
    y = far[:, :72]
    y.copy_(rnd(g, 48, 72))
    args = [xl.recv_topk_idx, xl.recv_topk_weights, lay.recv_base, lay.expert_off, xl.expert_count, xl.expert_rows]
    out = far[:lay.n_recv, 128:200]
    ep.pick_sum(y, *args, out=out)
    assert torch.equal(out, ep.pick_sum(y.contiguous(), *args))
    layer.close()
    logits = far.view(torch.float32)[:, 1024:1040]
    logits.copy_(rnd(g, 48, 16))
    got, _ = check_route(ep, logits, 3, True, None, 1.0)
    dw = rnd(g, 48, 3)
    into = far.view(torch.float32)[:, 2048:2064]
    assert torch.equal(ep.route_backward(logits, got, dw, dlogits=into), ep.route_backward(logits.contiguous(), got, dw))


def test_product_at_an_odd_address_of_scales_and_rows(ep):
    """Scales that start anywhere on 4 bytes, values on 16, outputs on 8 or 16."""
    g = gen(74)
    for K in (128, 640, 656):
        kb = -(-K // 128)
        base = torch.zeros(70, K + 48, dtype=torch.uint8, device="cuda")
        a = ep.Fp8Rows(base.view(F8)[:, 16:16 + K], torch.rand(70, kb + 3, device="cuda", generator=g)[:, 1:1 + kb])
        a.values.copy_(rnd(g, 70, K) * 30)
        off, count, M = places([30, 40])
        w, s = weights8(g, 2, 2, 136, K)
        buf = torch.zeros(70, 160, dtype=torch.uint8, device="cuda")
        out = ep.Fp8Rows(buf.view(F8)[:, 8:144], torch.zeros(70, 5, device="cuda")[:, 1:3])
        check_product(ep, a, w, s, off, count, out=out)
        assert (buf[:, :8] == 0).all() and (buf[:, 144:] == 0).all()
        w, s = weights8(g, 2, 136, K)
        wide = torch.zeros(70, 168, dtype=BF, device="cuda")
        check_product(ep, a, w, s, off, count, out=wide[:, 8:144])
        assert (wide[:, :8] == 0).all() and (wide[:, 144:] == 0).all()


def test_route_backward_leaves_padded_tokens_zero_whatever_the_loss(ep):
    g = gen(81)
    logits = rnd(g, 40, 64)
    mask = torch.arange(40, device="cuda") % 4 != 0
    logits[5] = R.NEG
    for renorm in (True, False):
        r = ep.route(logits, 4, renormalize=renorm, token_mask=mask, balance_coef=1.0)
        d = ep.route_backward(logits, r, torch.full((40, 4), float("nan"), device="cuda"),
                              torch.tensor(float("nan"), device="cuda"))
        assert (d[~mask] == 0).all() and (d[5] == 0).all()
        assert d[mask].isnan().any(1).sum() == mask.sum() - 1


@pytest.mark.parametrize("E,N,K,M", [(4096, 8, 16, 5000), (700, 72, 144, 300), (1, 8, 65536, 3), (1, 65536, 16, 5),
                                     (3, 16, 16384, 400)])
@pytest.mark.parametrize("gated", [False, True])
def test_product_at_its_largest_sizes(ep, E, N, K, M, gated):
    g = gen(E + N)
    count = torch.bincount(torch.randint(E, (M,), device="cuda", generator=g), minlength=E)
    off = count.cumsum(0) - count
    w, s = weights8(g, *((E, 2, N, K) if gated else (E, N, K)))
    check_product(ep, rows8(g, ep, M, K), w, s, off.int(), count.int())


@pytest.mark.parametrize("gated", [False, True])
def test_product_of_rows_that_are_not_there(ep, gated):
    """Without any row to read every place is zeros, and said so."""
    g = gen(83)
    w, s = weights8(g, *((2, 2, 64, 128) if gated else (2, 64, 128)))
    off, count, M = places([30, 4])
    rows = torch.zeros(M, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ep.expert_product(ep.Fp8Rows.empty(0, 128), w, s, off, count, rows=rows, status=status)
    assert status.item() == 1 and ((y.values.float() if gated else y) == 0).all()
    status.zero_()
    ep.expert_product(ep.Fp8Rows.empty(0, 128), w, s, off, torch.zeros_like(count), rows=rows, status=status)
    assert status.item() == 0


def test_pick_sum_with_long_segments(ep):
    """A rank's only expert lists every row: the search takes several rounds and ends on any of them."""
    g = gen(84)
    for T in (31, 32, 33, 1023, 1025, 40000):
        layer, r, lay, xl = receive_view(ep, 1, T, 2, 2, g)
        y = rnd(g, xl.expert_rows.shape[0], 8, dtype=BF)
        got = ep.pick_sum(y, xl.recv_topk_idx, xl.recv_topk_weights, lay.recv_base, lay.expert_off, xl.expert_count,
                          xl.expert_rows)
        # both experts list every row in order
        w = xl.recv_topk_weights.double()
        at = xl.recv_topk_idx.long() * T + torch.arange(T, device="cuda")[:, None]
        want = (w[..., None] * y[at].double()).sum(1)
        near(got, want, want.abs() * HALF_BF + (w[..., None] * y[at].double()).abs().sum(1) * 3 * U)
        layer.close()


@pytest.mark.parametrize("E,K", [(E, K) for E in (12, 60, 64, 68, 100, 250, 256, 260, 512, 1000, 1028, 4096)
                                 for K in (1, 6, 7, 12, 13, 24, 25, 32) if K <= E])
def test_route_at_the_bounds_of_its_forms(ep, E, K):
    """Odd tokens hold few values, so that their lists of candidates run over while their neighbours' do not."""
    g = gen(E * 33 + K)
    logits = rnd(g, 75, E) * 3
    logits[1::4] = torch.randint(0, 3, (19, E), device="cuda", generator=g).float()
    logits[3::8] = 0.5
    logits[7::8, K // 2:] = R.NEG
    for x in (logits, logits.to(BF), logits[:2], logits[1:2]):
        got, want = check_route(ep, x, K, True, None, 0.5)
        d = ep.route_backward(x, got, torch.ones(x.shape[0], K, device="cuda"))
        assert torch.isfinite(d).all() and d.shape == x.shape
        assert torch.equal(ep.route(x, K).topk_idx, got.topk_idx)
