"""Plain 64-bit forms of the operators in include/ep_ops.h, from their
formulas, for any device.  Masked or empty rows are handled by selection, not
by arithmetic, so that what stands in them cannot matter."""
import torch

BLOCK = 128
NEG = float("-inf")


def norm(x, weight, residual=None, eps=1e-6):
    """(y, h, r) of h = x + residual, r = 1 / sqrt(mean(h^2) + eps), y = h r weight."""
    h = x.double() + (0 if residual is None else residual.double())
    r = (h.square().mean(-1) + eps).rsqrt()
    return h * r[:, None] * weight.double(), h, r


def norm_grad(dout, h, weight, r, dresidual=None):
    """(dx, dweight) by the formula."""
    g, u = dout.double(), h.double() * r.double()[:, None]
    du = g * weight.double()
    dx = r.double()[:, None] * (du - u * (du * u).mean(-1, keepdim=True))
    return dx + (0 if dresidual is None else dresidual.double()), (g * u).sum(0)


def block_max(y):
    """Largest magnitude of each block of 128 columns, NaN kept."""
    parts = [y[:, c:c + BLOCK].abs().amax(1) for c in range(0, y.shape[1], BLOCK)]
    return torch.stack(parts, 1)


def spread(s, width):
    return s.repeat_interleave(BLOCK, -1)[..., :width]


def route(logits, topk, renormalize=True, mask=None, coef=None):
    """dict of idx, weights, p, lse, count, loss, slope."""
    x = logits.double().clone()
    T, E = x.shape
    live = torch.ones(T, dtype=torch.bool, device=x.device) if mask is None else mask
    x[~live] = NEG
    key = torch.where(x > NEG, x, NEG)          # NaN is not picked
    idx = torch.full((T, topk), -1, dtype=torch.int64, device=x.device)
    left = key.clone()
    rows = torch.arange(T, device=x.device)
    for k in range(topk):
        best = left.amax(1)
        at = (left == best[:, None]).int().argmax(1)          # the first of equals
        ok = best > NEG
        idx[ok, k] = at[ok]
        left[rows[ok], at[ok]] = NEG
    lse = torch.logsumexp(x, 1)
    p = torch.where((x > NEG) | x.isnan(), (x - lse[:, None]).exp(), 0.0)
    p = torch.where(((x > NEG) | x.isnan()).any(1)[:, None] & lse.isnan()[:, None], float("nan"), p)
    got = idx >= 0
    picked = x.gather(1, idx.clamp_min(0))
    if renormalize:
        w = torch.where(got, picked, NEG)
        w = torch.where(got, torch.softmax(w, 1), 0.0)
    else:
        w = torch.where(got, p.gather(1, idx.clamp_min(0)), 0.0)
    out = dict(idx=idx, weights=w, p=p, lse=torch.where(live, lse, float("inf")))
    if coef is not None:
        tv = max(1, int(live.sum()))
        out["count"] = torch.bincount(idx[got], minlength=E)
        out["slope"] = coef * E / (topk * tv * tv) * out["count"].double()
        out["loss"] = (out["slope"] * p.sum(0)).sum()
    return out


def route_grad(r, renormalize, dweights, dloss):
    """d logits for route()'s dict, by the formula."""
    p, idx = r["p"], r["idx"]
    got, at = idx >= 0, idx.clamp_min(0)
    dw = torch.where(got, dweights.double(), 0.0)
    g = (r["slope"] * dloss).expand_as(p)
    if renormalize:
        w = r["weights"]
        return p * (g - (p * g).sum(1, keepdim=True)) + torch.zeros_like(p).scatter_add_(
            1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
    g = g.scatter_add(1, at, dw)
    return p * (g - (p * g).sum(1, keepdim=True))


def product(values, scales, w, w_scales, off, count, rows=None):
    """(y, S) [places, (2,) N]: the products, and the sums of the terms'
    magnitudes; NaN at places that no expert holds, zeros for rows out of range."""
    a = values.double() * spread(scales.double(), values.shape[1])
    E, N, K = w.shape[0], w.shape[-2], w.shape[-1]
    m = w.double() * spread(spread(w_scales.double(), K).transpose(-1, -2), N).transpose(-1, -2)
    places = values.shape[0] if rows is None else rows.shape[0]
    if rows is not None:
        ok = (rows >= 0) & (rows < a.shape[0])
        a = torch.where(ok[:, None], a[rows.long().clamp(0, max(0, a.shape[0] - 1))], 0.0)
    shape = (places, *w.shape[1:-1])
    y = torch.full(shape, float("nan"), dtype=torch.float64, device=values.device)
    S = y.clone()
    for e, (o, n) in enumerate(zip(off.tolist(), count.tolist())):
        if n > 0 and o >= 0 and o + n <= places:
            part = a[o:o + n]
            y[o:o + n] = torch.einsum("mk,...nk->m...n", part, m[e])
            S[o:o + n] = torch.einsum("mk,...nk->m...n", part.abs(), m[e].abs())
    return y, S


def pick_sum(y, recv_topk_idx, recv_topk_weights, recv_base, off, count, expert_rows):
    """(out, S): the sums and the sums of the terms' magnitudes, row by row."""
    N, K = recv_topk_idx.shape
    per = off.shape[0] // recv_base.shape[0]
    out = torch.zeros(N, y.shape[1], dtype=torch.float64, device=y.device)
    S = out.clone()
    base, o, c = recv_base.tolist(), off.tolist(), count.tolist()
    where = {}
    er = expert_rows.tolist()
    for e in range(len(o)):
        for p in range(o[e], o[e] + c[e]):
            where[(e, er[p])] = p
    idx, w = recv_topk_idx.tolist(), recv_topk_weights.double().tolist()
    for r in range(N):
        d = max(i for i, b in enumerate(base) if b <= r)
        for k in range(K):
            if idx[r][k] >= 0:
                row = y[where[(d * per + idx[r][k], r)]].double()
                out[r] += w[r][k] * row
                S[r] += abs(w[r][k]) * row.abs()
    return out, S
