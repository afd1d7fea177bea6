"""Torch-facing operators around one layer's dispatch and combine: marshalling
of the C ABI in include/ep_ops.h, whose kernels do all the arithmetic.

A layer step with 8-bit rows, in the order of use:

    n = rms_norm(x, weight, residual=res, fp8=True)        # 8-bit rows, new residual stream
    r = route(logits, K, num_ranks=R)                      # picks and weights
    lay = layer.layout(r.topk_idx)                         # layer: EpLayer(hidden=Fp8Rows.packed_width(H))
    recv = layer.dispatch(n.out.packed, lay)               # values and scales travel as one row
    xl = layer.expert_layout(r.topk_idx, r.topk_weights, lay)
    h = expert_product(Fp8Rows.from_packed(recv, H), w13, s13, lay.expert_off, xl.expert_count, rows=xl.expert_rows)
    y = expert_product(h, w2, s2, lay.expert_off, xl.expert_count)
    z = pick_sum(y, xl.recv_topk_idx, xl.recv_topk_weights, lay.recv_base, lay.expert_off, xl.expert_count,
                 xl.expert_rows)
    out = layer2.combine(z, r.rank_weights, r.topk_idx, lay)

Every call enqueues on the current stream of its tensors' device and returns
without waiting; nothing is kept between calls.  A tensor of the wrong type
raises TypeError, of the wrong device, shape or strides ValueError."""
from __future__ import annotations

import dataclasses

import torch

from . import _ep

BLOCK = 128      # columns that share a scale

_DTYPES = {torch.float32: _ep.EP_DTYPE_F32, torch.bfloat16: _ep.EP_DTYPE_BF16}
_BF16, _F32, _I32, _FP8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


@dataclasses.dataclass
class Fp8Rows:
    """8-bit rows: `values` float8_e4m3fn [rows, width] and `scales` fp32
    [rows, ceil(width / 128)]; a value stands for value * scale of its block.
    Columns are dense, rows may be strided.  Rows made by empty() lie in one
    buffer each (the values, then the scales, padded to 16 bytes), so that
    `packed` -- the same memory as bf16 -- can be dispatched."""
    values: torch.Tensor
    scales: torch.Tensor

    @staticmethod
    def packed_width(width: int) -> int:
        """bf16 elements of a packed row: the `hidden` of the EpLayer that dispatches such rows."""
        return (_scales_at(width) + 4 * _blocks(width) + 15) // 16 * 8

    @classmethod
    def empty(cls, rows: int, width: int, device=None) -> "Fp8Rows":
        if width < 8 or width % 8:
            raise ValueError(f"width: {width}, expected a multiple of 8")
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        return cls.from_packed(torch.empty((rows, cls.packed_width(width)), dtype=_BF16, device=device), width)

    @classmethod
    def from_packed(cls, rows: torch.Tensor, width: int) -> "Fp8Rows":
        """The 8-bit rows inside a buffer of packed rows (a dispatch's recv)."""
        if not isinstance(rows, torch.Tensor):
            raise TypeError(f"rows: expected a torch.Tensor, got {type(rows).__name__}")
        if rows.dtype != _BF16:
            raise TypeError(f"rows: dtype {rows.dtype}, expected {_BF16}")
        if rows.dim() != 2 or rows.shape[1] != cls.packed_width(width) or not rows.is_contiguous():
            raise ValueError(f"rows: expected contiguous [*, {cls.packed_width(width)}], got {tuple(rows.shape)}")
        at = _scales_at(width)
        self = cls(rows.view(_FP8)[:, :width], rows.view(_F32)[:, at // 4:at // 4 + _blocks(width)])
        self._packed = rows
        return self

    @property
    def packed(self) -> torch.Tensor:
        rows = getattr(self, "_packed", None)
        if rows is None:
            raise ValueError("these rows do not lie in packed form (use Fp8Rows.empty or from_packed)")
        return rows

    def float(self) -> torch.Tensor:
        """What the rows stand for, in fp32 (for inspection; no kernel of this library)."""
        return self.values.float() * self.scales.repeat_interleave(BLOCK, 1)[:, :self.values.shape[1]]


def _scales_at(width: int) -> int:
    return (width + 3) // 4 * 4


@dataclasses.dataclass
class Normed:
    """rms_norm's outputs: out is a bf16 tensor or Fp8Rows; residual is the new
    residual stream (None without one); rstd fp32 [tokens] where asked for."""
    out: torch.Tensor | Fp8Rows
    residual: torch.Tensor | None
    rstd: torch.Tensor | None


@dataclasses.dataclass
class Routing:
    """route's outputs.  The fields after rank_weights are None unless the
    balance loss was asked for; lse and slope are kept for the backward pass."""
    topk_idx: torch.Tensor
    topk_weights: torch.Tensor
    rank_weights: torch.Tensor | None
    expert_count: torch.Tensor | None
    balance_loss: torch.Tensor | None
    lse: torch.Tensor | None
    slope: torch.Tensor | None
    renormalize: bool


def _check(t, name: str, dtype, device, shape) -> None:
    """Raise unless t is a tensor of `dtype` (one of them, if a tuple) and
    `shape` (None matches any size) on `device`, with dense columns."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    got = t.shape
    if len(got) != len(shape) or any(w is not None and g != w for g, w in zip(got, shape)):
        raise ValueError(f"{name}: shape {tuple(got)}, expected {tuple('*' if v is None else v for v in shape)}")


def _dense(t, name: str, dtype, device, shape) -> int:
    """_check of a contiguous tensor; its address."""
    _check(t, name, dtype, device, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _rows(t, name: str, dtype, device, shape, align: int) -> tuple[int, int]:
    """_check of a matrix whose columns are dense and whose rows start on
    multiples of `align` bytes; its address and row stride in elements."""
    _check(t, name, dtype, device, shape)
    n, width = t.shape
    stride = t.stride(0) if n > 1 else max(width, t.stride(0))
    size, ptr = t.element_size(), t.data_ptr()
    if n == 0:
        return ptr, -(-width * size // align) * align // size
    if n == 1 and stride * size % align:      # a single row's stride is never used
        stride = -(-width * size // align) * align // size
    if (width > 1 and t.stride(1) != 1) or stride < width:
        raise ValueError(f"{name}: strides {tuple(t.stride())}, expected dense columns in rows that do not overlap")
    if stride * size % align or ptr % align:
        raise ValueError(f"{name}: rows must start on multiples of {align} bytes "
                         f"(address {ptr:#x}, row stride {stride * size} bytes)")
    return ptr, stride


def _device_of(t, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{name}: on {t.device}, expected a CUDA device")
    return t.device


def _call(device: torch.device, fn, *args) -> None:
    """fn(*args, stream) on the current stream of `device`, made current for the call."""
    stream = torch.cuda.current_stream(device).cuda_stream
    if torch.cuda.current_device() == device.index:
        fn(*args, stream)
    else:
        with torch.cuda.device(device):
            fn(*args, stream)


def _check_hidden(h: int) -> None:
    if h < 8 or h % 8 or h > 32768:
        raise ValueError(f"hidden: {h}, expected a multiple of 8 up to 32768")


# ------------------------------------------------------------------ the norm

def rms_norm(x: torch.Tensor, weight: torch.Tensor, *, residual: torch.Tensor | None = None, eps: float = 1e-6,
             fp8: bool = False, save_rstd: bool = False, out: torch.Tensor | Fp8Rows | None = None,
             residual_out: torch.Tensor | None = None) -> Normed:
    """ep_rms_norm: h = x + residual, out = h / sqrt(mean(h^2) + eps) * weight.
    x, residual: bf16 [T, H]; weight: bf16 or fp32 [H].  With fp8 the output is
    Fp8Rows (packed, unless `out` gives other ones).  residual_out may be
    residual itself; without a residual no stream is returned.  save_rstd
    keeps what rms_norm_backward needs."""
    dev = _device_of(x, "x")
    _check(x, "x", _BF16, dev, (None, None))
    T, H = x.shape
    _check_hidden(H)
    if not eps >= 0:
        raise ValueError(f"eps: {eps}, expected at least 0")
    px, sx = _rows(x, "x", _BF16, dev, (T, H), 16)
    pr = sr = po = so = pv = sv = ps = ss = ph = sh = pd = 0
    if residual is not None:
        pr, sr = _rows(residual, "residual", _BF16, dev, (T, H), 16)
        if residual_out is None:
            residual_out = torch.empty((T, H), dtype=_BF16, device=dev)
        ph, sh = _rows(residual_out, "residual_out", _BF16, dev, (T, H), 16)
    elif residual_out is not None:
        raise ValueError("residual_out: there is no residual")
    pw = _dense(weight, "weight", (_BF16, _F32), dev, (H,))
    if pw % 16:
        raise ValueError("weight: must start on a multiple of 16 bytes")
    if fp8:
        if out is None:
            out = Fp8Rows.empty(T, H, dev)
        pv, sv, ps, ss = _fp8_rows(out, "out", dev, (T, H), 8)
    else:
        if out is None:
            out = torch.empty((T, H), dtype=_BF16, device=dev)
        po, so = _rows(out, "out", _BF16, dev, (T, H), 16)
    rstd = None
    if save_rstd:
        rstd = torch.empty((T,), dtype=_F32, device=dev)
        pd = rstd.data_ptr()
    if T:
        _call(dev, _ep.ep_rms_norm, T, H, px, sx, pr, sr, pw, _DTYPES[weight.dtype], eps, po, so, pv, sv, ps, ss,
              ph, sh, pd)
    return Normed(out, residual_out, rstd)


def rms_norm_backward(dout: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *,
                      dresidual: torch.Tensor | None = None,
                      dx: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """ep_rms_norm_backward: (dx, dweight) from the output's gradient, the
    residual stream h that rms_norm stored (x itself without a residual) and
    its rstd.  dresidual: the gradient that reaches h directly.  dx, bf16
    [T, H], is the gradient of x and of residual alike and may be given as
    dout or dresidual; dweight is fp32 [H]."""
    dev = _device_of(dout, "dout")
    _check(dout, "dout", _BF16, dev, (None, None))
    T, H = dout.shape
    _check_hidden(H)
    pg, sg = _rows(dout, "dout", _BF16, dev, (T, H), 16)
    ph, sh = _rows(h, "h", _BF16, dev, (T, H), 16)
    pw = _dense(weight, "weight", (_BF16, _F32), dev, (H,))
    if pw % 16:
        raise ValueError("weight: must start on a multiple of 16 bytes")
    pd = _dense(rstd, "rstd", _F32, dev, (T,))
    pr = sr = 0
    if dresidual is not None:
        pr, sr = _rows(dresidual, "dresidual", _BF16, dev, (T, H), 16)
    if dx is None:
        dx = torch.empty((T, H), dtype=_BF16, device=dev)
    px, sx = _rows(dx, "dx", _BF16, dev, (T, H), 16)
    dweight = torch.empty((H,), dtype=_F32, device=dev)
    size = _ep.ep_rms_norm_backward_workspace(T, H)
    work = torch.empty((size,), dtype=torch.uint8, device=dev)
    _call(dev, _ep.ep_rms_norm_backward, T, H, pg, sg, ph, sh, pw, _DTYPES[weight.dtype], pd, pr, sr, px, sx,
          dweight.data_ptr(), work.data_ptr(), size)
    return dx, dweight


def _fp8_rows(r, name: str, dev, shape, align: int) -> tuple[int, int, int, int]:
    if not isinstance(r, Fp8Rows):
        raise TypeError(f"{name}: expected Fp8Rows, got {type(r).__name__}")
    pv, sv = _rows(r.values, name + ".values", _FP8, dev, shape, align)
    ps, ss = _rows(r.scales, name + ".scales", _F32, dev, (r.values.shape[0], _blocks(r.values.shape[1])), 4)
    return pv, sv, ps, ss


# ---------------------------------------------------------------- the router

def route(logits: torch.Tensor, topk: int, *, renormalize: bool = True, token_mask: torch.Tensor | None = None,
          balance_coef: float | None = None, num_ranks: int | None = None) -> Routing:
    """ep_route: the topk largest of each token's logits [T, E] (fp32 or bf16)
    and their softmax weights; ties go to the lower expert, -inf and NaN are
    never picked (-1 and weight 0 where fewer are left).  token_mask: bool [T],
    False for padded tokens.  With balance_coef also the picks' counts per
    expert and the balance loss, and what route_backward needs.  With num_ranks
    also the weights with which EpLayer.combine adds the rows of pick_sum."""
    dev = _device_of(logits, "logits")
    _check(logits, "logits", (_F32, _BF16), dev, (None, None))
    T, E = logits.shape
    if not 1 <= E <= 4096:
        raise ValueError(f"logits: {E} experts, expected 1 to 4096")
    if not 1 <= topk <= min(32, E):
        raise ValueError(f"topk: {topk}, expected 1 to {min(32, E)}")
    if num_ranks is not None and (num_ranks < 1 or E % num_ranks):
        raise ValueError(f"num_ranks: {num_ranks} does not divide {E} experts")
    pl, sl = _rows(logits, "logits", (_F32, _BF16), dev, (T, E), logits.element_size())
    pm = 0 if token_mask is None else _dense(token_mask, "token_mask", torch.bool, dev, (T,))
    idx = torch.empty((T, topk), dtype=_I32, device=dev)
    weights = torch.empty((T, topk), dtype=_F32, device=dev)
    ranked = None if num_ranks is None else torch.empty((T, topk), dtype=_F32, device=dev)
    count = loss = slope = lse = None
    train = ()
    if balance_coef is not None:
        count = torch.empty((E,), dtype=_I32, device=dev)
        loss = torch.empty((), dtype=_F32, device=dev)
        slope = torch.empty((E,), dtype=_F32, device=dev)
        lse = torch.empty((T,), dtype=_F32, device=dev)
        size = _ep.ep_route_workspace(T, E)
        work = torch.empty((size,), dtype=torch.uint8, device=dev)
        train = (balance_coef, lse.data_ptr(), count.data_ptr(), loss.data_ptr(), slope.data_ptr(), work.data_ptr(),
                 size)
    if T or train:
        _call(dev, _ep.ep_route, T, E, topk, pl, _DTYPES[logits.dtype], sl, pm, 1 if renormalize else 0,
              idx.data_ptr(), weights.data_ptr(), num_ranks or 0, ranked.data_ptr() if ranked is not None else 0,
              *(train or (0.0, 0, 0, 0, 0, 0, 0)))
    return Routing(idx, weights, ranked, count, loss, lse, slope, bool(renormalize))


def route_backward(logits: torch.Tensor, routing: Routing, dweights: torch.Tensor,
                   dloss: torch.Tensor | None = None, *, dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """ep_route_backward: the logits' gradient from those of the picks' weights
    (fp32 [T, K]) and of the balance loss (an fp32 scalar on the device; None:
    the loss was not used).  dlogits may be given as the logits."""
    dev = _device_of(logits, "logits")
    if not isinstance(routing, Routing):
        raise TypeError(f"routing: expected a Routing, got {type(routing).__name__}")
    if routing.lse is None:
        raise ValueError("routing: made without balance_coef, it does not hold what the backward pass needs")
    _check(logits, "logits", (_F32, _BF16), dev, (None, None))
    T, E = logits.shape
    pl, sl = _rows(logits, "logits", (_F32, _BF16), dev, (T, E), logits.element_size())
    K = routing.topk_idx.shape[1]
    if dlogits is None:
        dlogits = torch.empty((T, E), dtype=logits.dtype, device=dev)
    pd, sd = _rows(dlogits, "dlogits", logits.dtype, dev, (T, E), logits.element_size())
    args = (_dense(routing.topk_idx, "routing.topk_idx", _I32, dev, (T, K)),
            _dense(routing.topk_weights, "routing.topk_weights", _F32, dev, (T, K)),
            _dense(routing.lse, "routing.lse", _F32, dev, (T,)),
            _dense(routing.slope, "routing.slope", _F32, dev, (E,)),
            _dense(dweights, "dweights", _F32, dev, (T, K)),
            0 if dloss is None else _dense(dloss, "dloss", _F32, dev, ()))
    if T:
        _call(dev, _ep.ep_route_backward, T, E, K, pl, _DTYPES[logits.dtype], sl, 1 if routing.renormalize else 0,
              *args, pd, sd)
    return dlogits


# -------------------------------------------------------------- the experts

def expert_product(a: Fp8Rows, w: torch.Tensor, w_scales: torch.Tensor, expert_off: torch.Tensor,
                   expert_count: torch.Tensor, *, rows: torch.Tensor | None = None,
                   out: torch.Tensor | Fp8Rows | None = None,
                   status: torch.Tensor | None = None) -> torch.Tensor | Fp8Rows:
    """ep_expert_product over expert-major places: expert e's are
    expert_off[e] .. + expert_count[e], place p's row is a[rows[p]], or a[p]
    without rows.
    w float8_e4m3fn [E, N, K]: a @ w[e].T, bf16 [places, N].
    w [E, 2, N, K] (gate, up): silu(a @ gate.T) * (a @ up.T) as Fp8Rows.
    w_scales fp32 [E(, 2), ceil(N / 128), ceil(K / 128)].
    Places that no expert holds are left as they are.  status: int32 [1] on the
    device, set to EP_ERR_INVALID_ARG where a place or row is out of range."""
    if not isinstance(a, Fp8Rows):
        raise TypeError(f"a: expected Fp8Rows, got {type(a).__name__}")
    dev = _device_of(a.values, "a.values")
    pa, sa, ps, ss = _fp8_rows(a, "a", dev, (None, None), 16)
    A, K = a.values.shape
    if not isinstance(w, torch.Tensor):
        raise TypeError(f"w: expected a torch.Tensor, got {type(w).__name__}")
    gated = w.dim() == 4
    if not gated and w.dim() != 3:
        raise ValueError(f"w: shape {tuple(w.shape)}, expected [E, N, K] or [E, 2, N, K]")
    E, N = w.shape[0], w.shape[-2]
    if K < 16 or K % 16 or K > 65536:
        raise ValueError(f"a: {K} columns, expected a multiple of 16 up to 65536")
    if N < 8 or N % 8 or N > 65536:
        raise ValueError(f"w: {N} rows, expected a multiple of 8 up to 65536")
    if not 1 <= E <= 4096:
        raise ValueError(f"w: {E} experts, expected 1 to 4096")
    pair = (2,) if gated else ()
    pw = _dense(w, "w", _FP8, dev, (E, *pair, N, K))
    if pw % 16:
        raise ValueError("w: must start on a multiple of 16 bytes")
    pws = _dense(w_scales, "w_scales", _F32, dev, (E, *pair, _blocks(N), _blocks(K)))
    off = _dense(expert_off, "expert_off", _I32, dev, (E,))
    count = _dense(expert_count, "expert_count", _I32, dev, (E,))
    places, pr = A, 0
    if rows is not None:
        pr = _dense(rows, "rows", _I32, dev, (None,))
        places = rows.shape[0]
    st = 0 if status is None else _dense(status, "status", _I32, dev, (1,))
    po = so = pv = sv = pos = sos = 0
    if gated:
        if out is None:
            out = Fp8Rows.empty(places, N, dev)
        pv, sv, pos, sos = _fp8_rows(out, "out", dev, (places, N), 8)
    else:
        if out is None:
            out = torch.empty((places, N), dtype=_BF16, device=dev)
        po, so = _rows(out, "out", _BF16, dev, (places, N), 16)
    if places:
        _call(dev, _ep.ep_expert_product, places, A, E, K, N, 1 if gated else 0, pa, sa, ps, ss, pw, pws, off, count,
              pr, po, so, pv, sv, pos, sos, st)
    return out


def pick_sum(y: torch.Tensor, recv_topk_idx: torch.Tensor, recv_topk_weights: torch.Tensor, recv_base: torch.Tensor,
             expert_off: torch.Tensor, expert_count: torch.Tensor, expert_rows: torch.Tensor, *,
             out: torch.Tensor | None = None, status: torch.Tensor | None = None) -> torch.Tensor:
    """ep_pick_sum: for each receive row the sum of its picks' rows of y (bf16
    [places, H], the experts' output) times their weights -- the expert_out of
    EpLayer.combine, taken with route's rank_weights.  The other arguments are
    fields of the Layout (recv_base, expert_off) and the ExpertLayout.
    status as in expert_product, for picks whose place is not found."""
    dev = _device_of(y, "y")
    _check(y, "y", _BF16, dev, (None, None))
    M, H = y.shape
    if H < 8 or H % 8:
        raise ValueError(f"y: {H} columns, expected a multiple of 8")
    py, sy = _rows(y, "y", _BF16, dev, (M, H), 16)
    pi = _dense(recv_topk_idx, "recv_topk_idx", _I32, dev, (None, None))
    N, K = recv_topk_idx.shape
    pw = _dense(recv_topk_weights, "recv_topk_weights", _F32, dev, (N, K))
    pb = _dense(recv_base, "recv_base", _I32, dev, (None,))
    po = _dense(expert_off, "expert_off", _I32, dev, (None,))
    R, E = recv_base.shape[0], expert_off.shape[0]
    if not 1 <= K <= 32:
        raise ValueError(f"recv_topk_idx: {K} picks, expected 1 to 32")
    if not 1 <= R <= 64 or E < R or E % R or E > 4096:
        raise ValueError(f"recv_base, expert_off: {R} ranks do not divide {E} experts")
    pc = _dense(expert_count, "expert_count", _I32, dev, (E,))
    pe = _dense(expert_rows, "expert_rows", _I32, dev, (M,))
    st = 0 if status is None else _dense(status, "status", _I32, dev, (1,))
    if out is None:
        out = torch.empty((N, H), dtype=_BF16, device=dev)
    pz, sz = _rows(out, "out", _BF16, dev, (N, H), 16)
    if N:
        _call(dev, _ep.ep_pick_sum, N, M, H, K, R, E, py, sy, pi, pw, pb, po, pc, pe, pz, sz, st)
    return out
