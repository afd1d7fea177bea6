"""The operators' host side without a GPU: sizes and addresses that are refused
before any device call, workspace sizes, and packed rows' geometry."""
import pytest


@pytest.fixture(scope="module")
def ep():
    from combine_ep_layout_04_gb300 import build
    build.build()
    from combine_ep_layout_04_gb300 import _ep
    return _ep


BAD = 1    # EP_ERR_INVALID_ARG


@pytest.mark.parametrize("tokens,hidden,wtype,eps", [(-1, 64, 0, 1e-6), (1, 7, 0, 1e-6), (1, 0, 0, 1e-6),
                                                     (1, 32776, 0, 1e-6), (1, 64, 2, 1e-6), (1, 64, 0, -1.0),
                                                     (1, 64, 0, float("nan")), (1 << 31, 64, 0, 1e-6)])
def test_norm_sizes(ep, tokens, hidden, wtype, eps):
    assert ep.lib.ep_rms_norm(tokens, hidden, 256, 64, None, 0, 256, wtype, eps, 256, 64, None, 0, None, 0, None, 0, None,
                              None) == BAD


def test_norm_addresses(ep):
    def call(x=256, xs=64, w=256, out=256, os=64, v=None, vs=0, s=None, ss=0):
        return ep.lib.ep_rms_norm(4, 64, x, xs, None, 0, w, 0, 1e-6, out, os, v, vs, s, ss, None, 0, None, None)
    assert call(x=None) == call(w=None) == call(out=None) == BAD                  # missing
    assert call(x=264) == call(w=260) == call(out=258) == BAD                     # not on 16 bytes
    assert call(xs=63) == call(xs=68) == call(xs=56) == call(os=60) == BAD        # strides
    assert call(v=256, vs=64) == call(v=260, vs=64, s=256, ss=1) == BAD           # scales missing, values not on 8
    assert call(v=256, vs=60, s=256, ss=1) == call(v=256, vs=64, s=256, ss=0) == BAD
    assert ep.lib.ep_rms_norm(0, 64, None, 0, None, 0, None, 0, 1e-6, None, 0, None, 0, None, 0, None, 0, None,
                              None) == ep.EP_OK                                   # nothing to do


def test_norm_backward_workspace(ep):
    assert ep.ep_rms_norm_backward_workspace(0, 64) == 0
    assert ep.ep_rms_norm_backward_workspace(-1, 64) == ep.ep_rms_norm_backward_workspace(4, 63) == 0
    for tokens, hidden in ((1, 8), (5, 2048), (100000, 7168), (100000, 32768)):
        size = ep.ep_rms_norm_backward_workspace(tokens, hidden)
        assert size >= hidden * 4 and size % (hidden * 4) == 0


@pytest.mark.parametrize("tokens,experts,topk,ranks", [(-1, 8, 2, 0), (4, 0, 1, 0), (4, 4097, 2, 0), (4, 8, 0, 0),
                                                       (4, 8, 9, 0), (4, 64, 33, 0), (4, 8, 2, 3), (4, 8, 2, -1)])
def test_route_sizes(ep, tokens, experts, topk, ranks):
    assert ep.lib.ep_route(tokens, experts, topk, 256, 0, experts, None, 1, 256, 256, ranks, None, 0.0, None, None, None,
                           None, None, 0, None) == BAD
    assert ep.lib.ep_route_backward(tokens if ranks == 0 else -1, experts, topk, 256, 0, experts, 1, 256, 256, 256, 256,
                                    256, None, 256, experts, None) == BAD


def test_route_workspace(ep):
    assert ep.ep_route_workspace(4, 0) == ep.ep_route_workspace(-1, 4) == 0
    assert ep.ep_route_workspace(0, 64) > 0            # the loss of no tokens is computed too
    assert ep.ep_route_workspace(131072, 4096) > ep.ep_route_workspace(1, 4096)


@pytest.mark.parametrize("change", [dict(places=-1), dict(experts=0), dict(experts=4097), dict(width=8), dict(width=24),
                                    dict(width=65552), dict(out=4), dict(out=12), dict(gated=2), dict(values=None),
                                    dict(values=264), dict(value_stride=72), dict(value_stride=1 << 31), dict(scale_stride=0),
                                    dict(w=None), dict(w=8), dict(ws=None), dict(off=None), dict(count=None),
                                    dict(out_bf16=None), dict(out_stride=60), dict(out_values=256), dict(places=5)])
def test_product_arguments(ep, change):
    a = dict(places=4, a_rows=4, experts=2, width=64, out=64, gated=0, values=256, value_stride=64, scales=256,
             scale_stride=1, w=256, ws=256, off=256, count=256, rows=None, out_bf16=256, out_stride=64, out_values=None,
             ovs=0, out_scales=None, oss=0, status=None, stream=None)
    a.update(change)
    assert ep.lib.ep_expert_product(*a.values()) == BAD


def test_pick_sum_arguments(ep):
    def call(rows=4, places=4, hidden=64, topk=2, ranks=2, experts=4, y=256, ys=64, idx=256, out=256, os=64):
        return ep.lib.ep_pick_sum(rows, places, hidden, topk, ranks, experts, y, ys, idx, 256, 256, 256, 256, 256, out, os,
                                  None, None)
    assert {call(rows=-1), call(places=-1), call(hidden=60), call(topk=0), call(topk=33), call(ranks=3), call(ranks=65),
            call(experts=1), call(y=None), call(y=264), call(ys=60), call(idx=None), call(out=None), call(os=56)} == {BAD}
    assert call(rows=0, idx=None, out=None) == ep.EP_OK


def test_packed_rows_hold_values_and_scales(ep):
    from combine_ep_layout_04_gb300 import Fp8Rows
    for width in range(8, 2000, 8):
        size = 2 * Fp8Rows.packed_width(width)
        assert size % 16 == 0 and size >= width + 4 * ((width + 127) // 128) and size < width + 4 * ((width + 127) // 128) + 20
    import torch
    rows = Fp8Rows.from_packed(torch.zeros(3, Fp8Rows.packed_width(264), dtype=torch.bfloat16), 264)
    assert rows.values.shape == (3, 264) and rows.scales.shape == (3, 3) and rows.packed.shape[0] == 3
