"""Host-side checks of the few-token layer and the block norms (no GPU): every
refusal comes before any launch.  Fake device addresses are used, so these run
only where no CUDA device is present."""
import ctypes

import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild

FAKE = 1 << 20
MISALIGNED = FAKE + 8
BIG = 1 << 40
no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device addresses: host-only check")


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mb.load()


def _d(**kw):
    base = dict(T=64, h=128, f=256, E=8, k=2, has_bias=0)
    base.update(kw)
    return mb.moe_dims(**base)


def _decode(lib, d, args=None, ws=FAKE, ws_bytes=BIG):
    return lib.moe_layer_decode(ctypes.byref(d), *(args or [FAKE, FAKE, None] + [FAKE] * 6), ws, ws_bytes, None)


def _decode_fp8(lib, d, args=None, ws=FAKE, ws_bytes=BIG):
    return lib.moe_layer_decode_fp8(ctypes.byref(d), *(args or [FAKE, FAKE, None] + [FAKE] * 4), ws, ws_bytes, None)


@no_device
@pytest.mark.parametrize("kw,code", [
    (dict(T=129), mb.MOE_ERR_UNSUPPORTED), (dict(sar=1), mb.MOE_ERR_UNSUPPORTED),
    (dict(T=-1), mb.MOE_ERR_INVALID_ARG), (dict(k=9, E=16), mb.MOE_ERR_UNSUPPORTED),
    (dict(k=5, E=4), mb.MOE_ERR_INVALID_ARG), (dict(E=65), mb.MOE_ERR_UNSUPPORTED),
    (dict(h=96), mb.MOE_ERR_UNSUPPORTED), (dict(f=72), mb.MOE_ERR_UNSUPPORTED),
    (dict(capacity=-1), mb.MOE_ERR_INVALID_ARG), (dict(sar=2), mb.MOE_ERR_INVALID_ARG),
])
def test_decode_dims_refused(lib, kw, code):
    d = _d(**kw)
    assert _decode(lib, d) == code
    assert _decode_fp8(lib, d) == code
    for op in (mb.OP_LAYER_DECODE, mb.OP_LAYER_DECODE_FP8):
        assert mb.moe_workspace_bytes(d, op) == 0


@no_device
@pytest.mark.parametrize("kw", [dict(h=192), dict(f=192)])
def test_decode_fp8_wants_multiples_of_128(lib, kw):
    d = _d(**kw)
    assert _decode_fp8(lib, d) == mb.MOE_ERR_UNSUPPORTED
    assert mb.moe_workspace_bytes(d, mb.OP_LAYER_DECODE_FP8) == 0
    assert mb.moe_workspace_bytes(d, mb.OP_LAYER_DECODE) > 0


@no_device
@pytest.mark.parametrize("bad", [None, MISALIGNED])
@pytest.mark.parametrize("at", range(9))
def test_decode_pointers_refused(lib, at, bad):
    if at == 2 or (at >= 7 and bad is None):  # the bias is unused here; the routing outputs are optional
        return
    args = [FAKE, FAKE, None] + [FAKE] * 6
    args[at] = bad
    assert _decode(lib, _d(), args) == mb.MOE_ERR_INVALID_ARG


@no_device
@pytest.mark.parametrize("bad", [None, MISALIGNED, FAKE + 16])
def test_decode_buffers_refused(lib, bad):
    assert _decode(lib, _d(), ws=bad) == mb.MOE_ERR_INVALID_ARG
    assert _decode_fp8(lib, _d(), ws=bad) == mb.MOE_ERR_INVALID_ARG
    assert _decode_fp8(lib, _d(), [FAKE, FAKE, None, bad, FAKE, FAKE, FAKE]) == mb.MOE_ERR_INVALID_ARG
    assert _decode(lib, _d(has_bias=1)) == mb.MOE_ERR_INVALID_ARG
    assert lib.moe_layer_decode(None, *[FAKE] * 10, BIG, None) == mb.MOE_ERR_INVALID_ARG


@no_device
@pytest.mark.parametrize("T", [1, 128])
def test_decode_workspace_too_small(lib, T):
    for op, call in ((mb.OP_LAYER_DECODE, _decode), (mb.OP_LAYER_DECODE_FP8, _decode_fp8)):
        d = _d(T=T)
        assert call(lib, d, ws_bytes=mb.moe_workspace_bytes(d, op) - 1) == mb.MOE_ERR_WORKSPACE


def _nd(**kw):
    base = dict(T=16, h=128, gate=mb.GATE_CHANNEL)
    base.update(kw)
    return mb.norm_dims(**base)


def _fwd(lib, nd, args=None):
    return lib.moe_block_norm_fwd(ctypes.byref(nd), *(args or [FAKE] * 7), None)


def _bwd(lib, nd, args=None, ws=FAKE, ws_bytes=BIG):
    return lib.moe_block_norm_bwd(ctypes.byref(nd), *(args or [FAKE] * 12), ws, ws_bytes, None)


@no_device
@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), mb.MOE_ERR_INVALID_ARG), (dict(h=0), mb.MOE_ERR_INVALID_ARG),
    (dict(h=-8), mb.MOE_ERR_INVALID_ARG), (dict(h=12), mb.MOE_ERR_UNSUPPORTED),
    (dict(h=8200), mb.MOE_ERR_UNSUPPORTED), (dict(gate=3), mb.MOE_ERR_INVALID_ARG),
    (dict(gate=-1), mb.MOE_ERR_INVALID_ARG), (dict(eps=0.0), mb.MOE_ERR_INVALID_ARG),
    (dict(eps=float("nan")), mb.MOE_ERR_INVALID_ARG), (dict(eps=-1e-5), mb.MOE_ERR_INVALID_ARG),
    (dict(alpha=float("inf")), mb.MOE_ERR_INVALID_ARG), (dict(beta=float("nan")), mb.MOE_ERR_INVALID_ARG),
])
def test_norm_dims_refused(lib, kw, code):
    nd = _nd(**kw)
    assert _fwd(lib, nd) == code
    assert _bwd(lib, nd) == code
    assert mb.moe_norm_workspace_bytes(nd) == 0
    nd = _nd()
    nd.res_f32 = 2
    assert _fwd(lib, nd) == mb.MOE_ERR_INVALID_ARG
    assert lib.moe_block_norm_fwd(None, *[FAKE] * 7, None) == mb.MOE_ERR_INVALID_ARG
    assert lib.moe_block_norm_bwd(None, *[FAKE] * 13, BIG, None) == mb.MOE_ERR_INVALID_ARG


# r, y, w_post, gate, w_pre, r_out, u
@no_device
@pytest.mark.parametrize("args", [
    [None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE],        # no residual
    [FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE],        # a gate kind without its gate
    [FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE],        # nowhere to put r_out
    [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None],        # nowhere to put u
    [FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE],        # u without w_pre
    [FAKE, None, None, None, None, None, None],        # nothing to do
    [FAKE, None, FAKE, None, FAKE, None, FAKE],        # w_post without y
    [FAKE, None, None, None, FAKE, FAKE, FAKE],        # r_out without y
] + [[MISALIGNED if i == j else FAKE for i in range(7)] for j in range(7)])
def test_norm_forward_pointers_refused(lib, args):
    assert _fwd(lib, _nd(), args) == mb.MOE_ERR_INVALID_ARG


# r_out, y, w_post, gate, w_pre, du, dr_out, dr, dy, dw_post, dgate, dw_pre
def _without(*missing):
    return [None if i in missing else FAKE for i in range(12)]


@no_device
@pytest.mark.parametrize("args", [
    _without(0), _without(3), _without(5), _without(7), _without(8), _without(9), _without(10), _without(11),
    _without(4), _without(2), _without(1), _without(1, 2, 8, 9), _without(1, 2, 8, 10),
] + [[MISALIGNED if i == j else FAKE for i in range(12)] for j in range(12)])
def test_norm_backward_pointers_refused(lib, args):
    assert _bwd(lib, _nd(), args) == mb.MOE_ERR_INVALID_ARG


@no_device
def test_norm_backward_buffers_refused(lib):
    nd = _nd()
    assert _bwd(lib, nd, ws=None) == mb.MOE_ERR_INVALID_ARG
    assert _bwd(lib, nd, ws=FAKE + 16) == mb.MOE_ERR_INVALID_ARG
    assert _bwd(lib, nd, ws_bytes=mb.moe_norm_workspace_bytes(nd) - 1) == mb.MOE_ERR_WORKSPACE


def test_an_error_raises(lib):
    with pytest.raises(mb.MoeError, match="moe_block_norm_fwd"):
        mb.moe_block_norm_fwd(_nd(h=12), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, stream=0)
