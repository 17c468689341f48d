"""Host-side checks of the block-scaled e4m3 operators (no GPU): every refusal
comes before any launch.  Fake device addresses are used, so these run only
where no CUDA device is present."""
import ctypes

import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild

FAKE = 1 << 20
MISALIGNED = FAKE + 8
BIG = 1 << 50
no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device addresses: host-only check")
BAD, UNS, SMALL = mb.MOE_ERR_INVALID_ARG, mb.MOE_ERR_UNSUPPORTED, mb.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mb.load()


def _gd(**kw):
    return mb.moe_gemm_dims(**{**dict(rows=64, K=256, N=512, E=4, trans_b=0, out_f32=0), **kw})


def _fd(**kw):
    return mb.moe_ffn_dims(**{**dict(rows=64, h=256, f=512, E=4, dw_bf16=0), **kw})


def _gemm(lib, d, args=None, ws=FAKE, n=BIG):
    return lib.moe_gemm_fp8_block(ctypes.byref(d), *(args or [FAKE] * 6), ws, n, None)


def _fwd(lib, d, args=None, ws=FAKE, n=BIG):
    return lib.moe_gated_ffn_fwd(ctypes.byref(d), *(args or [FAKE] * 12), ws, n, None)


def _bwd(lib, d, args=None, ws=FAKE, n=BIG):
    return lib.moe_gated_ffn_bwd(ctypes.byref(d), *(args or [FAKE] * 16), ws, n, None)


@no_device
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), BAD), (dict(K=0), BAD), (dict(N=-16), BAD), (dict(E=0), BAD), (dict(trans_b=2), BAD),
    (dict(out_f32=-1), BAD), (dict(E=65), UNS), (dict(K=24), UNS), (dict(N=8), UNS), (dict(K=(1 << 20) + 16), UNS),
    (dict(N=1 << 21), UNS), (dict(rows=2 ** 31 - 1, N=1 << 20), UNS),
])
def test_gemm_dims_refused(lib, kw, code):
    d = _gd(**kw)
    assert _gemm(lib, d) == code
    assert mb.moe_gemm_workspace_bytes(d) == 0


@no_device
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), BAD), (dict(h=0), BAD), (dict(f=-64), BAD), (dict(E=0), BAD), (dict(dw_bf16=2), BAD),
    (dict(E=65), UNS), (dict(h=96), UNS), (dict(f=160), UNS), (dict(h=1 << 21), UNS), (dict(f=1 << 21), UNS),
    (dict(rows=2 ** 31 - 1, f=1 << 20), UNS),
])
def test_ffn_dims_refused(lib, kw, code):
    d = _fd(**kw)
    assert _fwd(lib, d) == code and _bwd(lib, d) == code
    assert mb.moe_ffn_workspace_bytes(d, 0) == 0 and mb.moe_ffn_workspace_bytes(d, 1) == 0


@no_device
def test_null_dims(lib):
    assert lib.moe_gemm_fp8_block(None, *[FAKE] * 7, BIG, None) == BAD
    assert lib.moe_gated_ffn_fwd(None, *[FAKE] * 13, BIG, None) == BAD
    assert lib.moe_gated_ffn_bwd(None, *[FAKE] * 17, BIG, None) == BAD
    assert lib.moe_gemm_workspace_bytes(None) == 0 and lib.moe_ffn_workspace_bytes(None, 0) == 0


@no_device
@pytest.mark.parametrize("bad", [None, MISALIGNED])
def test_pointers_refused(lib, bad):
    for n, call, d, optional in ((6, _gemm, _gd(), ()), (12, _fwd, _fd(), ()), (16, _bwd, _fd(), ())):
        for i in range(n):
            args = [FAKE] * n
            args[i] = bad
            assert call(lib, d, args) == BAD, (n, i)
        assert call(lib, d, ws=bad) == BAD
        assert call(lib, d, ws=FAKE + 128) == BAD


@no_device
def test_optional_pointers_reach_the_workspace_check(lib):
    """What may be absent passes the pointer checks: the workspace of 0 bytes is refused then."""
    assert _gemm(lib, _gd(E=1), [FAKE] * 4 + [None, FAKE], n=0) == SMALL
    assert _gemm(lib, _gd(), [FAKE] * 4 + [None, FAKE], n=0) == BAD         # several groups want offsets
    assert _fwd(lib, _fd(E=1), [FAKE, None] + [FAKE] * 10, n=0) == SMALL
    assert _fwd(lib, _fd(), [FAKE] * 8 + [None] * 3 + [FAKE], n=0) == SMALL
    assert _fwd(lib, _fd(), [FAKE] * 8 + [None, FAKE, None, FAKE], n=0) == BAD
    assert _bwd(lib, _fd(), [FAKE] * 13 + [None] * 3, n=0) == SMALL
    assert _bwd(lib, _fd(), [FAKE] * 13 + [None, FAKE, FAKE], n=0) == BAD
    assert _bwd(lib, _fd(E=1), [FAKE, FAKE, None] + [FAKE] * 13, n=0) == SMALL


@no_device
def test_workspace_too_small(lib):
    assert _gemm(lib, _gd(), n=mb.moe_gemm_workspace_bytes(_gd()) - 1) == SMALL
    assert _fwd(lib, _fd(), n=mb.moe_ffn_workspace_bytes(_fd(), 0) - 1) == SMALL
    assert _bwd(lib, _fd(), n=mb.moe_ffn_workspace_bytes(_fd(), 1) - 1) == SMALL
    d = mb.dims(64, 128, 192, 8, 2)
    nf, nb = (mb.moe_workspace_bytes(d, op) for op in (mb.OP_LAYER_FWD_FP8_BLOCK, mb.OP_LAYER_BWD_FP8_BLOCK))
    P = ctypes.byref(d)
    assert lib.moe_layer_fwd_fp8_block(P, FAKE, FAKE, None, *[FAKE] * 8, FAKE, nf - 1, None) == SMALL
    assert lib.moe_layer_bwd_fp8_block(P, *[FAKE] * 15, FAKE, nb - 1, None) == SMALL
    d = mb.dims(64, 128, 192, 8, 2, sar=True)
    P = ctypes.byref(d)
    assert lib.moe_layer_fwd_fp8_block(P, FAKE, FAKE, None, *[FAKE] * 8, FAKE, BIG, None) == UNS
    assert lib.moe_layer_bwd_fp8_block(P, *[FAKE] * 15, FAKE, BIG, None) == UNS
    assert mb.moe_workspace_bytes(d, mb.OP_LAYER_FWD_FP8_BLOCK) == 0


@no_device
def test_quantisers_refuse(lib):
    rows = lib.moe_quantize_rows_fp8_block
    assert rows(FAKE, 4, 24, None, 1, 4, FAKE, FAKE, None) == BAD        # n not a multiple of 16
    assert rows(FAKE, 8, 32, None, 1, 4, FAKE, FAKE, None) == BAD        # rows beyond the source without idx
    assert rows(FAKE, 4, 32, FAKE, 0, 4, FAKE, FAKE, None) == BAD        # div
    assert rows(FAKE, -1, 32, None, 1, 4, FAKE, FAKE, None) == BAD
    for i in (0, 6, 7):
        args = [FAKE, 4, 32, None, 1, 4, FAKE, FAKE, None]
        for bad in (None, MISALIGNED):
            args[i] = bad
            assert rows(*args) == BAD
    assert rows(None, 0, 32, None, 1, 0, None, None, None) == mb.MOE_OK  # nothing to do
    w = lib.moe_quantize_weights_fp8_block
    for E, K, N in ((0, 16, 16), (1, 24, 16), (1, 16, 8), (1, 0, 16), (1, 16, -16)):
        assert w(FAKE, E, K, N, FAKE, FAKE, None) == BAD
    assert w(FAKE, 2 ** 30, 1024, 1024, FAKE, FAKE, None) == UNS
    for i in (0, 4, 5):
        args = [FAKE, 2, 32, 32, FAKE, FAKE, None]
        for bad in (None, MISALIGNED):
            args[i] = bad
            assert w(*args) == BAD
