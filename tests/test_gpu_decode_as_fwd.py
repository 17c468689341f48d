"""moe_layer_decode_fp8_as_fwd: the few-token layer with the activation scales of moe_layer_fwd_fp8, against the 64-bit
formula with those scales and against that call.

Tolerance: 5e-3, the layer's own parity limit.  Between the two calls there are three roundings to bf16 (the layer's O, and y
on both sides), each at most 2^-8 / sqrt(3) in the mean square and independent of the others: 3.9e-3."""
import ctypes

import pytest
import torch

import tests.test_gpu_decode as base
from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild
from tests.helpers import rel_l2

TOL = 5e-3


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mb.load()


class Run(base.Run):
    def __init__(self, cfg, inp, capacity=0):
        super().__init__(cfg, inp, capacity, fp8=True)

    def call(self, stream=None):
        v = self.dev
        mb.moe_layer_decode_fp8_as_fwd(self.d, v["x"], v["Wg"], v.get("b"), self.qw, self.y, self.idx, self.gates, self.ws,
                                       stream=stream)


def of_the_layer(run):
    v = run.dev
    saved = torch.zeros(mb.moe_saved_bytes(run.d), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(mb.moe_workspace_bytes(run.d, mb.OP_LAYER_FWD_FP8), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(run.y)
    mb.moe_layer_fwd_fp8(run.d, v["x"], v["Wg"], v.get("b"), run.qw, y, saved, ws)
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(base.F8_SHAPES))
def test_as_the_layer(lib, name, monkeypatch):
    cfg, inp = base.inputs(**base.F8_SHAPES[name])
    run = Run(cfg, inp)
    run.call()
    y = of_the_layer(run)
    assert run.ok()
    assert rel_l2(run.y.double().cpu(), y.double().cpu()) <= TOL
    product = base.quant_rows
    monkeypatch.setattr(base, "quant_rows", lambda v, weights=False: product(v, weights=True))
    base.check(cfg, inp, run, fp8=True)


@pytest.mark.gpu
def test_as_the_layer_with_drops(lib):
    cfg, inp = base.inputs(T=60, h=256, f=128, E=6, k=2, seed=51)
    run = Run(cfg, inp, capacity=9)
    run.call()
    y = of_the_layer(run)
    assert run.ok()
    assert rel_l2(run.y.double().cpu(), y.double().cpu()) <= TOL


FAKE = 1 << 20


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses: host-only check")
def test_refusals(lib):
    def call(d, args=None, ws=FAKE, ws_bytes=1 << 40):
        return lib.moe_layer_decode_fp8_as_fwd(ctypes.byref(d), *(args or [FAKE, FAKE, None] + [FAKE] * 4), ws, ws_bytes, None)

    d = mb.dims(64, 128, 256, 8, 2)
    assert call(mb.dims(129, 128, 256, 8, 2)) == mb.MOE_ERR_UNSUPPORTED
    assert call(mb.dims(64, 192, 256, 8, 2)) == mb.MOE_ERR_UNSUPPORTED
    for at in range(7):
        if at != 2:
            args = [FAKE, FAKE, None] + [FAKE] * 4
            args[at] = FAKE + 8
            assert call(d, args) == mb.MOE_ERR_INVALID_ARG
    assert call(d, ws=None) == mb.MOE_ERR_INVALID_ARG
    assert call(d, ws_bytes=mb.moe_workspace_bytes(d, mb.OP_LAYER_DECODE_FP8) - 1) == mb.MOE_ERR_WORKSPACE
