"""The few-token layer where the cases of test_gpu_decode.py do not reach: its precision, element by element, and headers that were
not left zero."""
import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild
from tests.test_gpu_decode import Run, check, inputs, layer64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mbuild.build()
    return mb.load()


def half_step(v):
    """Half of the distance between bf16 numbers (8 significant bits) at v."""
    return torch.ldexp(torch.ones_like(v), torch.frexp(v)[1] - 9)


@pytest.mark.parametrize("kw", [dict(T=5, h=512, f=256, E=8, k=2, seed=91), dict(T=33, h=320, f=64, E=4, k=1, seed=92),
                                dict(T=128, h=256, f=320, E=4, k=2, seed=93), dict(T=70, h=192, f=128, E=64, k=8, seed=94)])
def test_only_y_is_rounded(kw):
    """Each element is within half a step of its 64-bit value, and what H's 16 bits leave of |H| |W2|: two parts of 8 bits,
    2^-8 of 2^-8 at most, and as much again for the fp32 sums (of at most 512 terms: 2^-24 each, growing as their root)."""
    cfg, inp = inputs(**kw)
    run = Run(cfg, inp)
    run.call()
    assert run.ok()
    y, mag, _, _ = layer64(inp, cfg.k)
    over = (run.y.double().cpu() - y).abs() - half_step(y) - 2.0 ** -15 * mag
    assert over.max() <= 0, over.max()


def test_values_that_bf16_does_not_hold():
    """H past bf16's largest number is infinite as before, with no NaN from its low part."""
    cfg, inp = inputs(T=3, h=64, f=64, E=2, k=1, seed=95)
    inp["x"] = torch.full_like(inp["x"], 2.0 ** 58)
    inp["W1"], inp["W3"], inp["W2"] = (torch.full_like(inp[n], 1.0) for n in ("W1", "W3", "W2"))
    run = Run(cfg, inp)
    run.call()
    assert run.ok()
    assert torch.isinf(run.y.float()).all() and (run.y > 0).all()


GROUPS = slice(128, 192)    # the header's bytes that count each token group's router units


@pytest.mark.parametrize("routing", [True, False])
@pytest.mark.parametrize("fp8", [False, True])
def test_expert_ids_that_no_router_wrote(fp8, routing):
    """A dirty header keeps every group from choosing its experts: the ids are what the buffer held.  Those out of range are
    recorded and not placed, and the next call is right."""
    cfg, inp = inputs(T=50, h=256, f=256, E=6, k=3, seed=96)
    run = Run(cfg, inp, fp8=fp8)
    run.ws[256:] = 0xFF
    run.ws[GROUPS] = 0x40
    stale = torch.tensor([6, -1, 2 ** 31 - 1, -2 ** 31, 1000, 64, 255, 256], dtype=torch.int32, device="cuda")
    run.idx.copy_(stale.repeat(cfg.T * cfg.k // 8 + 1)[:cfg.T * cfg.k].view(cfg.T, cfg.k))
    run.idx[7] = torch.tensor([2, 4, 6], dtype=torch.int32)
    run.call(routing=routing)
    torch.cuda.synchronize()
    assert mb.moe_read_device_status(run.ws) == mb.MOE_ERR_DEVICE_INDEX
    rest = [t for t in range(cfg.T) if t != 7 or not routing]
    assert (run.y[rest] == 0).all()
    run.call()
    assert run.ok()
    check(cfg, inp, run, fp8=fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_one_expert_for_every_slot(fp8):
    """The same with ids in range, all of one expert: T * k rows for it, of which T are placed."""
    cfg, inp = inputs(T=128, h=128, f=256, E=8, k=8, seed=97)
    run = Run(cfg, inp, fp8=fp8)
    run.ws[GROUPS] = 0x40
    run.idx.fill_(5)
    run.gates.fill_(0.25)
    run.call()
    torch.cuda.synchronize()
    assert mb.moe_read_device_status(run.ws) == mb.MOE_ERR_DEVICE_INDEX
    assert torch.isfinite(run.y.float()).all()
    run.call()
    assert run.ok()
    check(cfg, inp, run, fp8=fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_wait_that_runs_out(fp8):
    """A barrier's counter that starts far below zero never gets to its target: every block gives up after its limit of 4
    seconds, the status says so, and the workspace serves the next call."""
    cfg, inp = inputs(T=6, h=128, f=128, E=4, k=2, seed=98)
    run = Run(cfg, inp, fp8=fp8)
    run.ws[67] = 0xC0    # the top byte of the arrivals' 32-bit counter
    run.call()
    torch.cuda.synchronize()
    assert mb.moe_read_device_status(run.ws) == mb.MOE_ERR_DEVICE_TIMEOUT
    assert (run.y == 7).all()
    assert not run.ws[:256].any()
    run.call()
    assert run.ok()
    check(cfg, inp, run, fp8=fp8)
