"""The few-token layer where the cases of test_gpu_decode.py do not reach: its precision, element by element."""
import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild
from tests.test_gpu_decode import Run, inputs, layer64

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
