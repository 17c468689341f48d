"""The few-token layer in phases long enough for later rounds (pieces that go to whichever block is free) in FC1 and FC2, and
with more FC2 tiles than its table holds: against the 64-bit formula, computed on the GPU, and call against call.

Tolerances: bf16 weights: half a step of bf16 for y's one rounding and 2^-15 of sum_j g_j |H_j| |W2| for H's 16 bits and the
fp32 sums, whose errors are independent over the f terms (f >= 1408 here: at most 2^-18 of that sum), element by element;
e4m3: 5e-3 as in test_gpu_decode.py."""
import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild
from tests.helpers import rel_l2
from tests.test_gpu_decode_edges import half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mbuild.build()
    return mb.load()


def rounds(steps, tile_steps):
    """The layer's rule: later rounds where a block's share is long against a tile."""
    blocks = torch.cuda.get_device_properties(0).multi_processor_count
    return 4 if steps // blocks >= max(48, 6 * max(4, tile_steps // 8)) else 1


def codes(v, quotient):
    """Rows of e4m3 values: scale amax / 448, or amax times the reciprocal as the few-token layer's activations have it."""
    v = v.float()
    a = v.abs().amax(-1, keepdim=True)
    s = a / torch.full_like(a, 448.0) if quotient else a * torch.full_like(a, 1.0).div_(torch.full_like(a, 448.0))
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (v / s).to(torch.float8_e4m3fn).double() * s.double()


CASES = {
    "wide_experts": dict(T=32, h=4096, f=14336, E=8, k=2, bias=False, seed=101),
    "skewed": dict(T=61, h=2048, f=5120, E=32, k=4, bias=True, seed=102),
    "many_tiles": dict(T=128, h=6400, f=1408, E=64, k=8, bias=False, seed=103),
    "short_contraction": dict(T=128, h=512, f=6400, E=48, k=6, bias=True, seed=104),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_long_phases(name, fp8):
    c = CASES[name]
    T, h, f, E, k = (c[n] for n in ("T", "h", "f", "E", "k"))
    g = torch.Generator("cuda").manual_seed(c["seed"])
    n = lambda shape, std, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda").normal_(0, std, generator=g)  # noqa: E731
    x, Wg = n((T, h), 1.0), n((h, E), h ** -0.5, torch.float32)
    W1, W3, W2 = n((E, h, f), h ** -0.5), n((E, h, f), h ** -0.5), n((E, f, h), f ** -0.5)
    b = -0.8 * torch.log1p(torch.arange(E, dtype=torch.float32, device="cuda")) if c["bias"] else None
    d = mb.dims(T, h, f, E, k, has_bias=c["bias"])
    ws = torch.zeros(mb.moe_workspace_bytes(d, mb.OP_LAYER_DECODE_FP8 if fp8 else mb.OP_LAYER_DECODE), dtype=torch.uint8, device="cuda")
    y, idx, gates = torch.empty_like(x), torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    if fp8:
        qw = torch.zeros(mb.moe_fp8_weight_bytes(d), dtype=torch.uint8, device="cuda")
        mb.moe_quantize_weights_fp8(d, W1, W3, W2, qw)

    def call():
        if fp8:
            mb.moe_layer_decode_fp8(d, x, Wg, b, qw, y, idx, gates, ws)
        else:
            mb.moe_layer_decode(d, x, Wg, b, W1, W3, W2, y, idx, gates, ws)

    call()
    torch.cuda.synchronize()
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
    first = y.clone()
    # the reference, expert by expert
    logits = x.double() @ Wg.double() + (0 if b is None else b.double())
    top, want = torch.sort(logits, dim=-1, descending=True, stable=True)
    want, p = want[:, :k], torch.softmax(top[:, :k], -1)
    assert torch.equal(idx.long(), want) and (gates.double() - p).abs().max() <= 1e-5
    ref, mag, active = torch.zeros(T, h, dtype=torch.float64, device="cuda"), torch.zeros(T, h, dtype=torch.float64, device="cuda"), 0
    for e in range(E):
        t, j = torch.nonzero(want == e, as_tuple=True)
        if not len(t):
            continue
        active += 1
        xe, w1, w3, w2 = x[t].double(), W1[e].double(), W3[e].double(), W2[e].double()
        if fp8:
            xe = codes(x[t], False)
            w1, w3, w2 = (codes(w[e].t().contiguous(), True).t() for w in (W1, W3, W2))
        a = xe @ w1
        hh = a * torch.sigmoid(a) * (xe @ w3)
        if fp8:
            hh = codes(hh.to(torch.bfloat16), False)
        gate = p[t, j][:, None]
        ref.index_add_(0, t, gate * (hh @ w2))
        mag.index_add_(0, t, gate * (hh.abs() @ w2.abs()))
    step = 128 if fp8 else 64
    tiles1, tiles2 = active * -(-f // 128), active * -(-h // 256)
    assert rounds(tiles1 * (h // step), h // step) == 4 and (rounds(tiles2 * (f // step), f // step) == 4 or name == "short_contraction")
    assert tiles2 > 1024 or name != "many_tiles"
    if fp8:
        assert rel_l2(y.double().cpu(), ref.cpu()) <= 5e-3
    else:
        over = (y.double() - ref).abs() - half_step(ref) - 2.0 ** -15 * mag
        assert over.max() <= 0, over.max()
    for _ in range(50):
        y.fill_(3.0)
        call()
        assert torch.equal(y, first)
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
