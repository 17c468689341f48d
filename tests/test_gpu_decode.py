"""The few-token layer (moe_layer_decode, moe_layer_decode_fp8) against a plain
64-bit implementation of its formula.

Tolerances.  bf16 weights: H and y are each rounded once to bf16 (at most 2^-8
of each element, 2^-8 / sqrt(3) in the mean square), everything else is fp32.
Over the tensor the two errors, independent of each other, come to at most
sqrt(2 / 3) 2^-8 = 3.2e-3; TOL_Y is 2^-8.  Each element's limit is
1.1 * 2^-9 (|ref| + sum_j g_j |H_j| |W2|): y's own rounding in full, since the
sum is at least |ref|, and H's far below its worst case, which would need every
rounding of a row to fall the same way.  e4m3: the codes and scales are computed alike
here, but an fp32 sum that lands on the other side of a rounding boundary of
H's bf16 value or code moves one code by a step (2^-3 relative, at most a few
in 10^3 elements): 5e-3, the layer's own parity tolerance.  Gates: 1e-5.
"""
import math

import numpy as np
import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild
from tests.helpers import conditioned_inputs, rel_l2, small_config

pytestmark = pytest.mark.gpu

TOL_Y = 2 * 2.0 ** -9
TOL_Y_F8 = 5e-3
TOL_GATE = 1e-5


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mbuild.build()
    return mb.load()


# ------------------------------------------------------------ the reference
def route64(x, Wg, b, k):
    l = x.double() @ Wg.double()
    if b is not None:
        l = l + b.double()
    top, idx = torch.sort(l, dim=-1, descending=True, stable=True)
    return idx[:, :k], torch.softmax(top[:, :k], -1)


def kept(idx, E, capacity):
    """keep[t, j]: whether expert idx[t, j] takes the assignment (its first `capacity`, in order)."""
    keep = torch.ones_like(idx, dtype=torch.bool)
    if capacity:
        seen = [0] * E
        for t in range(idx.shape[0]):
            for j in range(idx.shape[1]):
                e = int(idx[t, j])
                keep[t, j] = seen[e] < capacity
                seen[e] += 1
    return keep


def quant_rows(v, weights=False):
    """Activations: scale amax * fp32(1 / 448); weights (as moe_quantize_weights_fp8 writes them): amax / 448."""
    v = v.float()
    s = v.abs().amax(-1, keepdim=True)
    s = s / 448.0 if weights else s * (torch.ones(()) / 448.0)
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (v / s).to(torch.float8_e4m3fn).double() * s.double()


def layer64(inp, k, capacity=0, fp8=False):
    """y and, for the element bound, sum_j g_j |H_j| |W2|."""
    x, E = inp["x"], inp["W1"].shape[0]
    idx, gates = route64(x, inp["Wg"], inp["b"], k)
    keep = kept(idx, E, capacity)
    y = torch.zeros(x.shape, dtype=torch.float64)
    mag = torch.zeros_like(y)
    for e in range(E):
        t, j = torch.nonzero((idx == e) & keep, as_tuple=True)
        if not len(t):
            continue
        xe, W1, W3, W2 = x[t].double(), inp["W1"][e].double(), inp["W3"][e].double(), inp["W2"][e].double()
        if fp8:
            xe = quant_rows(x[t])
            W1, W3, W2 = (quant_rows(inp[n][e].t().contiguous(), weights=True).t() for n in ("W1", "W3", "W2"))
        a, b = xe @ W1, xe @ W3
        h = a * torch.sigmoid(a) * b
        if fp8:
            h = quant_rows(h.to(torch.bfloat16))
        g = gates[t, j][:, None]
        y.index_add_(0, t, g * (h @ W2))
        mag.index_add_(0, t, g * (h.abs() @ W2.abs()))
    return y, mag, idx, gates


# ------------------------------------------------------------ the call
class Run:
    def __init__(self, cfg, inp, capacity=0, fp8=False, has_bias=None):
        self.d = mb.dims_of(cfg, has_bias=inp["b"] is not None if has_bias is None else has_bias, capacity=capacity)
        self.fp8 = fp8
        self.dev = {n: v.cuda() for n, v in inp.items() if isinstance(v, torch.Tensor)}
        self.ws = torch.zeros(mb.moe_workspace_bytes(self.d, mb.OP_LAYER_DECODE_FP8 if fp8 else mb.OP_LAYER_DECODE),
                              dtype=torch.uint8, device="cuda")
        self.y = torch.full((cfg.T, cfg.h), 7.0, dtype=torch.bfloat16, device="cuda")
        self.idx = torch.full((cfg.T, cfg.k), -1, dtype=torch.int32, device="cuda")
        self.gates = torch.full((cfg.T, cfg.k), -1.0, dtype=torch.float32, device="cuda")
        if fp8:
            self.qw = torch.zeros(mb.moe_fp8_weight_bytes(self.d), dtype=torch.uint8, device="cuda")
            mb.moe_quantize_weights_fp8(self.d, self.dev["W1"], self.dev["W3"], self.dev["W2"], self.qw)

    def call(self, stream=None, routing=True):
        v = self.dev
        out = (self.y, self.idx if routing else None, self.gates if routing else None, self.ws)
        if self.fp8:
            mb.moe_layer_decode_fp8(self.d, v["x"], v["Wg"], v.get("b"), self.qw, *out, stream=stream)
        else:
            mb.moe_layer_decode(self.d, v["x"], v["Wg"], v.get("b"), v["W1"], v["W3"], v["W2"], *out, stream=stream)

    def ok(self):
        torch.cuda.synchronize()
        return mb.moe_read_device_status(self.ws) == mb.MOE_OK


def inputs(bias=False, **kw):
    cfg = small_config(name="decode", **kw)
    inp = conditioned_inputs(cfg)
    inp = {n: v for n, v in inp.items() if isinstance(v, torch.Tensor) and n != "dy"}
    if not bias:
        inp["b"] = None
    return cfg, inp


def check(cfg, inp, run, capacity=0, fp8=False):
    y, mag, idx, gates = layer64(inp, cfg.k, capacity, fp8)
    got = run.y.double().cpu()
    np.testing.assert_array_equal(run.idx.cpu().numpy(), idx.numpy())
    assert (run.gates.double().cpu() - gates).abs().max() <= TOL_GATE
    assert rel_l2(got, y) <= (TOL_Y_F8 if fp8 else TOL_Y), rel_l2(got, y)
    if not fp8:
        assert ((got - y).abs() <= 1.1 * 2.0 ** -9 * (y.abs() + mag) + 1e-30).all()
    # a token none of whose slots is placed gets exactly zero
    none = ~kept(idx, cfg.E, capacity).any(1)
    assert (got[none] == 0).all()


SHAPES = {
    "one_token": dict(T=1, h=64, f=64, E=4, k=2, seed=21),
    "one_token_long": dict(T=1, h=1088, f=704, E=8, k=2, seed=22),
    "two_tokens": dict(T=2, h=192, f=320, E=3, k=1, seed=23),
    "single_expert": dict(T=5, h=128, f=192, E=1, k=1, seed=24),
    "k_equals_E": dict(T=9, h=256, f=448, E=4, k=4, seed=25),
    "k8_E64": dict(T=31, h=320, f=128, E=64, k=8, seed=26),
    "fill_16": dict(T=16, h=512, f=256, E=8, k=2, seed=27),
    "past_16": dict(T=17, h=448, f=576, E=10, k=3, seed=28),
    "fill_64": dict(T=64, h=256, f=1408, E=16, k=6, seed=29),
    "past_64": dict(T=65, h=2048, f=192, E=64, k=6, seed=30),
    "last_but_one": dict(T=127, h=576, f=320, E=5, k=2, seed=31),
    "largest": dict(T=128, h=512, f=512, E=8, k=2, seed=32),
    "largest_k8": dict(T=128, h=192, f=128, E=9, k=8, seed=33),
    "wide": dict(T=3, h=6400, f=64, E=16, k=1, seed=34),
    "narrow": dict(T=77, h=64, f=2048, E=2, k=2, seed=35),
}


@pytest.mark.parametrize("name", list(SHAPES))
def test_matches_the_formula(name):
    cfg, inp = inputs(**SHAPES[name])
    run = Run(cfg, inp)
    run.call()
    assert run.ok()
    check(cfg, inp, run)


F8_SHAPES = {
    "one_token": dict(T=1, h=128, f=128, E=4, k=2, seed=41),
    "one_token_long": dict(T=1, h=1152, f=640, E=8, k=2, seed=42),
    "k8_E64": dict(T=31, h=256, f=128, E=64, k=8, seed=43),
    "past_16": dict(T=17, h=384, f=512, E=10, k=3, seed=44),
    "fill_64": dict(T=64, h=256, f=1408, E=16, k=6, seed=45),
    "largest": dict(T=128, h=512, f=384, E=8, k=2, seed=46),
    "single_expert": dict(T=128, h=128, f=256, E=1, k=1, seed=47),
    "wide": dict(T=3, h=6400, f=128, E=16, k=1, seed=48),
}


@pytest.mark.parametrize("name", list(F8_SHAPES))
def test_e4m3_matches_the_formula(name):
    cfg, inp = inputs(**F8_SHAPES[name])
    run = Run(cfg, inp, fp8=True)
    run.call()
    assert run.ok()
    check(cfg, inp, run, fp8=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("capacity", [1, 5])
def test_capacity_drops(fp8, capacity):
    cfg, inp = inputs(T=60, h=256, f=128, E=6, k=2, seed=51)
    run = Run(cfg, inp, capacity=capacity, fp8=fp8)
    run.call()
    assert run.ok()
    check(cfg, inp, run, capacity, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_every_token_on_one_expert(fp8):
    """A bias that leaves all but k experts without tokens, some of them at minus infinity."""
    cfg, inp = inputs(T=128, h=128, f=256, E=12, k=2, seed=52)
    b = torch.full((12,), -float("inf"))
    b[3], b[7], b[11] = 50.0, 40.0, -1e4
    inp["b"] = b
    run = Run(cfg, inp, fp8=fp8)
    run.call()
    assert run.ok()
    check(cfg, inp, run, fp8=fp8)


def test_ties_go_to_the_lower_id():
    cfg, inp = inputs(T=20, h=128, f=64, E=7, k=3, seed=53)
    inp["Wg"] = torch.zeros_like(inp["Wg"])
    run = Run(cfg, inp)
    run.call()
    assert run.ok()
    assert (run.idx.cpu() == torch.arange(3, dtype=torch.int32)).all()
    check(cfg, inp, run)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_row_that_is_not_finite_stays_alone(fp8):
    cfg, inp = inputs(T=40, h=256, f=128, E=8, k=2, seed=54)
    run = Run(cfg, inp, fp8=fp8)
    run.call()
    assert run.ok()
    clean = run.y.clone()
    run.dev["x"][7] = float("nan")
    run.dev["x"][21, 5] = float("inf")
    run.call()
    assert run.ok()
    assert ((run.idx >= 0) & (run.idx < cfg.E)).all()
    rest = [t for t in range(cfg.T) if t not in (7, 21)]
    assert torch.equal(run.y[rest], clean[rest])
    assert not torch.isfinite(run.y[7].float()).any()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_row_of_zeros(fp8):
    cfg, inp = inputs(T=18, h=128, f=128, E=4, k=2, seed=55)
    inp["x"][3] = 0
    run = Run(cfg, inp, fp8=fp8)
    run.call()
    assert run.ok()
    assert (run.y[3] == 0).all()
    assert (run.idx[3].cpu() == torch.tensor([0, 1], dtype=torch.int32)).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_same_bits_whatever_the_workspace_held(fp8):
    """Twenty calls on other inputs in between, and a workspace full of other bytes past its first 256."""
    cfg, inp = inputs(T=37, h=1024, f=384, E=16, k=4, seed=56)
    run = Run(cfg, inp, fp8=fp8)
    run.call()
    assert run.ok()
    first = (run.y.clone(), run.idx.clone(), run.gates.clone())
    x = run.dev["x"].clone()
    for i in range(20):
        run.dev["x"].copy_(torch.roll(x, i + 1, 0))
        run.call()
    run.dev["x"].copy_(x)
    run.ws[256:] = 0xFF
    run.y.fill_(3.0)
    run.call()
    assert run.ok()
    for a, b in zip(first, (run.y, run.idx, run.gates)):
        assert torch.equal(a, b)


def test_a_workspace_serves_other_shapes_in_turn():
    big = max(mb.moe_workspace_bytes(mb.dims(*s), mb.OP_LAYER_DECODE) for s in ((128, 512, 512, 8, 2), (1, 1024, 2048, 16, 2)))
    ws = torch.zeros(big, dtype=torch.uint8, device="cuda")
    for rep in range(2):
        for kw in (dict(T=128, h=512, f=512, E=8, k=2, seed=57), dict(T=1, h=1024, f=2048, E=16, k=2, seed=58)):
            cfg, inp = inputs(**kw)
            run = Run(cfg, inp)
            run.ws = ws
            run.call()
            assert run.ok()
            check(cfg, inp, run)


def test_routing_outputs_are_optional():
    cfg, inp = inputs(T=11, h=128, f=64, E=4, k=2, seed=59)
    run = Run(cfg, inp)
    run.call()
    want = run.y.clone()
    run.y.zero_()
    run.call(routing=False)
    assert run.ok()
    assert torch.equal(run.y, want)


def test_no_tokens():
    d = mb.dims(0, 128, 64, 4, 2)
    w = torch.zeros(4 * 128 * 64, dtype=torch.bfloat16, device="cuda")
    Wg = torch.zeros(128, 4, device="cuda")
    ws = torch.zeros(max(256, mb.moe_workspace_bytes(d, mb.OP_LAYER_DECODE)), dtype=torch.uint8, device="cuda")
    before = mb.moe_kernel_launches()
    mb.moe_layer_decode(d, None, Wg, None, w, w, w, None, None, None, ws)
    assert mb.moe_kernel_launches() == before


@pytest.mark.parametrize("fp8", [False, True])
def test_on_a_side_stream_and_in_a_graph(fp8):
    cfg, inp = inputs(T=12, h=256, f=256, E=8, k=2, seed=60)
    run = Run(cfg, inp, fp8=fp8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run.call()
    s.synchronize()
    assert run.ok()
    check(cfg, inp, run, fp8=fp8)
    want = run.y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run.call()
    # replays read the inputs as they are then
    x = run.dev["x"].clone()
    run.dev["x"].copy_(torch.flip(x, (0,)))
    for _ in range(3):
        g.replay()
    assert run.ok()
    assert torch.equal(run.y, torch.flip(want, (0,)))


def test_agrees_with_the_layer_call():
    cfg, inp = inputs(T=100, h=512, f=448, E=8, k=2, seed=61)
    run = Run(cfg, inp)
    run.call()
    v = run.dev
    saved = torch.zeros(mb.moe_saved_bytes(run.d), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(mb.moe_workspace_bytes(run.d, mb.OP_LAYER_FWD), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(run.y)
    mb.moe_layer_fwd(run.d, v["x"], v["Wg"], None, v["W1"], v["W3"], v["W2"], y, saved, ws)
    assert run.ok()
    # the layer call also rounds A, B's product chain and O: one more rounding than this one
    assert rel_l2(run.y.double().cpu(), y.double().cpu()) <= TOL_Y + 2.0 ** -9
    assert math.isfinite(float(run.y.float().sum()))


@pytest.mark.parametrize("fp8", [False, True])
def test_long_tiles_in_few_pieces(fp8):
    """Few tiles of very many k-steps (FC2: 4 for each expert, 912 steps of 64 each): the phase is long, but its pieces
    are short against its tiles.  The reference runs on the GPU in 64 bits; TOL_Y as above."""
    T, h, f, E, k = 2, 1024, 58368, 2, 2
    g = torch.Generator("cuda").manual_seed(71)
    n = lambda shape, std: torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)  # noqa: E731
    x, W1, W3, W2 = n((T, h), 1.0), n((E, h, f), h ** -0.5), n((E, h, f), h ** -0.5), n((E, f, h), f ** -0.5)
    Wg = torch.randn(h, E, generator=g, device="cuda") * h ** -0.5
    d = mb.dims(T, h, f, E, k)
    ws = torch.zeros(mb.moe_workspace_bytes(d, mb.OP_LAYER_DECODE_FP8 if fp8 else mb.OP_LAYER_DECODE),
                     dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)
    if fp8:
        qw = torch.zeros(mb.moe_fp8_weight_bytes(d), dtype=torch.uint8, device="cuda")
        mb.moe_quantize_weights_fp8(d, W1, W3, W2, qw)
        mb.moe_layer_decode_fp8(d, x, Wg, None, qw, y, None, None, ws)
    else:
        mb.moe_layer_decode(d, x, Wg, None, W1, W3, W2, y, None, None, ws)
    torch.cuda.synchronize()
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
    p = torch.softmax(x.double() @ Wg.double(), -1)  # k = E: every expert, with its probability
    ref = torch.zeros(T, h, dtype=torch.float64, device="cuda")
    q = (lambda v, w=False: quant_rows(v.cpu(), w).cuda()) if fp8 else (lambda v, w=False: v.double())
    for e in range(E):
        w1, w3, w2 = (q(w[e].t().contiguous(), True).t() if fp8 else w[e].double() for w in (W1, W3, W2))
        a, b = q(x) @ w1, q(x) @ w3
        hh = a * torch.sigmoid(a) * b
        ref += p[:, e:e + 1] * ((q(hh.to(torch.bfloat16)) if fp8 else hh) @ w2)
    assert rel_l2(y.double().cpu(), ref.cpu()) <= (TOL_Y_F8 if fp8 else TOL_Y)


@pytest.mark.parametrize("T,E", [(1, 8), (1, 64), (3, 33), (40, 64)])
def test_routing_holds_over_many_calls(T, E):
    """The router's shared-memory phases follow each other closely: 300 calls on one input give the same bits, those of
    the formula."""
    cfg, inp = inputs(T=T, h=4096, f=64, E=E, k=min(E, 4), seed=72 + E + T)
    run = Run(cfg, inp)
    got = []
    for i in range(300):
        run.idx.fill_(-1)
        run.gates.fill_(-1.0)
        run.call()
        got.append((run.idx.clone(), run.gates.clone()))
    assert run.ok()
    idx, gates = route64(inp["x"], inp["Wg"], None, cfg.k)
    for a, b in got:
        assert torch.equal(a, got[0][0]) and torch.equal(b, got[0][1])
    assert (got[0][0].cpu() == idx).all() and (got[0][1].double().cpu() - gates).abs().max() <= TOL_GATE


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, overlap as they like."""
    runs = []
    for seed in (81, 82):
        cfg, inp = inputs(T=24, h=512, f=1024, E=8, k=2, seed=seed)
        runs.append((cfg, inp, Run(cfg, inp), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for _, _, run, s in runs:
            run.call(stream=s)
    torch.cuda.synchronize()
    for cfg, inp, run, _ in runs:
        assert run.ok()
        check(cfg, inp, run)


def test_after_a_launch_failure_on_the_host():
    """The injected failure reports MOE_ERR_CUDA; the workspace serves the next call."""
    cfg, inp = inputs(T=6, h=128, f=128, E=4, k=2, seed=83)
    run = Run(cfg, inp)
    mb.moe_test_fail_launch_after(1)
    with pytest.raises(mb.MoeError):
        run.call()
    torch.cuda.synchronize()
    run.call()
    assert run.ok()
    check(cfg, inp, run)
