"""A backward workspace that was sized once for the most rows serves every smaller call."""
import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    mbuild.build()
    return mb.load()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("h", [8, 768, 1536, 2056, 4096, 5120, 6400, 8192])
def test_the_size_never_falls_as_rows_are_added(h, f32):
    sizes = [mb.moe_norm_workspace_bytes(mb.norm_dims(T, h, res_f32=f32)) for T in list(range(2600)) + [10 ** 4, 10 ** 6, 2 ** 31 - 1]]
    assert sizes[0] > 0 and sizes == sorted(sizes)


@pytest.mark.parametrize("op", [mb.OP_LAYER_DECODE, mb.OP_LAYER_DECODE_FP8])
@pytest.mark.parametrize("h,f,E,k", [(128, 128, 64, 1), (4096, 14336, 8, 2), (6400, 256, 64, 8), (2048, 1408, 64, 6)])
def test_nor_that_of_the_few_token_layer(h, f, E, k, op):
    sizes = [mb.moe_workspace_bytes(mb.dims(T, h, f, E, k), op) for T in range(129)]
    assert sizes[0] > 0 and sizes == sorted(sizes)


@pytest.mark.gpu
@pytest.mark.parametrize("f32", [False, True])
def test_one_workspace_for_fewer_rows(f32):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    h, most = 4096, 1000
    g = torch.Generator("cuda").manual_seed(3)
    res = torch.float32 if f32 else torch.bfloat16
    n = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    r, y, du, dr_out = n(most, h, dtype=res), n(most, h), n(most, h), n(most, h, dtype=res)
    w = 1 + 0.1 * n(h, dtype=torch.float32)
    ws = torch.zeros(mb.moe_norm_workspace_bytes(mb.norm_dims(most, h, res_f32=f32)), dtype=torch.uint8, device="cuda")
    for T in (1000, 303, 304, 305, 152, 1, 999):
        nd = mb.norm_dims(T, h, res_f32=f32)
        got = []
        for space in (ws, torch.zeros(mb.moe_norm_workspace_bytes(nd), dtype=torch.uint8, device="cuda")):
            out = [torch.empty(T, h, dtype=res, device="cuda"), torch.empty(T, h, dtype=torch.bfloat16, device="cuda"),
                   torch.empty_like(w), torch.empty_like(w)]
            mb.moe_block_norm_bwd(nd, r[:T], y[:T], w, None, w, du[:T], dr_out[:T], out[0], out[1], out[2], None, out[3], space)
            torch.cuda.synchronize()
            assert mb.moe_read_device_status(space) == mb.MOE_OK
            got.append(out)
        for a, b in zip(*got):
            assert torch.equal(a, b) and torch.isfinite(a.float()).all()
