"""Without a post-norm dy = beta gate G holds no y: rows of y that are not finite leave it as it is."""
import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild
from tests.test_gpu_block_norm import KINDS, backward64, close, dims, make, run_bwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mbuild.build()
    return mb.load()


@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("gate", list(KINDS))
@pytest.mark.parametrize("T,h", [(9, 264), (310, 4096), (309, 7168)])
def test_dy_without_a_post_norm(T, h, gate, f32, pre):
    v = make(T, h, f32, gate, post=False, pre=pre, seed=17)
    v["y"][2, 3] = float("nan")
    v["y"][4, h - 1] = float("inf")
    v["y"][T - 1] = -float("inf")
    got, ref = run_bwd(dims(T, h, f32, gate, 1.25, 0.5), v, gate), backward64(v, 1.25, 0.5, gate)
    assert torch.isfinite(ref["dy"]).all()
    close(got["dy"], ref["dy"], "dy")
    close(got["dr"], ref["dr"], "dr")
