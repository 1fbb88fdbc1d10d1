"""The gated linear recurrence at sizes where its launches could go wrong."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


import gated_deltanet_chunked_delta_amd as gdn  # noqa: E402
from gated_deltanet_chunked_delta_amd import blocks  # noqa: E402


def test_more_chunks_than_one_dimension_of_a_grid():
    """6e8 tokens of one channel, every value checked: without decay the states are sums of whole
    numbers and so are the gradients, exact in fp32 (sums of 1e5 tokens' -1, 0 and 1, their
    products below 2^24: walks of 260 steps' deviation)."""
    B, T = 6000, 100_001
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randint(-1, 2, (B, T, 1), generator=g, device="cuda", dtype=torch.int8).float() for _ in range(2))
    zero = torch.zeros_like(x)
    y, hT = gdn.gated_recurrence(x, zero, output_final_state=True)
    dx, dg = blocks.gdn_rec_bwd(x, zero, dy)[:2]
    for b in range(0, B, 500):
        s = slice(b, b + 500)
        h = x[s].double().cumsum(1)
        dh = dy[s].double().flip(1).cumsum(1).flip(1)
        assert torch.equal(y[s].double(), h) and torch.equal(hT[s].double(), h[:, -1]), b
        assert torch.equal(dx[s].double(), dh) and torch.equal(dg[s].double(), dh * (h - x[s])), b
