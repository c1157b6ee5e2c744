"""The embedding at the largest number of tokens that its entries take."""
import pytest
import torch

pytestmark = pytest.mark.gpu

MOST = (1 << 31) - 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    from lm_head_selected_gb300 import build
    build.build()
    if torch.cuda.mem_get_info()[1] < 100 << 30:
        pytest.skip("takes 62 GB of device memory")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N", [MOST, MOST - 6])
def test_forward_of_the_most_tokens(N):
    import lm_head_selected_gb300 as llp
    w = torch.tensor([[1.5], [2.0], [-3.0], [0.25], [7.0]], dtype=torch.bfloat16, device="cuda")
    t = torch.arange(N, device="cuda").remainder_(7).sub_(1)  # -1 .. 5, the first and last invalid
    out = llp.embedding_fwd(t, w)
    assert out.shape == (N, 1)
    want = torch.zeros(7, dtype=torch.bfloat16, device="cuda")
    want[1:6] = w[:, 0]
    step = 1 << 28
    for a in range(0, N, step):
        part = out[a:a + step, 0]
        assert torch.equal(part, want.roll(-(a % 7)).repeat(-(-len(part) // 7))[:len(part)])


def test_backward_of_the_most_tokens():
    """Few of them valid, at both ends and around every power of two."""
    import lm_head_selected_gb300 as llp
    V = 6
    at = torch.tensor(sorted({min(max((1 << k) + d, 0), MOST - 1) for k in range(32) for d in (-1, 0, 1)} | {5, 6, 9}))
    rows = torch.arange(len(at)) % V
    value = (torch.arange(len(at)) % 11 - 5).to(torch.bfloat16)
    t = torch.full((MOST,), -100, dtype=torch.int64, device="cuda")
    t[at.cuda()] = rows.cuda()
    g = torch.full((MOST, 1), float("nan"), dtype=torch.bfloat16, device="cuda")
    g[at.cuda(), 0] = value.cuda()
    got = llp.embedding_bwd(g, t, V)
    want = torch.zeros(V, dtype=torch.float32).index_add_(0, rows, value.float())  # small whole numbers: exact
    assert torch.equal(got.float().cpu()[:, 0], want)
