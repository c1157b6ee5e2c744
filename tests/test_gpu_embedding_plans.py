"""The embedding gradient's plans by the size of the table and the number of a row's tokens:
two table rows per thread of the sort, more sort blocks than multiprocessors, and rows whose
pieces are joined in groups over several slices of the columns."""
import pytest
import torch

from operator_bounds import DTYPES
from test_gpu_embedding import _check_bwd, _tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from lm_head_selected_gb300 import build
    build.build()


# 128 blocks with one row per thread up to 131072 rows, with two up to 262144; then 256, 512 blocks
@pytest.mark.parametrize("V", [131073, 152064, 200064, 262143, 262144, 262145, 524289, 600001])
@pytest.mark.parametrize("N,D,dtype", [(700, 8, torch.bfloat16), (5000, 8, torch.float32), (3000, 9, torch.float16)])
def test_large_tables(V, N, D, dtype):
    g = torch.Generator().manual_seed(V + N)
    for kind in ("uniform", "zipf", "descending", "last_rows"):
        t = _tokens(kind, N, V, g)
        go = torch.randn(N, D, generator=g).to(dtype)
        _check_bwd(go, t, V, dtype)
        if kind != "descending":
            _check_bwd(go, t, V, dtype, scale=0.75, base=torch.randn(V, D, generator=g).to(dtype))


@pytest.mark.parametrize("V", [200064, 262145])
def test_large_tables_do_not_depend_on_the_other_tokens(V):
    import lm_head_selected_gb300 as llp
    g = torch.Generator().manual_seed(V)
    t = _tokens("zipf", 9000, V, g)
    go = torch.randn(9000, 16, generator=g).cuda()
    full = llp.embedding_bwd(go, t.cuda(), V)
    assert torch.equal(full, llp.embedding_bwd(go, t.cuda(), V))
    for v in (0, 1, 17, int(t[(t >= 0) & (t < V)].max())):
        sel = torch.nonzero(t == v).flatten()
        assert torch.equal(full[v], llp.embedding_bwd(go[sel.cuda()], t[sel].cuda(), V)[v])


# slices have 256 columns in fp32, 512 in 16 bits
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [600, 601, 1100, 1101, 2056])
@pytest.mark.parametrize("counts", [(2100, 33, 600, 1), (513, 512, 544), (20000, 40)])
def test_groups_of_pieces_over_several_slices(dtype, D, counts):
    g = torch.Generator().manual_seed(D + len(counts))
    V = len(counts) + 2
    t = torch.cat([torch.full((n,), i + 1) for i, n in enumerate(counts)] + [torch.tensor([-100, V])])
    t = t[torch.randperm(len(t), generator=g)]
    go = torch.randn(len(t), D, generator=g).to(dtype)
    _check_bwd(go, t, V, dtype)
    _check_bwd(go, t, V, dtype, scale=0.5, base=torch.randn(V, D, generator=g).to(dtype))
    wide = torch.randn(len(t), D + 7, generator=g).to(dtype).cuda()
    _check_bwd(wide[:, 3:3 + D], t, V, dtype, base=torch.randn(V, D, generator=g).to(dtype))
