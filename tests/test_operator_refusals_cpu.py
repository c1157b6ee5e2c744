"""What the autograd entry points of the operators around the head say to arguments that are
no tensors, or tensors without columns: their own errors, before anything is copied."""
import pytest
import torch

import lm_head_selected_gb300 as llp

X, T = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int64)


@pytest.mark.parametrize("call", [
    lambda: llp.layer_norm(None), lambda: llp.layer_norm([1.0, 2.0]), lambda: llp.layer_norm(X.numpy()),
    lambda: llp.layer_norm(torch.tensor(1.0)), lambda: llp.layer_norm(torch.zeros(3, 0)),
    lambda: llp.dropout(None, 0.1, 1), lambda: llp.dropout(X.numpy(), 0.1, 1),
    lambda: llp.embedding(T, None), lambda: llp.embedding(None, None), lambda: llp.embedding(T, 3.0)])
def test_no_tensors(call):
    with pytest.raises(ValueError):
        call()


def test_nothing_is_copied_before_a_tensor_is_refused(monkeypatch):
    def copied(self, *args, **kwargs):
        raise AssertionError("copied")
    monkeypatch.setattr(torch.Tensor, "contiguous", copied)
    for call in (lambda: llp.layer_norm(X.t()), lambda: llp.dropout(X.t(), 0.1, 1), lambda: llp.embedding(T, X.t())):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf"), 1e39, -1e300])
def test_embedding_refuses_a_scale_that_is_not_finite(scale):
    """In the C entries, before any device call; 1e39 is infinite in fp32."""
    from lm_head_selected_gb300 import _lib, build
    build.build()
    lib = _lib.load()
    bad_shape = -2
    for N in (0, 4):  # null pointers: nothing could be launched if the check were missing
        assert lib.embedding_fwd(None, None, 0, N, 10, 8, scale, -100, None, None) == bad_shape
        for accumulate in (0, 1):
            assert lib.embedding_bwd(None, None, 8, 0, N, 10, 8, scale, -100, accumulate, None, None, 0,
                                     None) == bad_shape
    assert lib.embedding_fwd(None, None, 0, 0, 10, 8, 3.4028234e38, -100, None, None) == 0
