"""The alternatives that amp_token_logprobs_forward lists: identifiers and log probabilities lie in
rows of one length.  Tensors without memory stand in for the GPU's, so no GPU is needed."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


@pytest.fixture(scope="module")
def G():
    from loss_scaling_master_gb300 import build as B
    B.build()
    import loss_scaling_master_gb300 as pkg
    return pkg


@pytest.mark.parametrize("shape", [(4, 20), (4, 2), (20,), (4, 3, 1), ()], ids=str)
def test_rows_of_another_length_are_refused(G, shape):
    """[4, 20] log probabilities next to [4, 3] identifiers would be filled three to a row, so from
    the second row on they would be another row's."""
    with FakeTensorMode():
        e = lambda s, t=torch.float32: torch.empty(s, dtype=t, device="cuda:0")
        with pytest.raises(ValueError, match="top_logp: rows of"):
            G.amp_token_logprobs_forward(e((4, 64)), e((4,), torch.int64), e((4,)),
                                         top_ids=e((4, 3), torch.int64), top_logp=e(shape))
