"""rstd = 1 / sqrt(variance + eps), to 2 ulp and the same whatever the row's length
and alignment: on rows whose mean and variance fp32 holds exactly, so that the sum
under the root is the same number at every length."""
import numpy as np
import pytest
import torch

from test_gpu_ops import G, dev, place  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
A = np.arange(1, 16, dtype=np.float32)      # rows of +a, -a: mean 0, variance a^2 (8 bits)
EPS = np.exp2(np.random.default_rng(7).uniform(-12, 4, 40)).astype(np.float32)


def rstds(G, dev, cols, lead):
    """rstd of every row under every eps."""
    x = place(torch.from_numpy(np.outer(A, np.tile([1.0, -1.0], cols // 2)).astype(np.float32)), dev, lead)
    y = torch.empty(x.numel() + 1, device=dev)[lead:lead + x.numel()].view(x.shape)
    mean, rstd = torch.empty(len(A), device=dev), torch.empty(len(A), device=dev)
    got = []
    for eps in EPS:
        G.amp_layer_norm_forward(x, None, None, float(eps), y, mean, rstd)
        assert not mean.any()
        got.append(rstd.cpu().numpy())
    return np.stack(got)


def test_rstd_is_the_same_at_every_length(G, dev):
    first = rstds(G, dev, 32, 0)
    var = (A.astype(np.float64) ** 2 + EPS.astype(np.float64)[:, None]).astype(np.float32)
    want = 1 / np.sqrt(var.astype(np.float64))
    ulp = np.spacing(want.astype(np.float32)).astype(np.float64)
    assert (np.abs(first - want) <= 2 * ulp).all()
    for cols in (32, 256, 1024, 2048, 4096, 8192, 16384, 32768):
        for lead in (0, 1):
            assert np.array_equal(rstds(G, dev, cols, lead), first), (cols, lead)
