"""The sites and seeds that the documentation gives the micro-batches of a step and the ranks of a
data-parallel one draw masks of their own, none of them those of another step's."""
import itertools

import pytest
import torch

from test_gpu_ops import G, dev  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def test_micro_batches_and_ranks_draw_their_own_masks(G, dev):
    seed, dropouts, micro, ranks, n = 0x5EED, 2, 3, 2, 1 << 16
    x = torch.ones(64, n // 64, device=dev)
    step = torch.zeros(1, dtype=torch.int32, device=dev)
    masks = {}
    for s, r, d, m in itertools.product(range(2), range(ranks), range(dropouts), range(micro)):
        step.fill_(s)
        y = torch.empty_like(x)
        G.amp_dropout_forward(x, 0.5, seed + r, d * micro + m, y, step=step)
        masks[s, r, d, m] = (y != 0).flatten()
    for a, b in itertools.combinations(masks, 2):
        # fair coins agree in half of the places, up to six standard deviations
        agree = (masks[a] == masks[b]).float().mean().item()
        assert abs(agree - 0.5) < 6 * 0.5 / n ** 0.5, (a, b, agree)
