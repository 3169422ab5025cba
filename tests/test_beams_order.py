"""Selections at the borders of how sums are held, on the GPU.  Bars as in test_beams."""
import numpy as np
import pytest
import torch

import beams_oracle as bo
import dlrm_embedding_interaction_amd as dl
from test_beams import check_select
from test_history import gen, randn

pytestmark = pytest.mark.gpu

BORDER = 2.0 ** 20          # logits beyond it are summed against another reference


def run_of(*pieces):
    """A row of 512 logits for each list of (count, logit less the border), the rest of the 512 never taken."""
    row = []
    for piece in pieces:
        row += [x for n, x in piece for _ in range(n)]
        row += [-float("inf")] * (-len(row) % 512)
    return row


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_on_both_sides_of_the_border(sign):
    """Rows whose maximum passes +-2^20 while most of their sum lies on the side that it came from, and the other way
    round; parts of rows on both sides; next to rows that stay on one side."""
    if sign > 0:
        up = run_of([(1, 250.0)], [(424, 299.5)], [(1, 300.5)])
        back = run_of([(1, 300.5)], [(424, 299.5)], [(1, 250.0)])
        low, high = 255.0, 257.0
    else:
        up = run_of([(1, -300.0)], [(424, -212.5)], [(1, -211.5)])
        back = run_of([(1, -211.5)], [(424, -212.5)], [(1, -300.0)])
        low, high = -257.0, -255.0
    near = run_of([(3, low), (400, low - 0.5)], [(7, low)], [(9, low - 1.0)])
    rows = torch.tensor([up, back, near, near[::-1]])[None] + sign * BORDER
    s = torch.tensor([[-1.0, -1.25, -1.0, -2.0]])
    check_select(rows, s, 100)
    check_select(rows[:, :1], None, 3)
    # 40000 logits: twenty parts of a row, some on either side
    x = torch.full((2, 3, 40000), low)
    x[:, :, 13000:29000] = high
    x += 0.125 * torch.randint(-8, 5, x.shape, generator=gen(71))
    x[1] = x[1].flip(1)
    check_select(x + sign * BORDER, None, 64)
