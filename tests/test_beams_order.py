"""Selections at the borders of how sums are held, on the GPU.  Bars as in test_beams."""
import pytest
import torch

import dlrm_embedding_interaction_amd as dl
from test_beams import check_select
from test_history import gen

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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("items", [1900, 3001, 20000])
def test_rows_of_the_same_logits_tie_in_any_order(dtype, items):
    """Beams of one score whose rows hold the same logits in other orders, a rising one among them: what a sum stands
    against follows the order of the row, its logarithm may not.  Equal scores go by beam, logit and item."""
    tops = [512.0 * k + 280.0 for k in (*range(-24, 25), -100, -77, 50, 70, 88, 99)]      # fp16 holds 65504
    groups, beams, keep = len(tops), 4, 60
    rows = torch.empty((groups, beams, items), dtype=dtype)
    for g, top in enumerate(tops):
        x = torch.rand(items, generator=gen(72 + g)) * -800.0
        x[-40:] *= 4.0 / 800.0
        x = (x + top).sort().values.to(dtype)
        for w in range(beams):
            rows[g, w] = x if w == 1 else x[torch.randperm(items, generator=gen(200 + 4 * g + w))]
    got = dl.history_select(rows.cuda(), torch.full((groups, beams), -2.0).cuda(), keep)
    s, p, i = (t.cpu() for t in got)
    for g in range(groups):
        want = sorted((-v, w, at) for w in range(beams) for at, v in enumerate(rows[g, w].tolist()))[:keep]
        assert p[g].tolist() == [w for _, w, _ in want], tops[g]
        assert i[g].tolist() == [at for _, _, at in want], tops[g]
        x = rows[g, 0].double()
        exact = -2.0 + (rows[g, p[g].long(), i[g].long()].double() - x.max() - torch.log(torch.exp(x - x.max()).sum()))
        # as test_beams; the logarithm's spacing at 52000 and its last rounding are below 2^-32 both
        assert float(((s[g].double() - exact).abs() - 2.0 ** -24 * exact.abs()).max()) <= 2.0 ** -27
