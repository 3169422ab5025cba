"""The event-history operators at the ends of their types' ranges, and where few bits would show.

Values that a row does not see leave it bit for bit as it was.  Where a result is compared with its formula, the bar
counts u = 2^-24 for each fp32 rounding, and half a step of the output's type.
"""
import math

import numpy as np
import pytest
import torch

import dlrm_embedding_interaction_amd as dl
import history_oracle as ho
from test_history import ALL, HALF, U, Pair, bound, f64, gen, randn, starts

MAX32 = torch.finfo(torch.float32).max


def encode(q, k, v, lens, pad=None, **kw):
    return dl.history_attention(q.cuda(), k.cuda(), v.cuda(), starts(lens).cuda(),
                                padding=None if pad is None else pad.cuda(), **kw).cpu()


# --- a row's bits are its own ----------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,dim", [([200, 61], 64), ([1300], 128)])
def test_encode_rows_do_not_depend_on_their_neighbours(dtype, lens, dim):
    """Logits of other rows, however large, move nothing in a row of ordinary ones."""
    n = sum(lens)
    q, k, v = (randn((n, 2, dim), s, dtype) for s in (17, 18, 19))
    want = encode(q, k, v, lens)
    loud = torch.arange(n) % 5 == 2
    q[loud] *= 60
    got = encode(q, k, v, lens)
    assert torch.equal(got[~loud], want[~loud])
    assert not torch.equal(got[loud], want[loud])
