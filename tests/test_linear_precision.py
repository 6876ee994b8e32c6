"""The limit on the error in norm tells three bf16 terms from two (CPU model of the chunk form)."""
import pytest
import torch

import linear_pairs as pairs
from linear_precision import LIMIT, error, inputs, model

SIZES = [(1, 300, 8, 8, 64, 64), (1, 161, 8, 4, 128, 128), (2, 500, 4, 4, 32, 128)]


def errors(x, **kw):
    want = pairs.prefill(*(x[n] for n in ("q", "k", "v", "g", "scale", "S0")))
    return [error(a, b) for a, b in zip(model(x, **kw), want)]


@pytest.mark.parametrize("size", SIZES)
def test_three_terms_are_within_and_two_are_not(size):
    x = inputs(*size, torch.float32, seed=size[1])
    o, S = errors(x, rows=3, weights=3, update=3)
    assert o < LIMIT / 3 and S < LIMIT / 3
    for kw, lost in ((dict(rows=2, weights=3, update=3), "oS"), (dict(rows=3, weights=2, update=3), "o"),
                     (dict(rows=3, weights=3, update=2), "S")):
        o, S = errors(x, **kw)
        print(kw, o, S)
        assert ("o" not in lost or o > 2 * LIMIT) and ("S" not in lost or S > 2 * LIMIT), (kw, o, S)


@pytest.mark.parametrize("size", SIZES)
def test_states_of_bf16_inputs(size):
    """bf16 rows are one term; only the update's three keep the state."""
    x = inputs(*size, torch.bfloat16, seed=size[1])
    assert errors(x, rows=1, weights=1, update=3)[1] < LIMIT / 3
    assert errors(x, rows=1, weights=1, update=2)[1] > 2 * LIMIT
