"""The comparison of tests/test_experts_exact_gpu.py finds planted mistakes (no GPU): a sum of zeros, one
without its last terms, its last row or half of its rows, at every length that those tests use."""

import pytest
import torch

from _exact import bf16_of, same, whole

LENGTHS = [72, 1096, 4104, 8200, 16392, 32768, 33000, 300000, 2**20]


def rejected(got, want):
    try:
        same(bf16_of(got), bf16_of(want), "planted")
    except AssertionError:
        return True
    return False


@pytest.mark.parametrize("length", LENGTHS)
def test_planted_mistakes_are_found(length):
    a, b = whole((32, length), 1).double(), whole((16, length), 2).double()
    want = a @ b.t()
    assert not rejected(want, want)
    assert rejected(torch.zeros_like(want), want)
    for left in (8, 64, length // 2):  # a vector, a step, half of the terms
        assert rejected(a[:, :-left] @ b[:, :-left].t(), want), left
        assert rejected(a[:, left:] @ b[:, left:].t(), want), left
    assert rejected(a @ b.t() + a[:, -8:] @ b[:, -8:].t(), want)  # taken twice


@pytest.mark.parametrize("length", LENGTHS)
def test_a_single_dropped_row_is_found(length):
    """Over the tests' outputs (thousands, here 4096), one term of the sum shows in some."""
    a, b = whole((64, length), 3).double(), whole((64, length), 4).double()
    a[:, -1], b[:, -1] = a[:, -1].sign() * 2, b[:, -1].sign() * 2
    assert rejected(a[:, :-1] @ b[:, :-1].t(), a @ b.t())


def test_partial_sums_stay_exact():
    """The largest magnitude a sum can have: 4 per product, a bias of 2."""
    assert 4 * max(LENGTHS) + 2 < 2**24
