"""The row-tile attention kernel's barriers in the model of attn_pipeline, with
the counts that the kernel has."""
import random

import pytest

import attn_pipeline as M

# pieces with one row tile before, after and between pieces with two
MIXED = [[(1, 1, True, 1, 1), (1, 2, True, 1, 1)], [(1, 2, True, 1, 1), (1, 1, True, 1, 1), (1, 2, True, 1, 1)],
         [(3, 1, False, 1, 1), (2, 2, True, 1, 1)], [(5, 1, True, 1, 1), (4, 2, True, 1, 1), (3, 1, True, 1, 1), (2, 2, True, 1, 1)]]


def faults(D, lists, seeds, **change):
    kw = {**M.kernel_counts(D), **change}
    n = 0
    for pieces in lists:
        for seed in seeds:
            try:
                M.run(D, pieces, seed, **kw)
            except M.Fault:
                n += 1
    return n


@pytest.mark.parametrize("D", [64, 128])
def test_no_order_of_events_breaks_the_pipeline(D):
    R = random.Random(D)
    assert faults(D, MIXED, range(40)) == 0
    for seed in range(500):
        assert faults(D, [M.random_pieces(R)], [seed]) == 0
    assert faults(D, [[(16, 1, True, 1, 1)], [(16, 2, True, 1, 1)], [(9, 1, True, 1, 0), (5, 1, False, 0, 1)]], range(60)) == 0


def test_the_model_sees_what_each_rule_prevents():
    """Without the softmax warps' wait for the queries, idle warps run ahead of
    a piece with one row tile; without the product warps' part in their release,
    one that has no work falls behind; with the last product's signal alone, heads
    of 64 take the end of the last but two for it."""
    assert faults(128, MIXED[:1], range(40), softmax_waits=False) > 20
    assert faults(128, [[(1, 1, False, 1, 1)] * 6], range(400), release=8) > 0
    assert faults(64, [[(16, 1, True, 1, 1)]], range(40), last_two=False) > 10
