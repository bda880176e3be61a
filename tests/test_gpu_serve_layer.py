"""The serving example end to end: one decoder layer over a paged cache, its
tokens as ragged chunks and token by token."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
def test_chunks_and_single_tokens_agree():
    import serve_layer

    chunk, single, key_error = serve_layer.run()
    # Both walk the same numbers; attention sums them in another order and may
    # round its bf16 output the other way (2^-8 of a value), which the int8
    # quantization that follows may turn into one step of 1/127 of a row's
    # largest value in some places.  Outputs are normalised rows: the relative
    # 2-norm of the difference stays well below one such step everywhere.
    diff = (chunk.float() - single.float()).norm() / chunk.float().norm()
    assert chunk.shape == single.shape and chunk.isfinite().all() and float(diff) < 1 / 127 + 2 ** -8
    # two bf16 roundings (the cached key, the key turned back) of 2^-8 each,
    # relative to a pair's length, at most sqrt(2) of the largest key
    assert key_error < 2 * 2 ** -8 * 2 ** 0.5
