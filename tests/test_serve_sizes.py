"""Sizes at the ends of their ranges, on the host: no GPU is touched."""
import ctypes

import pytest

from w8a8_int8_quantized_token_gb300 import binding, build_lib

UNSUPPORTED = -2
FAKE = 4096  # never dereferenced: argument checks fail first


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.lib()


def append(lib, heads, dk, dv, q_heads=0, pitch=1):
    """Pitches of 1 element rule the vector kernel out."""
    c = ctypes.pointer(binding._PagedCache(FAKE, FAKE, pitch, pitch, pitch, pitch, pitch, pitch, 8, 16, heads, dk, dv, 0))
    q = FAKE if q_heads else None
    return lib.wq_rope_append_paged(q, pitch, pitch, q_heads, FAKE, pitch, pitch, FAKE, pitch, pitch, None, FAKE, None, 0, 4,
                                    0, 0, c, q, pitch, pitch, None, None)


def test_append_refuses_more_elements_than_a_launch_has_threads_for(lib):
    """65536 heads of 16384 for keys and values are 2^31 elements a token, with
    queries 3 * 2^30: neither may wrap around in a 32-bit count."""
    assert append(lib, 65536, 16384, 16384) == UNSUPPORTED
    assert append(lib, 65536, 16384, 16384, q_heads=65536) == UNSUPPORTED
    assert append(lib, 1024, 8192, 8192) == UNSUPPORTED  # 2^24, 256 past the most


def test_rope_refuses_more_pairs_than_a_launch_has_threads_for(lib):
    call = lambda heads, D: lib.wq_rope(FAKE, 1, 1, FAKE, FAKE, 9, 4, heads, D, 2, 0, 0, 2, FAKE, 1, 1, None, None)
    assert call(65536, 16384) == UNSUPPORTED and call(65536, 257) == UNSUPPORTED  # the pair counts as one
