"""Sizes at the ends of their ranges, on the host: no GPU is touched."""
import ctypes
import os
import re
import subprocess

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


ONCE = r"""
#include <cstdio>
#include "wq_once.h"
int main() {
  wq::OncePerDevice once;
  int calls = 0;
  bool works = false;
  auto set = [&] { ++calls; return works; };
  auto step = [&](int device) { const bool ok = once(device, set); printf("%d%d ", ok, calls); };
  step(0); step(0);              // a failure is not kept
  works = true;
  step(0); step(0);              // a success is
  step(63); step(63); step(0);   // for its device alone
  works = false;
  step(5); step(63);
}
"""


def test_kernels_are_set_up_on_every_device_and_after_a_failure(tmp_path):
    src = tmp_path / "once.cpp"
    src.write_text(ONCE)
    subprocess.run(["g++", "-std=c++17", "-I", build_lib.CSRC, str(src), "-o", str(tmp_path / "once")], check=True)
    out = subprocess.run([str(tmp_path / "once")], capture_output=True, text=True, check=True).stdout
    assert out.split() == ["01", "02", "13", "13", "14", "14", "14", "05", "15"]


@pytest.mark.parametrize("name", ["wq_attn.cu", "wq_attn_tc.cu", "wq_block_norm.cu"])
def test_no_kernel_keeps_its_set_up_for_the_process(name):
    text = open(os.path.join(build_lib.CSRC, name)).read()
    assert "allow_smem(sized" in text and not re.search(r"static bool|cudaFuncSetAttribute", text)
