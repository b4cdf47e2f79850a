"""How the product reads scales (csrc/xp_scales.h), compiled for the host: every block's byte, and nothing behind
the last row's."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "collective_transport_plane_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "xp_scales.h"
int main() {
  for (unsigned rows = 1; rows <= 3; ++rows)
    for (unsigned blocks = 1; blocks <= 9; ++blocks) {
      const unsigned pitch = (blocks + 3) / 4 * 4, size = (rows - 1) * pitch + blocks;
      uint8_t* scales = static_cast<uint8_t*>(malloc(size));   // what is behind it is watched
      for (unsigned i = 0; i < size; ++i) scales[i] = (uint8_t)(17 * i + 3);
      for (unsigned r = 0; r < rows; ++r)
        for (unsigned g = 0; 4 * g < blocks; ++g) {
          const unsigned w = xp::scale_word(scales + r * pitch, g, blocks, r + 1 == rows);
          for (unsigned i = 0; i < 4 && 4 * g + i < blocks; ++i)
            if ((w >> 8 * i & 255) != scales[r * pitch + 4 * g + i]) return printf("row %u, block %u of %u\n", r, 4 * g + i, blocks), 1;
        }
      free(scales);
    }
  return puts("equal"), 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("scales")
    (at / "t.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-g", "-fsanitize=address", "-I", CSRC, "-o", str(at / "t"), str(at / "t.cpp")], check=True)
    return str(at / "t")


def test_scales_are_read_to_their_end_and_no_further(program):
    done = subprocess.run([program], capture_output=True, text=True, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert done.returncode == 0 and done.stdout == "equal\n", done.stdout + done.stderr[:2000]
