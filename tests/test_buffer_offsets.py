"""Loads past a buffer's end, by the range check of raw buffers (no GPU needed).

An offset is past the end if voff >= bytes - soff, in unsigned 32 bits. The
streams of the expert layer issue loads for tiles past an expert's last one and
for spans that a wave has not; those have to be past the end by that rule, with
no difference that wraps, and all others inside. bsq_lds.h's buffer_at decides
it: it is compiled for the host and called as the streams call it."""
import subprocess

import pytest

from block_scaled_bit_quantize_amd import build as B

PROGRAM = r"""
#include "bsq_lds.h"
#include <cstdio>
#include <cstdlib>
using bsqd::buffer_at;
static long bad, all;
static void check(bool wanted, bsqd::BufferAt at, uint32_t bytes, uint32_t size) {
  const bool wraps = at.soff > bytes;
  const bool read = at.voff < (uint32_t)(bytes - at.soff);
  const bool inside = (uint64_t)at.voff + at.soff + size <= bytes;
  ++all;
  if (wraps || read != wanted || (wanted && !inside)) ++bad;
}
// k_moe_stream (wide: 32 outputs a tile, W2; else 16 and their up rows) and k_moe_last (16 outputs a tile), whole spans
int main(int argc, char** argv) {
  const int width = atoi(argv[1]), K = atoi(argv[2]), waves = 8, ring = 6;
  const int nblk = K / 16, pitch = nblk * 8, spans = K / 256;
  for (int kind = 0; kind < 3; ++kind) {
    const int out = kind == 1 ? 32 : 16, up = kind == 0 ? width : 16, rows = kind == 0 ? 2 * width : width;
    const int tiles = (width + out - 1) / out, most = (spans + waves - 1) / waves;
    for (int wave = 0; wave < waves; ++wave) {
      const int sp0 = spans * wave / waves, cnt = spans * (wave + 1) / waves - sp0;
      for (int tile = 0; tile < tiles + ring; ++tile)
        for (int s = 0; s < most; ++s) {
          const bool some = tile < tiles && s < cnt, both = kind != 1 || tile * out + 16 < width;
          const int span = sp0 + s;
          for (int lane = 0; lane < 64; ++lane)
            for (int b = 0; b < (kind == 2 ? 2 : 4); ++b) {
              const int c = (b & 1) * 8 + (lane >> 3);
              const uint32_t v = (uint32_t)(c + (b >> 1) * up) * pitch + (lane & 7) * 16;
              check(some && (both || b < 2),
                    buffer_at(some, both || b < 2, v, (uint32_t)(tile * out) * pitch + span * 128), (uint32_t)rows * pitch, 16);
            }
        }
    }
  }
  printf("%ld %ld\n", bad, all);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("offsets")
    (d / "p.hip").write_text(PROGRAM)
    r = subprocess.run([B.HIPCC, "--offload-host-only", "-std=c++17", "-O1", "-I", B.CSRC, str(d / "p.hip"), "-o",
                        str(d / "p")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return str(d / "p")


@pytest.mark.parametrize("width,K", [(16, 256), (48, 512), (1536, 4096), (4096, 1536), (2048, 7168), (32768, 4096)])
def test_streams_past_the_end(program, width, K):
    bad, loads = map(int, subprocess.run([program, str(width), str(K)], capture_output=True, text=True,
                                         check=True).stdout.split())
    assert loads > 1000 and bad == 0
