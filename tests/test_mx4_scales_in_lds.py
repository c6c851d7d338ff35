"""Where the 4-bit tiles keep a row's scales in LDS (host only): for every number of
words a row can have and every stage, the eight bytes that are read (and cleared, where K
cuts them) are the stage's words, and what they take in of the next row is unused there
and has room behind the last row."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "conv_qpack_weights_amd", "csrc")

PROGRAM = r"""
#include "mx4_scales.hpp"
#include <cstdio>
using namespace qp;
static int bad(const char* what, bool wide, int G, int s) {
  std::printf("%s: wide=%d blocks=%d stage=%d\n", what, wide, G, s);
  return 1;
}
int main() {
  for (int wide = 0; wide < 2; ++wide)
    for (int G = wide ? 13 : 1; G <= (wide ? 4200 : 12); ++G) {
      const int words = (G + 3) / 4, stages = (G + 7) / 8, full = G / 8;
      for (int s = 0; s <= stages; ++s) {
        // a stage is read if it is one, and ahead of the loop's even ends
        if (s == stages && s != full / 2 * 2) continue;
        const int span = (s >> 1) * 4, over = mx_scales_over(words);
        const int late = wide && mx_scales_end(s) > words ? over : 0;
        const int at = mx_scales_at(s) + late, past = at + 8 - kMxScaleRow;
        if (at < 0 || at % 4 || past > 4) return bad("place", wide, G, s);
        if (past > kMxScaleRoom) return bad("no room behind the last row", wide, G, s);
        if (past > late) return bad("bytes of the next row in use", wide, G, s);
        if (s >= stages) continue;
        // the load of the span, as words of the row: none before its first or past its
        // last, and the stage's words where they are read
        if (wide) {
          const int first = span - late / 4;
          if (first < 0 || first + 4 > words) return bad("load outside the scales", wide, G, s);
          for (int w = 0; w < 2; ++w) {
            const int word = span + (s & 1) * 2 + w;
            if (word >= words) continue;
            if (at + 4 * w >= kMxScaleRow) return bad("a word is missed", wide, G, s);
            if (at + 4 * w != 4 * (word - first)) return bad("another word", wide, G, s);
          }
        } else if (at != (s & 1) * 8) {
          return bad("narrow place", wide, G, s);
        }
      }
    }
  return 0;
}
"""


def test_scales_have_their_places(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "scales.cpp", tmp_path / "scales"
    src.write_text(PROGRAM)
    subprocess.check_call([cxx, "-std=c++17", "-Wall", "-I", CSRC, str(src), "-o", str(exe)])
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
