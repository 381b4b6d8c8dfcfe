"""How a CTA of the 4-bit attention that gave up ends its copies (end_copies in csrc/kv4.h),
run on the host with its barriers played: every wait has to end, however far apart the two
copying warps stopped."""
import os
import shutil
import subprocess

import pytest

from sparse_verification_attention_gb300 import build_lib

PLAY = r"""
#include <cstdio>
#include <vector>
#include "kv4.h"

// An mbarrier of two arrivals a phase, all of whose bytes have landed.
struct Bar {
  uint32_t pending = 2, phases = 0;
  void arrive() {
    if (--pending == 0) pending = 2, ++phases;
  }
  bool done(uint32_t parity) const { return (phases & 1) != parity; }
};

int main() {
  int runs = 0, stuck = 0, wrong = 0, apart = 0;
  for (uint32_t stages = 1; stages <= 8; ++stages)
    // `used` tiles were taken out of the ring; either warp is at most `stages` tiles ahead
    for (uint32_t used = 0; used <= 20; ++used)
      for (uint32_t k = used; k <= used + stages; ++k)
        for (uint32_t v = used; v <= used + stages; ++v) {
          std::vector<Bar> full(stages);
          for (uint32_t i = 0; i < k || i < v; ++i) {
            if (i < k) full[i % stages].arrive();
            if (i < v) full[i % stages].arrive();
          }
          const std::vector<Bar> before = full;
          bool stays = false;  // without the arrivals some wait would not end
          for (uint32_t i = 0; i < k || i < v; ++i)
            if (i + stages >= (k > v ? k : v) && !before[i % stages].done(i / stages & 1)) stays = true;
          apart += k != v;
          if (stays != (k != v)) ++wrong;
          sva::end_copies(k, v, stages, [&](uint32_t st) { full[st].arrive(); },
                          [&](uint32_t st, uint32_t parity) { stuck += !full[st].done(parity); });
          for (uint32_t st = 0; st < stages; ++st) {  // exactly the tiles that were begun
            uint32_t n = 0;
            for (uint32_t i = st; i < k || i < v; i += stages) ++n;
            if (full[st].phases != n || full[st].pending != 2) ++wrong;
          }
          ++runs;
        }
  std::printf("%d %d %d %d\n", runs, apart, stuck, wrong);
}
"""


def test_every_wait_ends(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "play.cc", tmp_path / "play"
    src.write_text(PLAY)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build_lib.nvcc()))), "include")
    r = subprocess.run([cxx, "-std=c++17", "-w", "-I", build_lib.CSRC, "-I", build_lib.INCLUDE, "-I", cuda,
                        str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    runs, apart, stuck, wrong = map(int, subprocess.run([str(exe)], capture_output=True, text=True).stdout.split())
    assert runs > 5000 and apart > 4000 and stuck == 0 and wrong == 0
