"""When the kernels' waits are given up: the rule of csrc/waits.h, compiled for the host."""
import shutil
import subprocess

import pytest

from mxfp8_master_weight_gb300 import build

PROGRAM = r"""
#include <cassert>
#include <initializer_list>
#include "waits.h"
using namespace mxfp8::tc;

// Looks every `step` cycles until the wait is given up; the cycles counted from `from` on.
static unsigned long long lasts(unsigned step, unsigned from) {
  Patience p{from};
  unsigned long long t = 0;
  do t += step; while (!p.out(unsigned(from + t)) && t < 100 * 1000000000ull);
  return t;
}

int main() {
  // looked at all the time, a wait ends after kWaitCycles, wherever the clock stood
  for (unsigned from : {0u, 1u << 31, 0xffffffffu, 0xf0000000u})
    for (unsigned step : {1000000u, 4000003u, kPollCycles}) {
      const unsigned long long t = lasts(step, from);
      assert(t > kWaitCycles && t <= kWaitCycles + (unsigned long long)step);
    }
  // a pause of any length, the clock wrapped or not, counts as one interval: the wait goes on
  for (unsigned pause : {kWaitCycles, kWaitCycles + 1, 0xffffffffu, 1u << 31, kPollCycles + 1}) {
    Patience p{12345u};
    unsigned now = 12345u;
    assert(!p.out(now += 1000) && !p.out(now += pause) && !p.out(now += 1000));
    assert(p.spent == 2000 + kPollCycles);
  }
  // paused again and again for ten seconds between looks it still ends, after enough looks
  Patience p{0};
  unsigned now = 0, looks = 1;
  while (!p.out(now += 20000000000ull % (1ull << 32))) assert(++looks < 1000);
  assert(looks > 200);
  return 0;
}
"""


def test_patience(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", f"-I{build.CSRC}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
