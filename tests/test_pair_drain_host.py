"""Shutting down the product kernel's pipeline after a wait that ran out, on the CPU.

A model of the leader's barriers (arrivals and announced bytes of each slot) goes
through every pair of counts at which the two CTAs can have stopped, with the drain's
accounting compiled from the kernel's own header.  Each wait must end, and no load of
either CTA may be outside the stages that are waited for or known to be used.
"""
import shutil
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "mx_block_quantization_gb300" / "csrc"

MODEL = r'''
#include <cstdio>
#include <vector>
#include "pair_drain.h"
using namespace mxq;
constexpr int kHalf = 32768;
struct Barrier {  // one arrival a phase, bytes announced and not yet loaded
  int phase = 0, arrivals = 1;
  long tx = 0;
  void settle() { if (arrivals == 0 && tx == 0) ++phase, arrivals = 1; }
  void expect(long b) { tx += b; --arrivals; settle(); }
  void complete(long b) { tx -= b; settle(); }
  bool passed(int parity) const { return (phase & 1) != parity; }
};
int main() {
  int bad = 0, cases = 0;
  for (int stages = 2; stages <= 6; ++stages)
    for (int used = 0; used < 14; ++used)                    // stages the products were done with
      for (int own = used; own <= used + stages; ++own)
        for (int peer = used; peer <= used + stages; ++peer) {
          ++cases;
          std::vector<Barrier> full(stages);
          const int most = own < peer ? peer : own;
          for (int n = 0; n < most; ++n) {  // the peer's bytes may be there first
            Barrier& b = full[n % stages];
            if (n < peer) b.complete(kHalf);
            if (n < own) { b.expect(2 * kHalf); b.complete(kHalf); }
            if (n < used && b.phase != n / stages + 1) ++bad;  // the model itself
          }
          const PairDrain r = pair_drain(own, peer, stages);
          if (r.first > used || r.end != most) ++bad;        // a load that nobody waits for
          for (int n = r.first; n < r.end; ++n) {
            Barrier& b = full[n % stages];
            if (pair_unannounced(n, own)) b.expect(kHalf);
            if (pair_half_missing(n, peer)) b.complete(kHalf);
            if (!b.passed(n / stages & 1) || b.phase < n / stages + 1) ++bad;
          }
          for (const Barrier& b : full) if (b.tx != 0 || b.arrivals != 1) ++bad;
        }
  std::printf("cases %d bad %d\n", cases, bad);
  return bad != 0;
}
'''


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a C++ compiler")
def test_every_wait_ends_and_every_load_is_waited_for(tmp_path):
    (tmp_path / "model.cpp").write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", str(tmp_path / "model.cpp"), "-o", str(tmp_path / "model")],
                   check=True, timeout=120)
    r = subprocess.run([str(tmp_path / "model")], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.endswith("bad 0\n"), r.stdout
