"""The TMA producers' loop (csrc/ring.cuh, feed_ring), compiled for the host
against a model of a ring: one step at a time a copy lands, the consumer
releases a slot, or the consumer gives up (a bounded wait of its own ran out).
Whatever the order, the slots are used one round at a time and nothing is in
flight when the producer returns."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_nf4_quantized_20_b200", "csrc")

HARNESS = r"""
#include "ring.cuh"
#include <cstdio>
#include <deque>
#include <random>
#include <vector>

// One run: `n` steps through `stages` slots, of which `lead` are issued before
// the loop; the consumer gives up before its step `give_up`; copies land when
// someone waits for them, or at random.  Returns 0, or what went wrong.
static int run(int n, int stages, int lead, int give_up, bool stuck, unsigned seed) {
  std::mt19937 rng(seed);
  struct Slot {
    int issued = 0, landed = 0, released = 0;   // rounds
  };
  std::vector<Slot> slot(stages);
  std::deque<int> flying;   // slots with a copy on its way, oldest first
  int consumed = 0, bad = 0;
  bool aborted = false;
  auto start = [&](int s, int st) {
    if (s != st % stages || slot[s].issued != st / stages || slot[s].released != slot[s].issued) bad = 1;
    ++slot[s].issued;
    flying.push_back(s);
  };
  auto land = [&] {
    if (flying.empty()) return;
    const int s = flying.front();
    flying.pop_front();
    ++slot[s].landed;
  };
  auto consume = [&] {   // one step of the consumer, if its slot is full
    if (aborted || consumed == n) return;
    if (consumed >= give_up) {
      aborted = true;
      return;
    }
    const int s = consumed % stages;
    if (slot[s].landed > consumed / stages) {
      ++slot[s].released;
      ++consumed;
    }
  };
  auto others = [&] {
    for (int k = static_cast<int>(rng() % 4); k > 0; --k) (rng() & 1) ? land() : consume();
  };
  for (int st = 0; st < lead; ++st) start(st, st);
  others();
  qlora::feed_ring(
      lead, n, stages,
      [&](int s, unsigned parity) {
        others();
        // the parity that completes with the release of the round before
        if (parity != ((slot[s].issued & 1) ^ 1)) bad = 2;
        for (int i = 0; i < 1000 && slot[s].released < slot[s].issued && !aborted; ++i) (i & 1) ? land() : consume();
        return !aborted && slot[s].released == slot[s].issued;
      },
      [&](int s, int st) { start(s, st); },
      [&](int s, unsigned parity) {
        others();
        if (parity != ((slot[s].issued - 1) & 1)) bad = 3;
        if (stuck) return false;   // this wait runs out
        while (slot[s].landed < slot[s].issued && !flying.empty()) land();
        return slot[s].landed == slot[s].issued;
      });
  if (bad) return bad;
  if (stuck) return 0;
  if (!flying.empty()) return 4;   // the CTA would leave with copies on their way
  if (give_up >= n) {
    int all = 0;
    for (const Slot &s : slot) all += s.issued;
    if (all != n) return 5;        // nobody gave up: every step has to be issued
  }
  return 0;
}

int main() {
  for (int stages = 1; stages <= 6; ++stages)
    for (int n = 1; n <= 3 * stages + 1; ++n)
      for (int lead : {0, stages < n ? stages : n})
        for (int give_up = 0; give_up <= n; ++give_up)
          for (unsigned seed = 0; seed < 20; ++seed)
            for (int stuck = 0; stuck < 2; ++stuck)
              if (const int e = run(n, stages, lead, give_up, stuck != 0, seed)) {
                std::printf("fault %d: stages %d steps %d lead %d give_up %d seed %u stuck %d\n", e, stages, n, lead,
                            give_up, seed, stuck);
                return 1;
              }
  std::printf("ok\n");
  return 0;
}
"""


def test_no_copy_is_in_flight_when_the_producer_returns(tmp_path):
    cxx = os.environ.get("CXX", "g++")
    if shutil.which(cxx) is None:
        pytest.skip("no host compiler")
    src = tmp_path / "main.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "ring"
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("name", ["int8_gemm.cu", "int8_decode.cu", "da_int8.cu", "skinny_tc.cu"])
def test_the_one_cta_kernels_use_it(name):
    with open(os.path.join(CSRC, name)) as f:
        assert f.read().count("feed_ring(") == 1


@pytest.mark.parametrize("name", ["int8_gemm_2sm.cu", "gemm_fwd_2sm.cu", "gemm_dx_2sm.cu"])
def test_the_pair_kernels_settle_after_their_last_barrier(name):
    """A pair kernel's loads are counted in the other CTA's barriers too, so it
    gives them time instead -- where any warp's wait ran out, not the
    producer's alone: after the barrier that brings all warps' findings
    together, and before the CTA may leave."""
    with open(os.path.join(CSRC, name)) as f:
        code = [line.split("//")[0].strip() for line in f]
    code = [line for line in code if line]
    at = [i for i, line in enumerate(code) if line.startswith("settle_loads(")]
    assert [code[i] for i in at] == ["settle_loads(s_abort != 0);"]
    assert code[at[0] - 1] == "__syncthreads();" and code[at[0] + 1] == "cluster_arrive_wait();"
    # every role that stops early has said so before that barrier
    assert sum(line == "if (!ok) s_abort = 1;" for line in code[:at[0]]) >= 3
