"""The copies that a copying warp leaves behind: whichever wait for room runs out, every copy issued has been waited for when
its CTA leaves (csrc/spg_ring.cuh, compiled here for the CPU and run against a model of the ring)."""

import os
import subprocess

import query_aware_sparse_page_gb300._build as build

PROGRAM = r"""
#define __host__
#define __device__
#define __forceinline__ inline
#include "spg_ring.cuh"
#include <cstdio>
#include <set>
#include <tuple>

using Copy = std::tuple<uint32_t, int, uint32_t>;  // stage, part, phase

// `steps` steps of two parts, the wait number `fail` of those for room running out; what is left in flight at the end.
// by_steps: the drain counts whole steps alone.
template <int ST>
int left(int steps, int fail, bool by_steps) {
  spg::PartRing<ST, 2> ring;
  std::set<Copy> flying;
  int waits = 0, whole = 0;
  bool ok = true;
  for (int k = 0; ok && k < steps; ++k) {
    for (int part = 0; part < 2; ++part)
      ok = ok && ring.put(
          part,
          [&](uint32_t stage, uint32_t phase) {
            if (waits++ == fail) return false;
            flying.erase(Copy(stage, part, phase));  // read, so it has landed
            return true;
          },
          [&](uint32_t stage) { flying.insert(Copy(stage, part, ring.n[part] / ST)); });
    whole += ok;
  }
  if (by_steps) ring.n[0] = ring.n[1] = whole;
  ring.drain([&](uint32_t stage, int part, uint32_t phase) { flying.erase(Copy(stage, part, phase)); });
  return static_cast<int>(flying.size());
}

int main() {
  int old = 0;
  for (int steps = 0; steps < 14; ++steps)
    for (int fail = -1; fail < 2 * steps; ++fail) {
      if (left<2>(steps, fail, false) || left<4>(steps, fail, false)) {
        std::printf("steps %d, wait %d ran out: a copy is left\n", steps, fail);
        return 1;
      }
      old += left<2>(steps, fail, true) + left<4>(steps, fail, true);
    }
  std::printf("%d\n", old);
  return 0;
}
"""


def test_every_copy_issued_is_waited_for(tmp_path):
    (tmp_path / "ring.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "ring")
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{build.CSRC}", "-o", exe, str(tmp_path / "ring.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    # the model sees the fault: counted by whole steps, the first part of the step that failed would be left
    assert int(r.stdout) > 0


def test_the_latent_attention_kernel_counts_its_copies_so():
    with open(os.path.join(build.CSRC, "spg_latent_attention.cu"), encoding="utf-8") as f:
        code = f.read()
    body = code[code.index("void load_kv(") : code.index("void softmax(")]
    assert body.count("ring.put(") == 1 and body.count("tma_tile_4d(") == 1 and body.count("ring.drain(") == 1
