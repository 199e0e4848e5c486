"""The record mover of the compaction on the host: its copies replaced by a model that checks
their order, with every load in turn never landing."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_gemv_packkv_b200", "csrc")

MODEL = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "mover.cuh"
using packkv::kMoveStages;

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s (lost %ld of %ld)\n", __LINE__, #x, lost, total); std::exit(1); } } while (0)

static long total, lost;  // the load that never lands (-1: all do)

struct Load { int stage; long to; bool waited, stored, read; };
struct Model {
  std::vector<Load>* loads;
  std::vector<long>* stores;  // load numbers, in order
  int* gave_up;
  long on_stage(int s) { for (long i = (long)loads->size() - 1; i >= 0; --i) if ((*loads)[i].stage == s) return i; return -1; }
  void load(int s, const void* from, uint32_t bytes) {
    long n = (long)loads->size();
    CHECK(s == n % kMoveStages && from == (const void*)(16 * (n + 1)) && bytes == 16u * (n + 1));
    const long old = on_stage(s);
    CHECK(old < 0 || (*loads)[old].read);  // nobody still reads the stage
    loads->push_back({s, 0, false, false, false});
  }
  bool landed(int s, uint32_t phase) {
    const long i = on_stage(s);
    CHECK(i >= 0 && phase == ((i / kMoveStages) & 1));  // a load that was issued
    CHECK(!(*loads)[i].waited);
    (*loads)[i].waited = true;
    if (i == lost) ++*gave_up;
    return i != lost;
  }
  void store(int s, void* to, uint32_t bytes) {
    const long i = on_stage(s);
    CHECK(i != lost && (*loads)[i].waited && !(*loads)[i].stored);
    CHECK(to == (void*)(32 * (i + 1)) && bytes == 16u * (i + 1));
    (*loads)[i].stored = true;
    stores->push_back(i);
  }
  void await_reads() { for (size_t k = 0; k + 1 < stores->size(); ++k) (*loads)[(*stores)[k]].read = true; }
  void await_stores() { for (long i : *stores) (*loads)[i].read = true; }
};

int main() {
  for (total = 0; total < 14; ++total)
    for (lost = -1; lost < total; ++lost) {
      std::vector<Load> loads;
      std::vector<long> stores;
      int gave_up = 0;
      packkv::Mover<Model> m{{&loads, &stores, &gave_up}, 0, nullptr, 0u, false};
      for (long i = 0; i < total; ++i) m.move((void*)(32 * (i + 1)), (const void*)(16 * (i + 1)), 16u * (i + 1));
      m.finish();
      for (const Load& x : loads) CHECK(x.waited);             // none lands behind the end
      for (long i : stores) CHECK(loads[i].read);
      CHECK(gave_up == (lost >= 0));
      const long good = lost < 0 ? total : lost;
      CHECK((long)stores.size() == good);                        // everything before the lost one
      for (long i = 0; i < good; ++i) CHECK(stores[i] == i);
    }
  return 0;
}
"""


def test_every_load_is_waited_for(tmp_path):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "model.cc", tmp_path / "model"
    src.write_text(MODEL)
    r = subprocess.run([cc, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(exe), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
