"""Growing scratch buffers (csrc/grow.h) with an allocator that is made to fail."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "%s"
#include <assert.h>
#include <stdio.h>
#include <set>
using namespace adp;
std::set<float*> live;
int made = 0, fail_at = -1, stuck = 0;
int grow_(Grown<float>* b, size_t n) {
  return grow(b, n,
      [](float** p, size_t count) { if (made++ == fail_at) return 7; live.insert(*p = new float[count]); return 0; },
      [](float* p) { if (stuck) return 5; assert(live.erase(p) == 1); delete[] p; return 0; });
}
int main() {
  Grown<float> a, b;
  assert(grow_(&a, 0) == 0 && !a.p);
  assert(grow_(&a, 10) == 0 && a.n == 10 && grow_(&b, 10) == 0 && live.size() == 2);
  float* was = a.p;
  assert(grow_(&a, 10) == 0 && grow_(&a, 3) == 0 && a.p == was && a.n == 10);  // large enough
  fail_at = made;
  assert(grow_(&a, 20) == 7 && !a.p && a.n == 0 && live.size() == 1);  // the old one is gone, and so is its size
  assert(b.p && b.n == 10);                                             // the other one is untouched
  assert(grow_(&a, 10) == 0 && a.p && a.n == 10 && live.count(a.p));    // and what fitted before is made again
  stuck = 1;
  was = a.p;
  assert(grow_(&a, 20) == 5 && a.p == was && a.n == 10);
  stuck = 0;
  assert(grow_(&a, 20) == 0 && a.n == 20 && live.size() == 2);
  puts("ok");
}
"""


def test_a_buffer_that_could_not_grow_is_made_again(tmp_path):
    src, exe = tmp_path / "grow.cpp", tmp_path / "grow"
    src.write_text(PROGRAM % os.path.join(ROOT, "autoregressive_decode_persistent_gb300", "csrc", "grow.h"))
    subprocess.run(["g++", "-O1", "-std=c++17", str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"
