"""The library keeps a device's kind once it knows it, and only then (host code, with a fake of the
device's queries)."""
import os
import shutil
import subprocess

import pytest

import block_sparse_gqa_topk_gb300 as pkg

PROGRAM = r"""
#include "device_kind.h"
#include <cstdio>
using namespace msa;
int main() {
  int fails = 0, asked = 0;
  auto check = [&](const char* what, int got, int want) {
    if (got != want) { std::printf("%s: %d, not %d\n", what, got, want); ++fails; }
  };
  for (int broken = 0; broken < 3; ++broken) {  // each of the three queries fails once
    for (int kind = 0; kind < 2; ++kind) {
      std::atomic<int> kept{0};
      bool down = true;
      auto query = [&](DeviceAttr a, int* v) {
        ++asked;
        if (down && (int)a == broken) return false;
        *v = a == DeviceAttr::kSmCount ? 152 : a == DeviceAttr::kMajor ? 10 : kind == 0 ? 3 : 0;
        return true;
      };
      check("failed query", sm_count_of(&kept, query), 0);
      check("kept after it", kept.load(), 0);
      down = false;
      const int want = kind == 0 ? 152 : -1;
      check("answer", sm_count_of(&kept, query), want);
      asked = 0;
      down = true;
      check("kept answer", sm_count_of(&kept, query), want);
      check("queries for it", asked, 0);
    }
  }
  return fails != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_only_answers_are_kept(tmp_path):
    src, exe = tmp_path / "kind.cpp", tmp_path / "kind"
    src.write_text(PROGRAM)
    csrc = os.path.join(os.path.dirname(pkg.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", csrc, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
