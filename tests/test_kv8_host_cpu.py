"""Host parts of the 8-bit paged cache that need no GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PER_DEVICE = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"

static PerDevice known;
static std::atomic<int> asked;
static int sms(int dev) {
  return per_device(known, dev, [](int d) { ++asked; return d == 5 ? 0 : 100 + d; });
}
int main() {
  // each device has its own number, asked once; devices past the last slot and failures are asked again
  for (int pass = 0; pass < 3; ++pass)
    for (int d : {1, 0, 7, 63})
      if (sms(d) != 100 + d) return 1;
  if (asked != 4) return 2;
  for (int pass = 0; pass < 2; ++pass)
    if (sms(64) != 164 || sms(1000) != 1100 || sms(5) != 0) return 3;
  if (asked != 10) return 4;
  std::vector<std::thread> all;
  std::atomic<int> wrong{0};
  for (int t = 0; t < 16; ++t)
    all.emplace_back([&wrong] {
      for (int i = 0; i < 20000; ++i) wrong += sms(20 + i % 40) != 120 + i % 40;
    });
  for (auto& t : all) t.join();
  return wrong ? 5 : 0;
}
"""


def test_numbers_are_kept_for_each_device(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "p.cc", tmp_path / "p"
    src.write_text(PER_DEVICE)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-pthread", "-I",
                    os.path.join(ROOT, "scratch_decoder_only_b200", "csrc"), str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_an_unknown_kind_is_refused():
    from scratch_decoder_only_b200.kv8 import KV8Cache
    with pytest.raises(ValueError):
        KV8Cache.empty(1, 8, 2, 64, kind="fp8", device="cpu")
