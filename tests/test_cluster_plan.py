"""The FP8 projection's choice of how many CTAs share a tile's K, and the answers of the device that it keeps: the host code,
compiled by itself and driven with answers of a device that is not there. CPU only."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_07_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "at_once.h"
using msa::AtOnce;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

static AtOnce cache, other, shared;

int main() {
  int asked = 0;
  // a failure is not kept, an answer is, and zero is one
  CHECK(cache.get(0, 4, [&] { ++asked; return -1; }) == -1);
  CHECK(cache.get(0, 4, [&] { ++asked; return 36; }) == 36);
  CHECK(cache.get(0, 4, [&] { ++asked; return 99; }) == 36 && asked == 2);
  CHECK(cache.get(0, 8, [&] { ++asked; return 0; }) == 0 && cache.get(0, 8, [&] { ++asked; return 5; }) == 0 && asked == 3);
  // devices, sizes and kernels are apart; what has no place is asked for every time
  CHECK(cache.get(1, 4, [] { return 7; }) == 7 && cache.get(0, 2, [] { return 8; }) == 8 && other.get(0, 4, [] { return 9; }) == 9);
  for (int n : {-1, 9}) CHECK(cache.get(0, n, [] { return 3; }) == 3 && cache.get(0, n, [] { return 4; }) == 4);
  for (int d : {-1, 64}) CHECK(cache.get(d, 1, [] { return 3; }) == 3 && cache.get(d, 1, [] { return 4; }) == 4);

  // the cheapest split; those that the device has no room for are left out, forced ones too
  float us = 0.f;
  auto cost = [](int s, int room) { return 10.f / s + 100.f / room; };
  CHECK(msa::cheapest_split(8, 0, true, [](int) { return 10; }, cost, us) == 8);
  CHECK(msa::cheapest_split(8, 0, true, [](int s) { return s > 4 ? 0 : 10; }, cost, us) == 4 && us == 12.5f);
  CHECK(msa::cheapest_split(8, 0, true, [](int s) { return s == 4 ? -1 : s > 4 ? 0 : 10; }, cost, us) == 3);
  CHECK(msa::cheapest_split(8, 8, true, [](int s) { return s == 8 ? 0 : 10; }, cost, us) == 7);
  CHECK(msa::cheapest_split(8, 2, true, [](int) { return 10; }, cost, us) == 2 && us == 15.f);
  CHECK(msa::cheapest_split(4, 5, true, [](int) { return 10; }, cost, us) == 4);
  CHECK(msa::cheapest_split(8, 3, true, [](int) { return 0; }, cost, us) == 0);
  auto same = [](int, int) { return 1.f; };
  CHECK(msa::cheapest_split(8, 0, true, [](int) { return 1; }, same, us) == 8 && msa::cheapest_split(8, 0, false, [](int) { return 1; }, same, us) == 1);

  // many threads, some of whose questions fail
  std::vector<std::thread> threads;
  std::atomic<int> wrong{0};
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&, t] {
      for (int i = 0; i < 20000; ++i) {
        const int n = i % 9, v = shared.get(t % 3, n, [&] { return (i + t) % 5 == 0 ? -1 : 10 * n; });
        if (v != 10 * n && v != -1) ++wrong;
      }
    });
  for (auto& t : threads) t.join();
  CHECK(wrong == 0);
  for (int n = 0; n < 9; ++n) CHECK(shared.get(2, n, [] { return 777; }) == 10 * n);
  return 0;
}
"""


def test_kept_answers_and_choice(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
