"""The places that recorded launches keep (csrc/slot_pool.hpp), compiled for the host."""
import os
import subprocess

from _lib import ROOT

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>
#include "slot_pool.hpp"
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } } while (0)
static slope::SlotPool<192> pool;
static slope::SlotPool<65536> large;
int main() {
  for (int round = 0; round < 3; ++round) {
    std::vector<bool> seen(192, false);
    for (int i = 0; i < 192; ++i) {
      const uint32_t k = pool.take();
      CHECK(k < 192 && !seen[k]);
      seen[k] = true;
    }
    CHECK(pool.take() == 192 && pool.take() == 192);      // none is handed out twice
    for (uint32_t k : {7u, 100u, 191u, 0u}) pool.give_back(k);
    seen.assign(192, false);
    for (int i = 0; i < 4; ++i) seen[pool.take()] = true;
    CHECK(seen[7] && seen[100] && seen[191] && seen[0] && pool.take() == 192);
    for (int k = 0; k < 192; ++k) pool.give_back(k);
  }
  // one that is kept stays out of all later rounds; what is given back comes again last
  const uint32_t kept = pool.take();
  uint32_t last = kept;
  for (int i = 0; i < 1000; ++i) {
    const uint32_t k = pool.take();
    CHECK(k < 192 && k != kept && k != last);
    pool.give_back(k);
    last = k;
  }
  // threads
  std::vector<std::vector<uint32_t>> got(8);
  std::vector<std::thread> threads;
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&, t] {
      for (int i = 0; i < 8192 + 100; ++i) {
        const uint32_t k = large.take();
        if (k < 65536) got[t].push_back(k);
      }
    });
  for (auto& t : threads) t.join();
  std::vector<bool> seen(65536, false);
  size_t n = 0;
  for (auto& g : got)
    for (uint32_t k : g) {
      CHECK(!seen[k]);
      seen[k] = true;
      ++n;
    }
  CHECK(n == 65536 && large.take() == 65536);
  return 0;
}
"""


def test_places_are_kept_until_given_back(tmp_path):
    src, exe = tmp_path / "pool.cpp", tmp_path / "pool"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-pthread", "-I",
                           os.path.join(ROOT, "ring_attention_slope_gb300", "csrc"), str(src), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout
