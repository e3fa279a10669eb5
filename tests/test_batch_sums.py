"""Running sums over more sequences than a CTA has threads (csrc/batch_sums.h), compiled for the host:
threads stand for warps of one lane, and each in turn is held up behind a barrier while the others
go on into the next pass.  A slot that is written again before a slow warp has read it gives a wrong sum."""
import os
import shutil
import subprocess

import pytest

from hybrid_linear_attention_gb300 import build as kbuild

PROGRAM = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <thread>
#include <vector>
#include "batch_sums.h"

constexpr int WARPS = 6;
std::mutex m;
std::condition_variable cv;
int arrived = 0, phase = 0, slow = 0;

struct Cta {
  int w;
  int warp() const { return w; }
  bool last_lane() const { return true; }
  long long inclusive(long long x) const { return x; }
  void barrier() const {
    {
      std::unique_lock<std::mutex> l(m);
      const int mine = phase;
      if (++arrived == WARPS) arrived = 0, ++phase, cv.notify_all();
      else cv.wait(l, [&] { return phase != mine; });
    }
    if (w == slow) std::this_thread::sleep_for(std::chrono::milliseconds(20));
  }
};

int main() {
  const int passes = 5, n = passes * WARPS - 2;
  auto value = [&](int i) { return i < n ? 7ll * i * i + 3 : 0ll; };
  int bad = 0;
  for (slow = 0; slow < WARPS; ++slow) {
    kda::PassSums<WARPS> sums;
    std::vector<std::thread> t;
    std::vector<int> wrong(WARPS, 0);
    for (int w = 0; w < WARPS; ++w)
      t.emplace_back([&, w] {
        const Cta cta{w};
        int pass = 0;
        for (int round = 0; round < 2; ++round) {  // over the batch, and over it again
          long long before = 0, want = 0;
          for (int p = 0; p < passes; ++p) {
            const long long at = kda::sum_pass(cta, sums, pass, value(p * WARPS + w), before);
            long long here = want;
            for (int x = 0; x < w; ++x) here += value(p * WARPS + x);
            for (int x = 0; x < WARPS; ++x) want += value(p * WARPS + x);
            wrong[w] += at != here || before != want;
          }
        }
      });
    for (auto &x : t) x.join();
    for (int w = 0; w < WARPS; ++w) bad += wrong[w];
  }
  std::printf("%d\n", bad);
  return 0;
}
"""


def wrong_sums(tmp_path, header):
    """Wrong results of the program above with that text as batch_sums.h."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "batch_sums.h").write_text(header)
    (tmp_path / "main.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", str(tmp_path), str(tmp_path / "main.cpp"), "-o", str(tmp_path / "main")],
                   check=True)
    return int(subprocess.run([str(tmp_path / "main")], capture_output=True, text=True, check=True, timeout=120).stdout)


def header():
    with open(os.path.join(kbuild.CSRC, "batch_sums.h")) as f:
        return f.read()


def test_a_slow_warp_reads_its_own_pass(tmp_path):
    assert wrong_sums(tmp_path, header()) == 0


def test_one_place_for_the_sums_would_be_seen(tmp_path):
    """The same with a single place for all passes, as it was: the slow warps' sums are wrong."""
    text = header()
    assert text.count("pass++ & 1") == 1
    assert wrong_sums(tmp_path, text.replace("pass++ & 1", "pass++ & 0")) > 0
