"""The linear attention's tcgen05 kernel when a wait runs out: no warp is left at a barrier.

On the GPU the case cannot be made without a hang where the code is wrong, so the loop of the
warps that turn K into K' (the one group whose warps wait one by one and meet at a barrier without
a time limit) is taken from the kernel's source, compiled for the host with a thread for each warp,
and run with every wait failing in turn."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "ternary_weight_lm_b200", "csrc", "linattn_tc.cu")

HARNESS = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <set>
#include <thread>
#include <vector>

// a barrier of four warps that is open for a bounded time
struct Meeting {
  std::mutex m;
  std::condition_variable cv;
  int here = 0, round = 0;
  bool all = true, result = false, stuck = false;
  bool join(bool ok) {
    std::unique_lock<std::mutex> l(m);
    all = all && ok;
    if (++here == 4) {
      result = all;
      all = true;
      here = 0;
      ++round;
      cv.notify_all();
      return result;
    }
    const int mine = round;
    if (!cv.wait_for(l, std::chrono::seconds(5), [&] { return round != mine || stuck; }) || stuck) {
      stuck = true;
      cv.notify_all();
      return false;
    }
    return result;
  }
};

struct Bars { int full[2], scores[2], v[2], k[2], upd; };
struct Shared { Bars bars; };

template <bool kState>
void group(Meeting& meeting, int warp, int chunks, const std::set<int>& fails) {
  constexpr int lane = 0, kGroup = 128;
  Shared sh;
  int waits = 0;
  auto wait = [&](int&, int) { return fails.count(waits++) == 0; };
  auto arrive = [&](int&) {};
  auto clean_v = [&](int, int) {};
  auto find_exp = [&](int, int, int, int, bool ok, float* f) { *f = 1.0f; return meeting.join(ok); };
  auto named_bar_and = [&](int, int, bool ok) { return meeting.join(ok); };
  auto decay_k = [&](int, int, int, float) {};
  BODY
}

template <bool kState>
int run(const std::vector<std::set<int>>& fails) {
  Meeting meeting;
  std::vector<std::thread> t;
  for (int w = 0; w < 4; ++w) t.emplace_back([&, w] { group<kState>(meeting, 8 + w, 4, fails[w]); });
  for (auto& x : t) x.join();
  return meeting.stuck;
}

int main() {
  for (int n = 0; n < 11; ++n)            // waits of four chunks
    for (int who = 1; who < 16; ++who) {  // the warps that give up there
      std::vector<std::set<int>> fails(4);
      for (int w = 0; w < 4; ++w)
        if (who >> w & 1) fails[w].insert(n);
      if (run<false>(fails) || run<true>(fails)) {
        std::printf("wait %d, warps %x: a warp is left at the barrier\n", n, who);
        return 1;
      }
    }
  return 0;
}
"""


def test_a_wait_that_runs_out_leaves_no_warp_at_a_barrier(tmp_path):
    text = open(SOURCE).read()
    body = re.search(r"\} else if \(warp < 12\) \{\n(.*?)\n  \} else \{\n", text, re.S).group(1)
    assert "find_exp" in body and "wait(sh.bars.scores" in body
    body = "\n".join(x for x in body.splitlines() if "asm volatile" not in x)
    src, exe = tmp_path / "group.cpp", tmp_path / "group"
    src.write_text(HARNESS.replace("BODY", body))
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-w", "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout
