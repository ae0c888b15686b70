"""A warp's wait with a limit (csrc/waits.hpp), run by host threads that stand for lanes whose polls and clocks differ:
all lanes take part in the same votes, and leave together with one answer."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "event_tensor_task_b200", "csrc")
SHIM = r"""
#include <chrono>
#include <condition_variable>
#include <mutex>
#include <thread>
#include <vector>
#include "%s/waits.hpp"

// Votes of n lanes: a vote is complete when all lanes have come to the same one.
struct Votes {
  int n, here = 0, kind = -1, and_ = 1, or_ = 0, result = 0;
  long round = 0;
  bool broken = false;
  std::mutex m;
  std::condition_variable cv;
  int vote(int k, int p) {
    std::unique_lock<std::mutex> l(m);
    if (broken) return 0;
    if (here && k != kind) { broken = true; cv.notify_all(); return 0; }  // two lanes at different votes
    kind = k;
    and_ &= p, or_ |= p;
    if (++here == n) {
      result = k ? or_ : and_;
      here = 0, and_ = 1, or_ = 0, ++round;
      cv.notify_all();
      return result;
    }
    const long mine = round;
    if (!cv.wait_for(l, std::chrono::seconds(1), [&] { return broken || round != mine; })) broken = true;
    return broken ? 0 : result;
  }
};
struct Lane {  // sees it at its `sees`-th poll; its clock moves `step` a reading
  Votes& v;
  int sees, step;
  int polls = 0;
  unsigned long long t = 0;
  bool there() { return ++polls >= sees || v.broken; }
  bool all(bool p) { return v.vote(0, p); }
  bool any(bool p) { return v.vote(1, p); }
  unsigned long long now() { return v.broken ? 1000000 : t += step; }
};
bool alone_first(Lane& w, unsigned long long limit) {  // a vote that only lanes that were early reach
  if (w.there()) return true;
  bool lost = false;
  const unsigned long long t0 = w.now();
  while (!w.there()) if (w.now() - t0 > limit) { lost = true; break; }
  return !w.any(lost);
}
// 1 or 0: all lanes' answer; -1: they part, or answer differently
extern "C" int run(int together, int n, const int* sees, const int* step, int limit) {
  Votes v;
  v.n = n;
  std::vector<int> answer(n);
  std::vector<std::thread> lanes;
  for (int i = 0; i < n; ++i)
    lanes.emplace_back([&, i] {
      Lane w{v, sees[i], step[i]};
      answer[i] = together ? mk::wait_together(w, limit) : alone_first(w, limit);
      v.vote(2, 1);  // what the warp does next, together
    });
  for (auto& t : lanes) t.join();
  if (v.broken) return -1;
  for (int a : answer) if (a != answer[0]) return -1;
  return answer[0];
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    d = tmp_path_factory.mktemp("waits")
    (d / "shim.cpp").write_text(SHIM % CSRC)
    subprocess.run(["g++", "-std=c++17", "-pthread", "-shared", "-fPIC", "-o", str(d / "shim.so"), str(d / "shim.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "shim.so"))
    return lambda together, sees, step, limit: lib.run(together, len(sees), (ctypes.c_int * len(sees))(*sees),
                                                       (ctypes.c_int * len(sees))(*step), limit)


@pytest.mark.parametrize("sees,step,limit,answer", [
    ([1, 1, 1, 1], [1] * 4, 100, 1),
    ([1, 2, 1, 1], [1] * 4, 100, 1),            # one lane's first poll comes too soon
    ([1, 1, 7, 3], [1, 2, 1, 1], 100, 1),
    ([999, 999, 999, 999], [1] * 4, 50, 0),
    ([1, 999, 1, 999], [1] * 4, 50, 0),         # some lanes never see it
    ([999, 999, 999, 999], [1, 1, 40, 1], 50, 0),  # one lane's clock runs ahead
])
def test_lanes_stay_together(run, sees, step, limit, answer):
    assert run(1, sees, step, limit) == answer


def test_lanes_that_vote_by_their_own_polls_part(run):
    assert run(0, [1, 1, 1, 1], [1] * 4, 100) == 1
    assert run(0, [1, 2, 1, 1], [1] * 4, 100) == -1
