"""The hand-over of row blocks among a persistent CTA's roles (csrc/handover.h), compiled for the
host and run with a thread per role: with no wait giving up every block is taken once, in the same
order by all; when a wait gives up, at any point and in any role, every role still leaves its loop
and the members of the barrier group leave it in the same pass."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fwd_bwd_double_gb300", "csrc")

DRIVER = r"""
#include <atomic>
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <random>
#include <thread>
#include <vector>
#include "handover.h"
using namespace std::chrono_literals;

constexpr int kGroup = 8, kRoles = kGroup + 2;  // the barrier group, one that asks, one that only takes
std::atomic<int> aborted{0}, stuck{0};

struct Phases {  // completes a phase with every `count` arrivals
  std::mutex m;
  int count, pending, phase = 0;
  explicit Phases(int c) : count(c), pending(c) {}
  void arrive() {
    std::lock_guard<std::mutex> l(m);
    if (--pending == 0) pending = count, ++phase;
  }
  bool done(int parity) {
    std::lock_guard<std::mutex> l(m);
    return (phase & 1) != parity;
  }
};
bool bounded(Phases& b, int parity) {  // false once any wait has given up
  for (;;) {
    if (b.done(parity)) return true;
    if (aborted) return false;
    std::this_thread::yield();
  }
}

struct Vote {  // a barrier of the group with a vote; a member that waits for 20 s is stuck
  std::mutex m;
  std::condition_variable cv;
  int here = 0, round = 0;
  bool every = true, result = true;
  bool operator()(bool x) {
    std::unique_lock<std::mutex> l(m);
    every = every && x;
    if (++here == kGroup) {
      result = every, every = true, here = 0, ++round;
      cv.notify_all();
      return result;
    }
    const int r = round;
    if (!cv.wait_for(l, 20s, [&] { return round != r || stuck; })) stuck = 1, cv.notify_all();
    return round != r ? result : false;
  }
};

struct Cta {
  Phases known{1}, free_{kRoles};
  std::atomic<int> answer{-2}, left;
  std::vector<std::thread> answers;
  explicit Cta(int blocks) : left(blocks) {}
};
struct Role {
  Cta& c;
  std::mt19937& rng;
  void pause() const { if (rng() % 4 == 0) std::this_thread::sleep_for(std::chrono::microseconds(rng() % 60)); }
  bool wait_free(int n) const { return bounded(c.free_, n & 1); }
  bool wait_known(int n) const { pause(); return bounded(c.known, n & 1); }
  void request() const {
    const int us = rng() % 80;
    c.answers.emplace_back([this_c = &c, us] {
      std::this_thread::sleep_for(std::chrono::microseconds(us));
      const int k = this_c->left.fetch_sub(1);
      this_c->answer = k > 0 ? k : -1;
      this_c->known.arrive();
    });
  }
  int answer() const { pause(); return c.answer; }
  void taken() const { c.free_.arrive(); }
};

// One CTA over `blocks` further blocks; role `who` gives up in block `when` (-1: none does).
int trial(unsigned seed, int blocks, int who, int when) {
  aborted = stuck = 0;
  Cta cta(blocks);
  Vote vote;
  std::vector<int> took[kRoles];
  std::vector<std::thread> roles;
  for (int r = 0; r < kRoles; ++r)
    roles.emplace_back([&, r] {
      std::mt19937 rng(seed * 64 + r);
      Role me{cta, rng};
      for (int x = 0, n = 0; x >= 0 && !stuck; ++n) {
        took[r].push_back(x);
        if (r == who && n == when) aborted = 1;
        me.pause();  // the block's work
        if (r == kGroup && !fbd::handover::ask(me, n)) break;
        x = fbd::handover::take(me, n);
        if (r < kGroup) x = fbd::handover::agree(x, [&](bool some) { return vote(some); });
      }
    });
  for (auto& t : roles) t.join();
  for (auto& t : cta.answers) t.join();
  if (stuck) return std::printf("seed %u: a member of the group waits for one that has left\n", seed), 1;
  for (int r = 1; r < kGroup; ++r)
    if (took[r] != took[0]) return std::printf("seed %u: member %d took other blocks\n", seed, r), 1;
  if (when < 0)
    for (int r = 0; r < kRoles; ++r)
      if (took[r] != took[0] || static_cast<int>(took[r].size()) != blocks + 1)
        return std::printf("seed %u: role %d took %zu blocks\n", seed, r, took[r].size()), 1;
  return 0;
}

int main(int argc, char** argv) {
  const int trials = std::atoi(argv[1]);
  for (int t = 0; t < trials; ++t) {
    std::mt19937 rng(t);
    const int blocks = rng() % 6, who = rng() % kRoles;
    if (trial(t, blocks, who, t % 4 == 0 ? -1 : static_cast<int>(rng() % (blocks + 1)))) return 1;
  }
  return 0;
}
"""


RING = r"""
#include <cstdio>
#include "handover.h"

int main() {
  for (int stages = 1; stages <= 4; ++stages)
    for (int fills = 0; fills <= 20; ++fills) {
      int begun[4] = {0, 0, 0, 0};  // fills of each stage: the last one is phase begun - 1
      for (int t = 0; t < fills; ++t) ++begun[t % stages];
      for (int s = 0; s < stages; ++s) {
        if ((begun[s] > 0) != (s < fills)) return std::printf("stage %d of %d after %d fills\n", s, stages, fills), 1;
        if (begun[s] > 0 && fbd::handover::last_phase(fills, stages, s) != ((begun[s] - 1) & 1))
          return std::printf("phase of stage %d of %d after %d fills\n", s, stages, fills), 1;
      }
    }
  return 0;
}
"""


def run_on_host(tmp_path, source, *args):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "handover.cpp", tmp_path / "handover"
    src.write_text(source)
    subprocess.run([cxx, "-O2", "-std=c++17", "-pthread", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe), *args], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout


def test_every_role_leaves(tmp_path):
    run_on_host(tmp_path, DRIVER, "400")


def test_phases_a_cta_that_gave_up_waits_for(tmp_path):
    run_on_host(tmp_path, RING)
