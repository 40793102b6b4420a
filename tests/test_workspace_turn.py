"""The turns of calls that share a workspace: calls on one workspace wait for each other, calls on
others do not wait, whatever the first one waits for."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <future>
#include <thread>
#include <vector>
#include "workspace_turn.h"
using muon::WorkspaceTurn;
using namespace std::chrono_literals;

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  char a, b;
  {
    // a call whose launch blocks: another one on its workspace waits, others go on
    std::promise<void> let_go;
    std::promise<void> holds;
    auto first = std::async(std::launch::async, [&] {
      WorkspaceTurn turn(&a);
      holds.set_value();
      let_go.get_future().wait();
    });
    holds.get_future().wait();
    std::atomic<bool> done{false};
    auto same = std::async(std::launch::async, [&] { WorkspaceTurn turn(&a); done = true; });
    auto other = std::async(std::launch::async, [&] { WorkspaceTurn turn(&b); });
    auto none = std::async(std::launch::async, [&] { WorkspaceTurn turn(nullptr); });
    const bool went_on = other.wait_for(20s) == std::future_status::ready &&
                         none.wait_for(20s) == std::future_status::ready;
    const bool waited = same.wait_for(100ms) == std::future_status::timeout && !done;
    let_go.set_value();
    const bool then = same.wait_for(20s) == std::future_status::ready && done;
    first.wait();
    CHECK(went_on);
    CHECK(waited);
    CHECK(then);
  }
  // many threads on a few workspaces: never two in one
  constexpr int kSpaces = 3;
  char spaces[kSpaces];
  int inside[kSpaces] = {}, count[kSpaces] = {};
  std::atomic<int> bad{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 9; ++t)
    threads.emplace_back([&, t] {
      for (int i = 0; i < 3000; ++i) {
        const int s = (t + i * (t % 2)) % kSpaces;
        WorkspaceTurn turn(&spaces[s]);
        bad += inside[s]++ != 0;
        ++count[s];
        if (i % 100 == 0) std::this_thread::yield();
        --inside[s];
      }
    });
  for (auto& t : threads) t.join();
  CHECK(bad == 0);
  CHECK(count[0] + count[1] + count[2] == 27000);
  return 0;
}
"""


def test_turns(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "turns.cpp", tmp_path / "turns"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I",
                    os.path.join(ROOT, "newton_schulz_step_gb300", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout
