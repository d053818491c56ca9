"""Set-up that a device needs once (csrc/once.h), with host threads and no GPU."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>

#include "once.h"

static bq::OncePerDevice once;

static void pause(int ms) { std::this_thread::sleep_for(std::chrono::milliseconds(ms)); }

int main() {
  // eight first calls at the same time: the set-up takes a while, nobody returns before its end
  std::atomic<int> ready{0}, runs{0}, early{0}, failed{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([&] {
      const int rc = once.run(3, [&] {
        ++runs;
        pause(100);
        ready = 1;
        return 0;
      });
      if (!ready) ++early;
      if (rc) ++failed;
    });
  for (auto& t : threads) t.join();
  std::printf("runs %d early %d failed %d\n", int(runs), int(early), int(failed));

  // another device has a set-up of its own; a failure is returned and tried again
  int tries = 0;
  auto second = [&] { return ++tries < 3 ? -5 : 0; };
  const int a = once.run(4, second), b = once.run(4, second), c = once.run(4, second), d = once.run(4, second);
  std::printf("codes %d %d %d %d tries %d\n", a, b, c, d, tries);

  // a device that is not one: every call
  int calls = 0;
  for (int i = 0; i < 3; ++i) once.run(-1, [&] { return ++calls, 0; });
  std::printf("calls %d\n", calls);
}
"""


def test_every_caller_returns_after_the_set_up(tmp_path):
    cxx = os.environ.get("CXX", "g++")
    if shutil.which(cxx) is None:
        pytest.skip("no host C++ compiler")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", os.path.join(ROOT, "block_quant_gb300", "csrc"), str(src),
                    "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout.split("\n")
    assert out[:3] == ["runs 1 early 0 failed 0", "codes -5 -5 0 0 tries 3", "calls 3"]


def test_attributes_are_set_through_it():
    """No kernel attribute is set under a flag that other threads can see before it holds."""
    csrc = os.path.join(ROOT, "block_quant_gb300", "csrc")
    for name in sorted(os.listdir(csrc)):
        text = open(os.path.join(csrc, name)).read()
        if "cudaFuncSetAttribute(" in text:
            assert "OncePerDevice" in text, name
            assert "once_per_device" not in text, name
