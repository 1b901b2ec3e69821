"""The host's memory of launch queries and opt-ins (csrc/launch_cache.h), compiled alone: keys that
data decide, without end, must not stop it from remembering, and no thread may lower what
another's launch needs."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <stdio.h>
#include "launch_cache.h"
using namespace moeperm;
static QueryCache<256> cache;
static char kernels[400];
// One launch: 1 where it had to ask.
static int launch(int kernel, size_t smem, int dev = 0) {
  const LaunchKey k{&kernels[kernel], smem, 256, dev};
  const int answer = kernel * 7 + (int)(smem % 1000) + dev;
  int got = -1;
  if (cache.find(k, &got)) {
    if (got != answer) printf("wrong answer\n");
    return 0;
  }
  cache.keep(k, answer);
  cache.keep(k, answer);  // (two threads that asked at once)
  return 1;
}
int main() {
  int asked = 0;
  for (int q = 1; q <= 4096; ++q) asked += launch(0, 8192 + 8 * q);  // every number of groups
  for (int t = 1; t <= 2048; ++t) asked += launch(1, 1280 + 64 * t);  // every decode batch
  if (asked != 4096 + 2048) printf("%d asked of new keys\n", asked);
  // a program's hundred kernels and sizes, again and again, while new sizes keep coming
  for (int k = 2; k < 102; ++k) launch(k, 0);
  asked = 0;
  for (int i = 0; i < 100; ++i) {
    for (int k = 2; k < 102; ++k) asked += launch(k, 0);
    launch(0, 100000 + 8 * i);
  }
  printf("%d\n", asked);
  if (!launch(5, 0, 1) || launch(5, 0, 1) || launch(5, 0, 0)) printf("devices mixed up\n");
}
"""

OPT_INS = r"""
#include <stdio.h>
#include <atomic>
#include <chrono>
#include <thread>
#include "launch_cache.h"
using namespace moeperm;
constexpr int kKernels = 100;
static SmemOptIns<1024> opt_ins;
static std::atomic<size_t> limit[kKernels][4];  // what each "kernel" may take in each context
static std::atomic<int> sets{0}, refused{0}, there{0};
static char kernels[kKernels];
static void launch(int kernel, int ctx, int known, size_t dyn, int us = 0) {
  const int err = opt_ins.raise(&kernels[kernel], known ? ctx : 0, dyn, [&](size_t bytes) {
    ++sets;
    std::this_thread::sleep_for(std::chrono::microseconds(us));
    limit[kernel][ctx] = bytes;
    return 0;
  });
  if (err != 0 || limit[kernel][ctx] < dyn) ++refused;
}
// Two threads launch each kernel for the first time at once, one needing more than the other.
static void first_launches(int id) {
  for (int k = 0; k < kKernels; ++k) {
    ++there;
    while (there < 2 * (k + 1)) std::this_thread::yield();
    launch(k, 1, 1, id ? 200000 : 60000, id == k % 2 ? 50 : 500);
  }
}
int main() {
  std::thread a(first_launches, 0), b(first_launches, 1);
  a.join();
  b.join();
  for (int k = 0; k < kKernels; ++k) launch(k, 1, 1, 200000);
  printf("%d refused, set %s\n", (int)refused, sets <= 2 * kKernels ? "seldom" : "often");
  // the first launch of a context comes before its id is known
  launch(0, 3, 0, 200000);
  launch(0, 3, 1, 60000);
  if (limit[0][3] < 200000) printf("lowered\n");
  const int before = sets;
  launch(0, 3, 1, 190000);
  if (sets != before) printf("set again\n");
  // an error is not taken for an opt-in
  if (opt_ins.raise(&kernels[1], 3, 70000, [](size_t) { return 2; }) != 2) printf("error lost\n");
  launch(1, 3, 1, 70000);
  // a full table: everything is still set
  static SmemOptIns<4> small;
  static char many[9];
  for (int k = 0; k < 9; ++k) {
    size_t got = 0;
    small.raise(&many[k], 1, 50000, [&](size_t b) { got = b; return 0; });
    if (got != 50000) printf("not set\n");
  }
  printf("%d refused\n", (int)refused);
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")

    def compile_and_run(name, text):
        d = tmp_path_factory.mktemp(name)
        src, exe = d / "t.cpp", d / "t"
        src.write_text(text)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I" + os.path.join(ROOT, "combine_fp8_quant_gb300", "csrc"), str(src),
                        "-o", str(exe)], check=True)
        return subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout.split("\n")

    return compile_and_run


def test_new_keys_do_not_exhaust_the_cache(run):
    """10000 launches of keys that were asked for before, 100 new ones between them: displaced keys are asked
    for again, one in a hundred at most."""
    out = run("queries", PROGRAM)
    assert out[1:] == [""] and int(out[0]) <= 100


def test_opt_ins_only_rise(run):
    """Threads whose launches need different amounts of shared memory: no launch finds less than it needs."""
    assert run("opt_ins", OPT_INS) == ["0 refused, set seldom", "0 refused", ""]
