"""The host's memory of launch queries (csrc/launch_cache.h), compiled alone: keys that data
decide, without end, must not stop it from remembering."""
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
