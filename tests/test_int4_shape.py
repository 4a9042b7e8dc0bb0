"""The launch shape of the attention over packed rows, on the host alone: the header is
compiled with a fake of the residency query."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "mla_int4_shape.h"
using namespace dsa;
static int fails = 0;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); ++fails; } } while (0)
static bool is(Int4Shape s, int splits, int clusters) { return s.splits == splits && s.clusters == clusters; }

int main() {
  // a query that fails is asked again, one that answers is not (0 is an answer)
  OnceAsked kept;
  int asked = 0;
  CHECK(kept.get([&] { ++asked; return -1; }) == -1);
  CHECK(kept.get([&] { ++asked; return -1; }) == -1);
  CHECK(kept.get([&] { ++asked; return 74; }) == 74);
  CHECK(kept.get([&] { ++asked; return -1; }) == 74);
  CHECK(asked == 3);
  OnceAsked none;
  CHECK(none.get([&] { return 0; }) == 0 && none.get([&] { return 9; }) == 0);

  const auto b200 = [](int s) { return s == 4 ? 18 : s == 2 ? 37 : 74; };
  CHECK(is(int4_shape(1, 2048, 64, 148, b200), 4, 1));
  CHECK(is(int4_shape(18, 2048, 64, 148, b200), 4, 18));
  CHECK(is(int4_shape(19, 2048, 64, 148, b200), 2, 19));
  CHECK(is(int4_shape(37, 2048, 64, 148, b200), 2, 37));
  CHECK(is(int4_shape(38, 2048, 64, 148, b200), 1, 38));
  CHECK(is(int4_shape(2048, 2048, 64, 148, b200), 1, 74));
  CHECK(is(int4_shape(1, 128, 64, 148, b200), 2, 1));
  CHECK(is(int4_shape(1, 64, 64, 148, b200), 1, 1));

  // not known: no splits, but a wave of pairs over the device
  const auto fail = [](int) { return -1; };
  CHECK(is(int4_shape(1, 2048, 64, 148, fail), 1, 1));
  CHECK(is(int4_shape(2048, 2048, 64, 148, fail), 1, 74));
  const auto only_pairs = [](int s) { return s == 1 ? 60 : -1; };
  CHECK(is(int4_shape(2048, 2048, 64, 148, only_pairs), 1, 60));
  const auto zero = [](int) { return 0; };
  CHECK(is(int4_shape(5, 2048, 64, 1, zero), 1, 1));
  return fails != 0;
}
"""


def test_shape_and_failed_queries(tmp_path):
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "long_context_sparse_04_b200", "csrc"), str(src),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout

