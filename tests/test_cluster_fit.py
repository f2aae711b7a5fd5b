"""The kept answers on how many clusters run at once (csrc/cluster_fit.h, host
code): each GPU's own, and none that was no answer."""
import os
import shutil
import subprocess

import pytest

DRIVER = r"""
#include "cluster_fit.h"
#include <cstdio>
#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
int main() {
  static m2rnn::ClusterFit fit;
  int asked = 0;
  auto answers = [&](int n) { return [&asked, n] { ++asked; return n; }; };
  CHECK(fit.get(0, 2, 152, answers(140)) == 140 && asked == 1);
  CHECK(fit.get(0, 2, 152, answers(7)) == 140 && asked == 1);   // kept
  CHECK(fit.get(1, 2, 152, answers(66)) == 66 && asked == 2);   // another GPU's own
  CHECK(fit.get(0, 2, 152, answers(7)) == 140 && asked == 2);
  CHECK(fit.get(0, 8, 38, answers(0)) == 38 && asked == 3);     // no answer: not kept
  CHECK(fit.get(0, 8, 38, answers(36)) == 36 && asked == 4);
  CHECK(fit.get(0, 8, 38, answers(7)) == 36 && asked == 4);
  CHECK(fit.get(63, 8, 38, answers(31)) == 31 && fit.get(63, 8, 38, answers(7)) == 31 && asked == 5);
  CHECK(fit.get(64, 8, 38, answers(30)) == 30 && fit.get(0, 8, 38, answers(7)) == 36);  // beyond the table: asked anew
  CHECK(fit.get(64, 8, 38, answers(29)) == 29 && fit.get(-1, 8, 38, answers(28)) == 28);
  return 0;
}
"""


def test_answers_are_kept_by_device(tmp_path, root_dir):
    compiler = shutil.which("g++")
    if compiler is None:
        pytest.skip("no C++ compiler")
    source, program = tmp_path / "fit.cpp", tmp_path / "fit"
    source.write_text(DRIVER)
    subprocess.run([compiler, "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(root_dir, "matrix_state_non_gb300", "csrc"),
                    str(source), "-o", str(program)], check=True)
    run = subprocess.run([str(program)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
