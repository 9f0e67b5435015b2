"""The schedule rules of fastar_branch_attention, evaluated on the host: the
same functions that the kernels call, compiled into a small program."""
import os
import subprocess

import pytest

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include "branch.cuh"
using namespace fastar;
int main() {
  char what[32];
  while (scanf("%31s", what) == 1) {
    if (!strcmp(what, "key_units")) {
      int keys, TN;
      if (scanf("%d %d", &keys, &TN) != 2) return 1;
      printf("%d\n", key_units(keys, TN));
    } else {
      return 1;
    }
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    from merged_attention_autoregressive_gb300 import build
    d = tmp_path_factory.mktemp("schedule")
    src, exe = str(d / "rules.cu"), str(d / "rules")
    with open(src, "w") as f:
        f.write(PROGRAM)
    flags = [f for f in build.NVFLAGS if f not in ("-O3", "-lineinfo")]
    r = subprocess.run([build._nvcc(), *build.ARCH, *flags, src, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(*lines):
        text = "\n".join(" ".join(str(x) for x in line) for line in lines)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, env=dict(os.environ))
        assert r.returncode == 0, r.stderr
        return [[int(x) for x in line.split()] for line in r.stdout.splitlines()]

    return run


def test_units_of_any_number_of_keys(ask):
    cases = [(n, TN) for TN in (64, 128) for n in (0, 1, 63, 64, 65, 127, 128, 129, 10 ** 6, 2 ** 31 - 129,
                                                  2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 64, 2 ** 31 - 1)]
    got = ask(*[("key_units", n, TN) for n, TN in cases])
    assert [g[0] for g in got] == [-(-n // TN) for n, TN in cases]
