"""The schedule rules of fastar_branch_attention, evaluated on the host: the
same functions that the kernels call, compiled into a small program."""
import math
import os
import random
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
    } else if (!strcmp(what, "parts")) {
      long long U;
      int longest, items, G, fp32;
      if (scanf("%lld %d %d %d %d", &U, &longest, &items, &G, &fp32) != 5) return 1;
      printf("%d\n", branch_parts(U, longest, items, G, fp32 != 0));
    } else if (!strcmp(what, "whole")) {
      long long items, rows, own;
      int G, TM, TN, B, C;
      if (scanf("%lld %d %d %d %lld %d %d %lld", &items, &G, &TM, &TN, &rows, &B, &C, &own) != 8) return 1;
      printf("%d\n", branch_whole(items, G, TM, TN, rows, B, C, own) ? 1 : 0);
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


UNEVEN = [
    [257] + [10] * 39,               # one head full, the others near empty
    [257] + [20] * 11,
    [1000, 1],
    [28] * 12,
    [301] * 40,
    [22, 22],
    [1] * 152,
    [2 ** 22, 2 ** 21],
    [0 + 1, 2 ** 22],
]


def test_equal_parts_are_bounded_by_the_longest_item(ask):
    """In parts, the longest run is at most 4 units longer than the even cut's,
    or the parts are as few as the join's cost asks for."""
    rng = random.Random(3)
    cases = [(units, fp32) for units in UNEVEN for fp32 in (0, 1)]
    for _ in range(500):
        items = rng.choice((1, 2, 3, 5, 8, 12, 24, 40, 76, 100, 152))
        top = 2 ** rng.randint(0, 12)
        cases.append(([1 + (rng.randrange(top) if rng.random() < 0.5 else top // 7) for _ in range(items)], rng.randint(0, 1)))
    got = ask(*[("parts", sum(u), max(u), len(u), 304 if fp32 else 152, fp32) for u, fp32 in cases])
    cut = 0
    for (units, fp32), (parts,) in zip(cases, got):
        G = 304 if fp32 else 152
        n, even = G // len(units), -(-sum(units) // G)
        assert 0 <= parts <= n
        if parts == 0:
            cut += 1
            continue
        wanted = math.ceil(math.sqrt((48 if fp32 else 8) * max(units)))
        assert parts == min(n, wanted) or abs(parts - wanted) <= 1
        assert -(-max(units) // n) <= even + 4
        if parts == n:
            assert -(-max(units) // parts) <= even + 4
    assert 0 < cut < len(cases)


def test_parts_of_the_measured_calls(ask):
    # 12 heads of 28 units; 2 heads of 22; one head full beside near empty ones; 40 heads of 301
    assert ask(("parts", 336, 28, 12, 152, 0), ("parts", 44, 22, 2, 152, 0), ("parts", 647, 257, 40, 152, 0),
               ("parts", 477, 257, 12, 152, 0), ("parts", 12040, 301, 40, 152, 0)) == [[12], [14], [0], [0], [0]]


def _whole(H, g, new, own, C=0, fp32=False):
    """The rule's arguments for branches of `new` tokens with room for `own`."""
    TM, TN, G = (64, 64, 304) if fp32 else (128, 128, 152)
    rows = sum(new) * g
    return ("whole", H * -(-rows // TM), G, TM, TN, rows, len(new), C, own)


def test_items_are_left_whole_where_they_are_short(ask):
    ragged = [int(601 * ((b * 7919 + 104729) % 9973) / 9973) for b in range(9)]
    cases = [
        (_whole(4, 3, ragged, 864), 1),                              # as measured beside the rule
        (_whole(12, 1, [200] * 40, 512), 1),
        (_whole(12, 1, [20] * 300, 320), 1),
        (_whole(8, 1, [1] * 2560, 1024), 0),                         # 128 branches to a tile
        (_whole(40, 1, [1] * 640, 512), 0),
        (_whole(40, 1, [1] * 7 + [1024], 1024), 0),                  # long beside short
        (_whole(40, 1, [1] * 8 + [1000], 1024), 0),
        (_whole(8, 1, [250] * 16, 400, fp32=True), 0),
        (_whole(8, 1, [1] * 2560, 500, fp32=True), 0),
        (_whole(4, 3, ragged, 2048), 0),                             # long keys
        (_whole(4, 3, ragged, 200, C=900), 0),
        (_whole(1, 1, ragged, 864), 0),                              # few items
        (("whole", 2 ** 44, 152, 128, 128, 2 ** 31 - 300, 2 ** 31 - 300, 2 ** 31 - 1, 2 ** 31 - 256), 0),  # no overflow
    ]
    got = ask(*[c for c, _ in cases])
    assert [g[0] for g in got] == [want for _, want in cases]
