"""How the 4-bit calls count groups of rows (csrc/mx_plan.h, compiled here as
host code): segments that do not overlap keep all of their groups, and no
bounds whatever get more than the workspace holds."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_layer_15_amd", "csrc")

GROUPS = r"""
#include <algorithm>
#include <cstdio>
#include <vector>
#include "mx_plan.h"
// reads "S El unit bounds ..." lines; prints the room and the running numbers as the kernels form them
int main() {
  long long S;
  int El, unit;
  while (std::scanf("%lld %d %d", &S, &El, &unit) == 3) {
    std::vector<long long> b(El + 1);
    for (auto& v : b) std::scanf("%lld", &v);
    for (auto& v : b) v = std::max(0LL, std::min(v, S));
    const long long most = moe::mx_max_groups(S, El, unit);
    const int limit = (int)most / unit * unit;
    std::printf("%lld", most);
    int before = 0;
    for (int e = 0; e < El; ++e) {
      std::printf(" %d", before);
      before = moe::mx_add_groups(before, moe::mx_groups((int)std::max(0LL, b[e + 1] - b[e]), unit), limit);
    }
    std::printf(" %d\n", before);
  }
}
"""


def _ask(where, name, source, lines, *flags):
    src, exe = os.path.join(str(where), name + ".cpp"), os.path.join(str(where), name)
    with open(src, "w") as f:
        f.write(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", *flags, f"-I{CSRC}", src, "-o", exe], check=True)
    out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    return [[int(v) for v in row.split()] for row in out.stdout.splitlines()]


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_groups_of_any_bounds_fit_the_workspace(tmp_path):
    r = random.Random(1)
    cases = []
    for unit in (1, 4):
        for S in (1, 31, 32, 33, 127, 128, 129, 4096, 100003, 2 ** 31 - 1):
            for El in (1, 2, 4, 37, 511, 512):
                cuts = [sorted(r.randint(0, S) for _ in range(El - 1)) for _ in range(3)]
                good = [[0] + c + [S] for c in cuts] + [[0] * El + [S], [0] + [S] * El, list(range(El)) + [S]]
                # one row an expert, and segments of one row more than whole groups
                good.append([min(e * (32 * unit + 1), S) for e in range(El + 1)])
                bad = [[(e % 2) * S for e in range(El + 1)], [S - (e % 2) * S for e in range(El + 1)], [S] + [0] * El,
                       [r.randint(-2 ** 31, 2 ** 31 - 1) for _ in range(El + 1)], [r.randint(0, S) for _ in range(El + 1)]]
                cases += [(S, El, unit, b, b == sorted(b) and b[0] >= 0 and b[-1] <= S) for b in good + bad]
    rows = _ask(tmp_path, "groups", GROUPS, [f"{S} {El} {unit} " + " ".join(map(str, b)) for S, El, unit, b, _ in cases],
                "-fsanitize=undefined", "-fno-sanitize-recover=all")
    assert len(rows) == len(cases)
    held = 0
    for (S, El, unit, b, ordered), (most, *groups) in zip(cases, rows):
        want = [0]
        for e in range(El):
            lo, hi = (max(0, min(v, S)) for v in (b[e], b[e + 1]))
            want.append(want[-1] + -(-max(0, hi - lo) // (32 * unit)) * unit)
        assert all(x <= y for x, y in zip(groups, groups[1:]))
        assert groups[-1] <= most and all(v % unit == 0 for v in groups)
        if ordered:
            assert groups == want, (S, El, unit, b)
        else:
            held += want[-1] > most
    assert held > 100     # (bounds that would pass the end of the workspace are among them)
