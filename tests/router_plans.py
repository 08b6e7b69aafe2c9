"""Which kernel variants of the router's backward pass a list of cases reaches,
by the library's own rules (csrc/route_plan.h, compiled here as host code)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_layer_15_amd", "csrc")

SOURCE = r"""
#include <cstdio>
#include "route_plan.h"
using namespace moe;
// reads "T d E bf16 mask dw dx" lines, prints the launches' variants, ';' between them
int main() {
  long long T;
  int d, E, bf16, mask, dw, dx;
  while (std::scanf("%lld %d %d %d %d %d %d", &T, &d, &E, &bf16, &mask, &dw, &dx) == 7) {
    const char* act = bf16 ? "bf16" : "f32";
    const char* m = mask ? "masked" : "whole";
    const RowGeom g = gate_geom(T, E);
    const DwPlan p = dw_plan(T, d, E, bf16);
    const int Ep = padded_experts(E);
    std::printf("gate %s %d %d %d", act, g.V, g.L, g.C);
    if (dw && dx && products_in_one_launch(T, d, E, bf16)) {
      std::printf(";products %s %d %s", act, Ep, m);
    } else {
      if (dw) std::printf(";dw %s %dx%d %s", act, p.bc, p.be, m);
      if (dx) std::printf(";dx %s %d %s", act, Ep, !bf16 && Ep > 256 ? "any" : few_tokens(T, d) ? "few" : "many");
    }
    if (dw) {
      if (dw_tokens_per_split(T, p.splits) > kSegment) std::printf(";dw segments %s", m);
      std::printf(";dw %s %s", act, p.splits > 1 ? "parts" : "whole");
    }
    std::printf("\n");
  }
}
"""


def variants(cases, where):
    """For each case (T, d, E, k, act, mask or None, outputs) the set of variants; ``where``: a scratch folder."""
    src, exe = os.path.join(str(where), "plan.cpp"), os.path.join(str(where), "plan")
    if not os.path.exists(exe):
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", src, "-o", exe], check=True)
    lines = "".join(f"{T} {d} {E} {int(act == 'bf16')} {int(mask is not None)} {int('dw_router' in want)} "
                    f"{int('dx' in want)}\n" for T, d, E, _, act, mask, want in cases)
    out = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout
    return [set(row.split(";")) for row in out.splitlines()]


ALL = ("dlogits", "dx", "dw_router", "dbias")
DW = ("dlogits", "dw_router", "dbias")
DX = ("dlogits", "dx")


def _cases():
    """(tokens, hidden, experts, slots, act, mask, outputs): odd token counts, so that the last stage and the last part
    of every kernel end inside a tile; 640, 2176 and 4224 columns end inside a group of 256 or 512."""
    r = []
    masks = (None, "random")
    # few tokens: both products in one launch, and dx alone
    for E in (20, 50, 99, 100, 150, 250, 300, 380, 440, 500):
        r += [(133 + E, 384, E, 3, "bf16", m, ALL) for m in masks]
        r += [(77, 640, E, 3, "bf16", "random", DX), (77, 640, E + 1, 3, "f32", None, DX)]
    r += [(77, 640, 384, 3, "f32", "random", DX)]
    for E in (28, 60, 99, 150, 200, 251):
        r += [(97 + E, 384, E, 3, "f32", m, ALL) for m in masks]
    # many tokens, every width of a row of dL: dx in wide workgroups, dW_r in 128-column tiles
    for E in (30, 33, 128, 150, 256, 300, 384, 448, 511):
        r += [(4101, 640, E, 3, act, m, ALL) for act in ("bf16", "f32") for m in masks]
    # dW_r alone, whole or in parts; in 256-column tiles
    r += [(40, 128, E, 2, act, m, DW) for E in (16, 50, 131) for act in ("bf16", "f32") for m in masks]
    for T, d, E in ((16385, 4224, 20), (16385, 4224, 60), (4099, 4224, 129), (8201, 2176, 500)):
        r += [(T, d, E, 2, "bf16", m, DW) for m in masks]
    r += [(300, 7168, 4, 2, "bf16", "random", ALL), (1, 16384, 257, 2, "bf16", None, ALL)]
    # a part of more tokens than the mask bits that LDS holds at a time
    r += [(1100001, 128, 8, 2, act, m, DW) for act in ("bf16", "f32") for m in masks]
    # the gradient's rows on few lanes: many tokens
    for i, (T, E) in enumerate(((131077, 4), (65541, 8), (32771, 16), (32773, 28), (32775, 64), (16387, 128),
                                (8209, 256), (4103, 500), (32777, 3), (8211, 13), (8213, 29), (8215, 50), (8217, 99),
                                (8219, 150), (4105, 511))):
        r += [(T, 128, E, min(E, 3), "bf16", masks[i % 2], ALL), (T, 128, E, min(E, 3), "f32", masks[1 - i % 2], ALL)]
    return r


CASES = _cases()
