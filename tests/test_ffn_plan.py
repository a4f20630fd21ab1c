"""How the products of the gated feed-forward block are cut and dealt out to pairs of
CTAs (CPU only): every element of every product is computed exactly once, whatever the
sizes, and the gradient of few tokens gets wide tiles for the weights' gradients, whose
way out of TMEM is what they cost, beside narrow or split ones for dx."""
import random
import subprocess

import pytest

from implicit_gemm_convolution_vae_gb300.build import CSRC

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <set>
#include <tuple>
#include "vae_ffn_plan.h"
using namespace vae::ffn;
// Every tile of the plan once, within its product, and all of them the whole of it.
static int cover(const Group* g, int count, const Deal& d, int pairs) {
    std::set<std::tuple<int, int, int, int>> seen;
    long long area = 0, want = 0;
    int all = 0;
    for (int r = 0; r < d.n; ++r) all += d.pairs[r];
    if (all != pairs || d.n > kRuns) return 1;
    for (int q = 0; q < pairs; ++q) {
        Tile t;
        for (int i = 0; tile_at(g, d, q, i, &t); ++i) {
            const Group& h = g[t.g];
            if (!seen.insert({t.g, t.part, t.m0, t.n0}).second) return 2;
            if (t.m0 < 0 || t.m0 >= h.rows || t.n0 < 0 || t.n0 >= h.cols || t.n < 32 || t.n > kMaxCols || t.n % 32 != 0) return 3;
            if (t.k0 < 0 || t.k1 <= t.k0 || t.k1 > h.nk || t.part >= h.problems * h.splits || t.z != t.g + t.part / h.splits) return 4;
            if (t.subs < 1 || t.subs > h.tall || (h.tall > 1 && h.splits > 1)) return 5;
            area += 1LL * std::min(t.n, h.cols - t.n0) * std::min(256 * t.subs, h.rows - t.m0) * (t.k1 - t.k0);
        }
    }
    for (int k = 0; k < count; ++k) want += 1LL * g[k].rows * g[k].cols * g[k].nk * g[k].problems;
    return area != want ? 6 : 0;
}
int main() {
    int kind, m, c, f;
    while (scanf("%d %d %d %d", &kind, &m, &c, &f) == 4) {
        const Plan p = make_plan(kind, m, c, f);
        const int count = kind == kGrad ? 2 : 1;
        int bad = cover(p.group, count, p.deal, kPairs);
        for (int pairs : {1, 7, 60}) {  // (as on a device with fewer SMs)
            Deal d;
            deal_out(kind, p.group, count, pairs, &d);
            if (bad == 0) bad = cover(p.group, count, d, pairs);
        }
        if (bad == 0 && kind == kGrad) {  // dx alone
            Deal d;
            deal_out(kind, p.group, 1, kPairs, &d);
            bad = cover(p.group, 1, d, kPairs);
        }
        printf("%d %d %d %d %d %d\n", bad, p.group[0].wide, p.group[0].splits, p.group[1].wide, p.group[1].splits, p.group[0].tall);
    }
}
"""
GATE, DOWN, BACK_GATE, GRAD = range(4)


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """(fault, width, splits of the first group, of the second, tall) of many (kind, m, c, f)."""
    tmp = tmp_path_factory.mktemp("plan")
    src, exe = tmp / "plan.cpp", tmp / "plan"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, str(src),
                    "-o", str(exe)], check=True)

    def answers(cases):
        text = "".join("%d %d %d %d\n" % c for c in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return answers


def test_every_tile_once(plans):
    r = random.Random(11)
    sizes = [(1, 8, 8), (1 << 24, 8, 8), (1, 16384, 65536), (300, 64, 128), (4353, 640, 2568), (41001, 72, 136)]
    for _ in range(400):
        c = min(16384, 8 * r.randint(1, 2 ** r.randint(1, 9)))
        sizes.append((r.randint(1, 2 ** r.randint(1, 15)), c, min(65536, 8 * r.randint(1, 2 ** r.randint(1, 10)))))
    cases = [(kind, *s) for s in sizes for kind in range(4)]
    got = plans(cases)
    assert len(got) == len(cases)
    assert not [(c, g) for c, g in zip(cases, got) if g[0] != 0]


def test_weights_gradients_of_few_tokens_get_wide_tiles(plans):
    # tokens, c, f; measured in a graph: 55 us with 128 columns for both groups and 46 with 256 for the weights' gradients
    cases = [(GRAD, m, 1152, 4608) for m in (1, 40, 256, 1024)] + [(GRAD, 256, 2048, 5504), (GRAD, 1024, 512, 2048)]
    for case, g in zip(cases, plans(cases)):
        assert g[0] == 0 and g[3] == 256, (case, g)
    one, forty = plans([(GRAD, 1, 1152, 4608), (GRAD, 40, 1152, 4608)])
    assert one == forty and one[2] > 1  # dx's long sums are split


def test_large_gradients_keep_tiles_of_512_rows(plans):
    cases = [(GRAD, 16384, 1152, 4608), (GRAD, 4100, 576, 2304), (GRAD, 8192, 2048, 5504), (GRAD, 4096, 512, 2048)]
    assert all(g == (0, 256, 1, 256, 1, 2) for g in plans(cases))
