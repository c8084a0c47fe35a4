"""Which form the 8-bit layers' tests reach, asked of the library's own choice on the
host with g++ (moe_expert_8bit_plan.h, moe_expert_tile_choice.h): streamed experts of
each kind, small tiles, large tiles, and large tiles with the light remainders in a
launch of their own, taken or declined."""

import os
import subprocess

import pytest

from test_experts_8bit_forms_gpu import FORMS
from test_experts_8bit_gpu import SHAPES, TAIL
from test_experts_8bit_sums_gpu import STREAMED

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256

DRIVER = r"""
#include <cstdio>
#include "moe_expert_8bit_plan.h"
using namespace moe;
// lines of: max_rows experts n k gated count...  ->  the forms the experts' rows take
int main() {
    long long rows, e, n, k, gated;
    while (std::scanf("%lld %lld %lld %lld %lld", &rows, &e, &n, &k, &gated) == 5) {
        const Stream8Plan s = plan_stream8(rows, e, gated ? 2 * n : n, k, 256);
        const TileChoice t = choose_tiles8(rows, e, n, k, gated != 0, s.groups > 0, 256);
        const long long cols = (n + (gated ? 127 : 255)) / (gated ? 128 : 256);
        long long heavy = 0, light = 0, tiled = 0, streamed = 0;
        for (long long i = 0; i < e; ++i) {
            long long c;
            if (std::scanf("%lld", &c) != 1) return 1;
            if (c == 0) continue;
            (s.groups > 0 && c <= s.most_rows ? streamed : tiled) += c;
            const bool l = light_remainder(c);
            light += l ? cols : 0;
            heavy += ((c + kLargeTile - 1) / kLargeTile - l) * cols;
        }
        if (streamed) std::printf("stream%d ", s.groups);
        if (tiled && t.small) std::printf("small ");
        if (tiled && !t.small && !t.apart) std::printf("large ");
        if (tiled && t.apart) std::printf(remainders_apart(heavy, light, k / 2, 256) ? "apart " : light ? "room " : "none ");
        if (tiled && !t.small && (k / 2 + kStepT - 1) / kStepT >= 16) std::printf("long ");
        std::printf("\n");
    }
}
"""


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.cpp").write_text(DRIVER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "mixture_experts_token_amd", "csrc"),
                    str(d / "choice.cpp"), "-o", str(d / "choice")], check=True)

    def forms(shapes, gated):
        """shapes: (counts, max_rows, n, k)"""
        text = "".join("%d %d %d %d %d %s\n" % (rows, len(c), n, k, gated, " ".join(map(str, c)))
                       for c, rows, n, k in shapes)
        out = subprocess.run([str(d / "choice")], input=text, capture_output=True, text=True, check=True).stdout
        return [set(line.split()) for line in out.splitlines()]

    return forms


@pytest.mark.parametrize("gated", [0, 1])
def test_every_form_is_reached(choice, gated):
    shapes = [(c, sum(c) + TAIL, n, k) for c, n, k in SHAPES]
    found = choice(shapes, gated) + choice([(c, r, n, k) for c, r, n, k in FORMS], gated)
    assert len(found) == len(shapes) + len(FORMS)
    for form in ("stream1", "stream2", "stream4", "small", "large", "apart", "room", "none", "long"):
        assert any(form in f for f in found), form


@pytest.mark.parametrize("gated", [0, 1])
def test_the_named_forms(choice, gated):
    found = choice(FORMS, gated)
    assert [f & {"apart", "none", "large"} for f in found[:2]] == [{"apart"}, {"none"}]
    assert "room" in found[2]
    assert found[3] == {"large", "long"} and all("long" in f for f in found[:5])
    assert all("stream1" in f for f in found[5:]) and found[9] == {"stream1", "small"}


@pytest.mark.parametrize("gated", [0, 1])
def test_streamed_shapes_are_streamed(choice, gated):
    found = choice([(c, sum(c), n, k) for c, n, k in STREAMED], gated)
    assert all(len(f) == 1 for f in found)
    assert set.union(*found) == {"stream1", "stream2", "stream4"}
