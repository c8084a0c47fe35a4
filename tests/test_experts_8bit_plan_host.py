"""The 8-bit layers' streaming plan (moe_expert_8bit_plan.h) on the host: its
kernels' assumptions hold for any sizes, and the passes over an expert's weights
are bounded for any routing.
"""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "moe_expert_8bit_plan.h"
using namespace moe;
static void require(bool ok, const char* what, long long a, long long b, long long c, long long d) {
    if (!ok) { std::printf("%s: rows %lld experts %lld cols %lld k %lld\n", what, a, b, c, d); std::exit(1); }
}
int main() {
    const long long sizes[] = {1, 2, 3, 5, 8, 13, 64, 100, 256, 1000, 1024};
    const long long ks[] = {16, 32, 240, 256, 272, 512, 528, 768, 2048, 4096, 7168, 14336, 16400, 131056, 1 << 20};
    const long long cols[] = {8, 16, 200, 1536, 4096, 28672, 1 << 21};
    long long plans = 0;
    for (long long e : sizes)
    for (long long k : ks)
    for (long long c : cols)
        for (long long rows : {1LL, 2LL, e, e + 1, 2 * e, 2 * e + 1, 6 * e, 6 * e + 1, 12 * e, 12 * e + 1, 1LL << 30})
            for (int cus : {1, 8, 256}) {
                const Stream8Plan p = plan_stream8(rows, e, c, k, cus);
                if (p.groups == 0) { require(rows > 12 * e, "not streamed", rows, e, c, k); continue; }
                ++plans;
                require(rows <= 12 * e, "streamed", rows, e, c, k);
                require(p.groups == 1 || p.groups == 2 || p.groups == 4, "groups", rows, e, c, k);
                require(p.kw >= 1 && p.kw <= kStream8Waves && (p.kw & (p.kw - 1)) == 0, "kw", rows, e, c, k);
                // whole rounds of steps, which cover the row and no more than a round too many
                require(p.steps >= kStream8InFlight && p.steps % kStream8InFlight == 0, "steps", rows, e, c, k);
                const long long covered = (long long)p.steps * p.kw * kStream8Piece;
                require(covered >= k, "row", rows, e, c, k);
                require((long long)(p.steps - kStream8InFlight) * p.kw * kStream8Piece < k, "steps too many", rows, e, c, k);
                // byte positions of a row, past its end included, stay far below 2^31
                require(covered < (1LL << 21) + (1 << 14), "position", rows, e, c, k);
                // passes over an expert's weights
                require((p.most_rows + 4 * p.groups - 1) / (4 * p.groups) <= 4, "passes", rows, e, c, k);
            }
    std::printf("%lld plans\n", plans);
    return plans > 1000 ? 0 : 1;
}
"""


def test_plan(tmp_path):
    src = tmp_path / "plan.cpp"
    src.write_text(DRIVER)
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I",
                    os.path.join(ROOT, "mixture_experts_token_amd", "csrc"), str(src), "-o", exe], check=True)
    res = subprocess.run([exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout
