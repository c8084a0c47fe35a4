"""The choice between streaming and tiles (moe_expert_plan.h) checked on the host with g++.

How rows fall on the experts is only known on the device.  Whatever the
routing, what is streamed must stay within bounds that the plan is made for:
  * the x rows of a pass fit the kernel's LDS, and are a number it is built for;
  * an expert's weights are streamed at most kStreamPasses times, or else the
    passes past each expert's first are at most a quarter of the experts;
  * a plan that streams nothing says so.

The library holds the variants that calls reach and no others.
"""

import os
import re
import subprocess

from mixture_experts_token_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_token_amd", "csrc")

DRIVER = r'''
#include <cstdio>
#include <initializer_list>
#include "moe_expert_plan.h"
using namespace moe;
int main() {
  int fails = 0;
  long long streamed = 0;
  for (long long k : {8LL, 64LL, 768LL, 1024LL, 1096LL, 2048LL, 4096LL, 4104LL, 7168LL, 8192LL, 8200LL, 14336LL, 16384LL,
                      16392LL, 24576LL, 32768LL, 32776LL, 1LL << 20})
    for (long long e : {1LL, 2LL, 7LL, 8LL, 64LL, 128LL, 256LL, 1024LL})
      for (long long rows : {1LL, 2LL, 3LL, 8LL, 16LL, 33LL, 64LL, 128LL, 256LL, 511LL, 512LL, 2000LL, 2048LL, 6144LL, 6145LL, 1000000LL}) {
        const StreamPlan p = plan_stream(rows, e, k);
        const long long row = (k / 8 + kStreamBatchVecs - 1) / kStreamBatchVecs * kStreamBatchVecs * 16;
        if (p.x_rows == 0) {
          if (p.most_rows != 0) { ++fails; std::printf("FAIL nothing streamed, most_rows %lld\n", (long long)p.most_rows); }
          continue;
        }
        ++streamed;
        const bool built = p.x_rows == 1 || p.x_rows == 2 || p.x_rows == 4 || p.x_rows == 8;
        if (!built || p.x_rows * row > kStreamXLds || p.most_rows < 1) {
          ++fails;
          std::printf("FAIL k=%lld x_rows=%d most_rows=%lld\n", k, p.x_rows, (long long)p.most_rows);
        }
        for (long long used = 1; used <= e && used <= rows; ++used) {  // rows / used rows on each of `used` experts
          const long long c = rows / used;
          if (c > p.most_rows) continue;  // taken by the tiles
          const long long passes = (c + p.x_rows - 1) / p.x_rows;
          if (passes > kStreamPasses && used * (passes - 1) * 4 > e) {
            ++fails;
            std::printf("FAIL k=%lld experts=%lld: %lld rows on each of %lld experts, weights streamed %lld times\n", k, e, c, used, passes);
            break;
          }
        }
      }
  if (streamed == 0) ++fails;
  std::printf("%s (%d failures, %lld plans that stream)\n", fails ? "FAILED" : "ok", fails, streamed);
  return fails ? 1 : 0;
}
'''


def test_streamed_passes_are_bounded_for_any_routing(tmp_path):
    src = tmp_path / "stream_plan.cpp"
    src.write_text(DRIVER)
    exe = tmp_path / "stream_plan"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout[-3000:]


def test_every_variant_is_reached():
    """Activations 0 .. 3 of the gated layer's slopes, 1 .. 3 of the linear layer's (without one there is no pass)."""
    out = subprocess.run(["nm", "-C", binding.LIB_PATH], capture_output=True, text=True, check=True).stdout
    slopes = set(re.findall(r"__device_stub__expert_act_grad_kernel<(\w+), (\d)>", out))
    assert slopes == {("true", str(a)) for a in range(4)} | {("false", str(a)) for a in range(1, 4)}
    streams = set(re.findall(r"__device_stub__expert_stream_kernel<(\w+), (\d)>", out))
    assert streams == {(g, str(a)) for g in ("true", "false") for a in range(4)}
