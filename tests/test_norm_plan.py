"""How the norm's ring kernels share an SM out (csrc/ring.h), on the CPU: what is planned to run at once fits."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "device_triggered_transfers_gb300", "csrc")
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "ring.h"
int main(int, char** a) {
    auto n = [&](int i) { return (uint32_t)std::strtoul(a[i], nullptr, 10); };
    const uint32_t threads[3] = {n(6), n(7), n(8)};
    for (uint32_t cols = 1; cols <= 26000; ++cols) {
        if (n(1) && cols % 8) continue;
        const auto g = dtt::ring::plan(cols, n(1), (uint64_t)cols * n(2) + n(3), n(4), n(5), threads, n(9), n(10));
        if (g.ctas) std::printf("%u %u %u %u %u %u\n", cols, g.nch, g.threads, g.ctas, g.stages, g.smem);
    }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run([shutil.which("g++") or "c++", "-O1", "-std=c++17", "-I", CSRC, str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)
    return str(d / "plan")


FWD, BWD = 640, 2432                         # shared memory of the kernels beside their stages
# aligned, bytes a column, bytes besides, the kernel's own, columns of one chunk a thread, threads of an SM, least CTAs, most stages
PLANS = [(1, 4, 0, FWD, 1024, 1536, 1024, 512, 2, 2), (1, 4, 0, FWD, 1024, 1536, 1024, 512, 2, 8), (1, 2, 0, FWD, 1024, 1536, 1024, 512, 2, 8),
         (1, 8, 0, FWD, 1024, 1536, 1024, 512, 2, 8), (0, 4, 60, FWD, 2048, 1024, 1024, 512, 2, 2), (0, 8, 60, FWD, 2048, 1024, 1024, 512, 2, 8),
         (1, 4, 0, BWD, 2048, 1024, 512, 256, 1, 8), (1, 6, 0, BWD, 2048, 1024, 512, 256, 1, 8), (1, 8, 0, BWD, 2048, 1024, 512, 256, 1, 8),
         (1, 12, 0, BWD, 2048, 1024, 512, 256, 1, 8), (0, 6, 90, BWD, 2048, 1024, 512, 256, 1, 8), (0, 12, 90, BWD, 2048, 1024, 512, 256, 1, 8)]


@pytest.mark.parametrize("args", PLANS)
def test_the_planned_ctas_fit_an_sm(program, args):
    out = subprocess.run([program, *map(str, args)], check=True, stdout=subprocess.PIPE, text=True).stdout
    plans = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert plans and plans[0][0] > 256
    for cols, nch, threads, ctas, stages, smem in plans:
        assert threads % 32 == 0 and 64 <= threads <= 512 and threads * 8 * nch >= cols
        assert 2 <= stages <= args[9] or (ctas < 4 and stages <= 8)
        assert smem == stages * (cols * args[1] + args[2]) <= 200 * 1024
        # 228 KiB of an SM, 1 KiB of it reserved for each CTA
        assert ctas * (smem + args[3] + 1024) <= 228 * 1024, (cols, ctas, stages)
