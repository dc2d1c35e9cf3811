"""How the layer norm's ring kernels share an SM out (csrc/ring.h with csrc/norm.cu's constants), on the CPU: what is planned to run at once
fits, and the kernels' threads hold the row."""
import os
import re
import subprocess

import pytest

from test_norm_plan import CSRC

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "ring.h"
int main(int, char** a) {
    auto n = [&](int i) { return (uint32_t)std::strtoul(a[i], nullptr, 10); };
    const uint32_t threads[3] = {n(6), n(7), n(8)};
    for (uint32_t cols = 1; cols <= 26000; ++cols) {
        if (n(1) && cols % 8) continue;
        const auto g = dtt::ring::plan(cols, n(1), (uint64_t)cols * n(2) + n(3), n(4), n(5), threads, n(9), n(10), n(11));
        if (g.ctas) std::printf("%u %u %u %u %u %u\n", cols, g.nch, g.threads, g.ctas, g.stages, g.smem);
    }
}
"""
FWD, BWD, WIDE, ANY = 896, 4736, 768, 16 * 512           # shared memory beside the stages; threads of a wide row; no limit of two chunks
# aligned, bytes a column, bytes besides, the kernel's own, columns of one chunk a thread, threads of an SM, least CTAs, most stages, columns of two chunks
FORWARD = [(1, 2, 0, FWD, 1024, 1024, 768, 512, 2, 8, 4096), (1, 4, 0, FWD, 1024, 1024, 768, 512, 2, 2, 4096), (1, 4, 0, FWD, 1024, 1024, 768, 512, 2, 8, 4096),
           (1, 8, 0, FWD, 1024, 1024, 768, 512, 2, 8, 4096), (0, 2, 60, FWD, 2048, 1024, 1024, 512, 2, 8, ANY), (0, 8, 60, FWD, 2048, 1024, 1024, 512, 2, 2, ANY)]
BACKWARD = [(v, bytes_, 0 if v else 90, BWD, 2048, 1024, 512, 256, 1, 8, ANY) for v in (1, 0) for bytes_ in (4, 6, 8, 10, 12)]
# a CTA's most threads with one, two and four chunks (or 8 and 16 elements) a thread: the kernels' launch bounds
BOUNDS = {"forward": (128, 256, 512), "backward": (256, 512, 512), "elements": (512, 512)}


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", CSRC, str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)
    return str(d / "plan")


@pytest.mark.parametrize("args,forward", [(a, True) for a in FORWARD] + [(a, False) for a in BACKWARD])
def test_the_planned_ctas_fit_an_sm(program, args, forward):
    out = subprocess.run([program, *map(str, args)], check=True, stdout=subprocess.PIPE, text=True).stdout
    plans = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert plans and plans[0][0] > 256
    bounds = BOUNDS["elements"] if not args[0] else BOUNDS["forward" if forward else "backward"]
    for cols, nch, threads, ctas, stages, smem in plans:
        if not forward and not args[0] and ctas == 1 and nch == 2 and cols <= 8 * WIDE:      # the layer norm's wider rows
            wide = (cols + 255) // 256 * 32
            assert wide <= WIDE and wide * 8 >= cols
        assert threads % 32 == 0 and 64 <= threads <= bounds[{1: 0, 2: 1, 4: 2}[nch]] and threads * 8 * nch >= cols
        assert stages >= 2 and smem == stages * (cols * args[1] + args[2]) <= 200 * 1024
        # 228 KiB of an SM, 1 KiB of it reserved for each CTA
        assert ctas * (smem + args[3] + 1024) <= 228 * 1024, (cols, ctas, stages)


def test_the_constants_are_the_kernels():
    with open(os.path.join(CSRC, "norm.cu")) as f:
        text = f.read()
    assert re.search(r"kFwdOwn = MEAN \? (\d+)", text).group(1) == str(FWD) and re.search(r"kBwdOwn = MEAN \? (\d+)", text).group(1) == str(BWD)
    assert re.search(r"kWideThreads = (\d+)", text).group(1) == str(WIDE) and re.search(r"kLayerThreads = (\d+)", text).group(1) == "256"
