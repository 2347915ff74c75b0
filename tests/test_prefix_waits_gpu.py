"""The shared-prefix kernel's waits that run out: builds in which a role polls for another hardly ever or
not at all (copies and products in flight are still waited for), so that warps give up at their
first wait or somewhere on the way. The call returns, its status says so, and the device goes on.

Each build runs in a process of its own (the C++ statics of two copies of the library are one)."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

import pytest
import torch

import q4_moe_speculative_gb300 as dsm
from q4_moe_speculative_gb300 import build

pytestmark = pytest.mark.gpu

TIMEOUT = 5
POLLS = (0, 1, 2)
CASES = [   # prefixes, lens, R, Hq, kv, D, page, q8
    ([513], [11] * 13, 3, 8, 1, 128, 32, False),         # runs of two row tiles and of one
    ([700], [70, 30, 20, 8], 8, 16, 2, 128, 16, True),
    ([3000, 40, 0], [6, 3, 200, 0, 1, 70], 4, 6, 2, 64, 64, False),
    ([300] * 9, [5] * 36, 2, 3, 3, 64, 16, True),
    ([40000], [5] * 16, 1, 16, 2, 128, 64, False),       # every ring full, page after page
    ([130] * 40, [5] * 160, 4, 32, 8, 128, 64, False),   # many runs of a CTA
]


@pytest.fixture(scope="module")
def impatient(tmp_path_factory):
    build.build_library()
    folder = tmp_path_factory.mktemp("impatient")
    others = [build.BUILD / (s.stem + ".o") for s in build.sources() if s.stem != "prefix_tc"]

    def library(polls):
        obj, lib = folder / f"prefix_tc_{polls}.o", folder / f"libdsmoe_{polls}.so"
        for cmd in ([build._nvcc(), *build.NVCC_FLAGS, f"-DDS_PREFIX_WAIT_POLLS={polls}u", "-c",
                     str(build.CSRC / "prefix_tc.cu"), "-o", str(obj)],
                    [build._nvcc(), *build.ARCH, "-shared", "-o", str(lib), str(obj), *map(str, others)]):
            r = subprocess.run(cmd, capture_output=True, text=True)
            assert r.returncode == 0, r.stderr
        return lib

    with ThreadPoolExecutor(len(POLLS)) as pool:
        return dict(zip(POLLS, pool.map(library, POLLS)))


def run(polls, lib):
    from test_prefix_attn_gpu import DEV, check, problem
    dsm.N.LIB_PATH = Path(lib)
    ended = 0
    for i, case in enumerate(CASES):
        p = problem(*case, seed=31)
        ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
        for _ in range(3):
            got = dsm.prefix_attention(*p, workspace=ws)
            status = dsm.workspace_status(ws)
            print(i, status, flush=True)
            assert status == TIMEOUT or (polls and status == 0)
            ended += status == 0
            if status == 0 and i < 4:
                check(*p, got=got)
    x = torch.arange(1000, device=DEV)
    assert int(x.sum()) == 499500
    print("ended", ended)


@pytest.mark.parametrize("polls", POLLS)
def test_waits_that_run_out(impatient, polls):
    r = subprocess.run([sys.executable, __file__, str(polls), str(impatient[polls])], cwd=build.ROOT,
                       env={**os.environ, "PYTHONPATH": f"{build.ROOT}:{Path(__file__).parent}"},
                       capture_output=True, text=True, timeout=300)
    print(r.stdout)
    assert r.returncode == 0, r.stdout + r.stderr


if __name__ == "__main__":
    run(int(sys.argv[1]), sys.argv[2])
