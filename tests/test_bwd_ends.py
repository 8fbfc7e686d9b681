"""The causal backward's main kernel comes to its end when one of its waits runs out (CPU).

The file (csrc/attn_bwd.cu) is compiled unchanged against tests/fake_device, a model of
one CTA whose copies, products and commits complete in any order.  A copy or a commit
gets lost, or a wait runs out while the other warps still go on: no warp may stay at a
barrier that has no limit.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_gqa_query_b200", "csrc")
FAKE = os.path.join(ROOT, "tests", "fake_device")
CUDA_INC = "/usr/local/cuda/include"


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    if not shutil.which("g++") or not os.path.exists(os.path.join(CUDA_INC, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    folder = str(tmp_path_factory.mktemp("ends"))
    for path in [os.path.join(FAKE, n) for n in os.listdir(FAKE)] + [os.path.join(CSRC, n) for n in ("attn.cuh", "attn_bwd.cu")]:
        shutil.copy(path, folder)
    out = os.path.join(folder, "ends")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I", CUDA_INC, os.path.join(folder, "bwd_ends.cpp"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


@pytest.mark.parametrize("fault", ["nothing", "lost_copy", "lost_commit", "timeout"])
@pytest.mark.parametrize("d", [64, 128])
def test_every_warp_ends(exe, d, fault):
    r = subprocess.run([exe, str(d), "2", "1000", "2", "2", "1", "1", "1000", "1", fault], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    gave_up = int(r.stdout.split(",")[1].split()[0])
    assert (gave_up == 0) == (fault == "nothing"), r.stdout
