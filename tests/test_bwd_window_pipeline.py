"""Order of the waits inside the windowed backward's main kernel, on the CPU.

The kernel (csrc/attn_bwd_window.cu) is a pipeline of five roles over rings of
shared memory and over tensor memory that is full, handed from role to role by
mbarriers.  A wait names only a phase's parity, so a role that does not wait for
every phase of a barrier can be let through by the phase before the one it means,
when loads or products are late: results are then wrong without an error, on a
machine and a moment of their own.  Repeating a run on a GPU shows little of that.

Here the file is compiled unchanged against tests/fake_device: a model of one CTA
whose copies, products and commits complete in any order that the hardware allows,
with one kind of them made much later than the rest.  Every product, every read and
write of tensor memory and every reuse of shared memory is checked against the list
of (key tile, query tile) pairs that the CTA stands for.

Waits taken out of a copy of the source must be caught.  And when a wait runs out,
the kernel has to end.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_gqa_query_b200", "csrc")
FAKE = os.path.join(ROOT, "tests", "fake_device")
CUDA_INC = "/usr/local/cuda/include"

LATE = ["nothing", "copies", "commits", "products", "reads"]

# d, B, T, G, k, n_shared, sg, window, sinks
CASES = {
    "ragged": (64, 24, 1000, 3, 2, 1, 1, 200, 3),               # walks of a few pairs, several a CTA
    "one_pair_walks": (64, 300, 100, 2, 1, 1, 0, 50, 0),        # every pair is a walk's first and last
    "long_sink_walks": (64, 6, 5000, 2, 1, 1, 1, 300, 140),
    "two_rounds": (64, 40, 1400, 4, 1, 1, 1, 700, 3),
    "no_bound": (64, 4, 1300, 2, 3, 0, 0, 1300, 0),
    "d128_ragged": (128, 24, 1000, 3, 2, 1, 1, 200, 3),
    "d128_one_pair_walks": (128, 300, 100, 2, 1, 1, 0, 50, 0),
    "d128_two_rounds": (128, 32, 1400, 2, 1, 1, 0, 700, 3),
}


def build(folder, edit=None):
    if not shutil.which("g++") or not os.path.exists(os.path.join(CUDA_INC, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    for name in os.listdir(FAKE):
        shutil.copy(os.path.join(FAKE, name), folder)
    shutil.copy(os.path.join(CSRC, "attn.cuh"), folder)
    with open(os.path.join(CSRC, "attn_bwd_window.cu")) as f:
        src = f.read()
    if edit:
        assert src.count(edit[0]) == 1, edit[0]
        src = src.replace(*edit)
    with open(os.path.join(folder, "attn_bwd_window.cu"), "w") as f:
        f.write(src)
    exe = os.path.join(folder, "pipeline")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I", CUDA_INC, os.path.join(folder, "bwd_window_pipeline.cpp"), "-o",
                        exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def run(exe, case, trials, late):
    r = subprocess.run([exe, *map(str, CASES[case]), str(trials), "1", late], capture_output=True, text=True, timeout=300)
    return r.returncode, r.stdout + r.stderr


@pytest.fixture(scope="module")
def pipeline(tmp_path_factory):
    return build(str(tmp_path_factory.mktemp("pipeline")))


@pytest.mark.parametrize("late", LATE)
@pytest.mark.parametrize("case", list(CASES))
def test_every_pair_meets_its_own_tiles(pipeline, case, late):
    rc, out = run(pipeline, case, 100, late)
    assert rc == 0, out
    assert ("2 rounds" in out) == case.endswith("two_rounds")


@pytest.mark.parametrize("fault", ["lost_copy", "lost_commit", "timeout"])
@pytest.mark.parametrize("case", ["ragged", "one_pair_walks", "d128_ragged", "d128_one_pair_walks"])
def test_a_wait_that_runs_out_ends_the_kernel(pipeline, case, fault):
    """A copy or a commit never comes, or a wait runs out while the others still go on: every warp
    must come to the end, none may stay at a barrier that has no limit."""
    rc, out = run(pipeline, case, 400, fault)
    assert rc == 0, out


# a wait taken out of the source, where it must show
PLANTED = {
    "the drain reads dV, dK behind their parities alone":
        ("      if (!wait(&bar->dq_full, N)) break;\n",
         "      if (!c.last() || C::kWide) { if (!wait(&bar->dq_full, N)) break; }\n", "ragged", "copies"),
    "P over P that dV has not read":
        ("if (N > 0 && !wait(&bar->pv_done, N - 1)) break;", "", "ragged", "copies"),
    "dV, dK over the last key tile's":
        ("if (c.first() && c.item > 0 && !wait_w(&bar->acc_free, c.item - 1)) break;\n          tc_fence_after();\n"
         "          if (leader) {\n            product_ts(tmem + C::kDV",
         "tc_fence_after();\n          if (leader) {\n            product_ts(tmem + C::kDV", "one_pair_walks", "nothing"),
    "S over S that was not read":
        ("if (!none && !wait_w(&bar->s_free, N)) break;", "", "ragged", "nothing"),
    "K over K that dQ has not read":
        ("mbar_init(&bar->k_empty[i], 2); ", "mbar_init(&bar->k_empty[i], 1); ", "one_pair_walks", "commits"),
    "dS over dS that its products have not read":
        ("if (ch == 0 && N > 0) ok = wait(C::kWide ? &bar->dk_done : &bar->dq_full, N - 1);", "", "d128_ragged", "products"),
    "a staging buffer over one that is being stored":
        ("if (lane == 0) bulk_wait_read<0>();", "", "ragged", "reads"),
}


@pytest.mark.parametrize("what", list(PLANTED))
def test_a_missing_wait_is_caught(tmp_path, what):
    old, new, case, late = PLANTED[what]
    exe = build(str(tmp_path), (old, new))
    rc, out = run(exe, case, 300, late)
    assert rc == 1, out
