"""Kernels that use tensor memory hold it before they let the next kernel start (CPU).

pdl_launch_dependents lets the next kernel on the stream start its CTAs once every
CTA of this one has signalled.  They allocate their own tensor memory and then wait
for this grid to end.  A CTA that signals before it has its columns could therefore
wait for columns that a dependent holds, and the dependent for it.  So in every
kernel the allocation comes first in the text, and nothing lets another warp signal
before it: the signal is in the allocating warp's own block, or a CTA-wide barrier
lies between.
"""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_gqa_query_b200", "csrc")


def kernels(text):
    """(name, body) of every __global__ function."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__", text):
        open_ = text.index("{", m.start())
        name = re.findall(r"(\w+)\s*\((?:[^()]|\([^()]*\))*\)\s*$", text[m.start():open_])[-1]
        depth, i = 1, open_ + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield name, text[open_ + 1:i - 1]


def signals_behind_the_allocation(body):
    alloc = [m.end() for m in re.finditer(r"\btmem_alloc\w*\(", body)]
    signal = [m.start() for m in re.finditer(r"\bpdl_launch_dependents\(", body)]
    if not alloc or not signal:
        return True
    if signal[0] < max(alloc):
        return False
    between = body[max(alloc):signal[0]]
    depth, low = 0, 0
    for ch in between:
        depth += {"{": 1, "}": -1}.get(ch, 0)
        low = min(low, depth)
    # still inside the block of the allocation, and that is one warp's: if (warp == N) { ... }
    own = low == 0 and re.search(r"if \(warp == \d+\) \{\s*tmem_alloc\w*\($", body[:max(alloc)]) is not None
    return own or re.search(r"__syncthreads\(\)|\bcluster_sync\(\)", between) is not None


FOUND = [(os.path.basename(f), name, body) for f in sorted(glob.glob(os.path.join(CSRC, "*.cu")))
         for name, body in kernels(open(f).read()) if "tmem_alloc" in body]


def test_the_kernels_with_tensor_memory_are_found():
    names = {name for _, name, _ in FOUND}
    assert {"attn_cache_kernel", "attn_prefill_window_kernel", "attn_bwd_window_kernel", "attn_bwd_kernel"} <= names
    assert len(FOUND) >= 8


@pytest.mark.parametrize("file,name,body", FOUND, ids=[f"{f}:{n}" for f, n, _ in FOUND])
def test_tensor_memory_before_the_signal(file, name, body):
    assert signals_behind_the_allocation(body), f"{name} in {file} signals before it holds its tensor memory"


@pytest.mark.parametrize("body,good", [
    ("if (warp == 1) tmem_alloc(&b, 64); __syncthreads(); pdl_launch_dependents();", True),
    ("if (warp == 1) { tmem_alloc(&b, 64); pdl_launch_dependents(); } pdl_wait();", True),
    ("if (warp == 1) tmem_alloc(&b, 64); pdl_launch_dependents();", False),
    ("if (warp == 1) { tmem_alloc(&b, 64); } pdl_launch_dependents();", False),
    ("pdl_launch_dependents(); if (warp == 1) tmem_alloc(&b, 64); __syncthreads();", False),
    ("if (warp == 1) tmem_alloc(&b, 64);", True),
])
def test_the_rule_itself(body, good):
    assert signals_behind_the_allocation(body) == good


@pytest.mark.parametrize("file,name,body", FOUND, ids=[f"{f}:{n}" for f, n, _ in FOUND])
def test_an_aborted_cta_lets_its_products_land_before_it_frees_their_columns(file, name, body):
    """After a wait has run out products may still be in flight: freed columns could be another
    kernel's by the time they are written."""
    free = re.search(r"\btmem_dealloc\w*\(", body)
    land = re.search(r"\bdrain_after_abort\(", body)
    assert free and land and land.start() < free.start()
