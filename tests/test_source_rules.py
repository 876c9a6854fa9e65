"""Rules that the CUDA sources keep and that no run can show broken (no GPU is touched)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lora_co_serving_gb300", "csrc")


def source(path):
    """A file's text without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


FILES = {os.path.basename(p): source(p) for p in sorted(glob.glob(os.path.join(CSRC, "*.cu")) +
                                                        glob.glob(os.path.join(CSRC, "*.h")))}


def kernels():
    """(file, name, parameter list, body) of every kernel."""
    for name, text in FILES.items():
        for m in re.finditer(r"__global__\s+void\s+(?:__\w+__\s*\([^()]*\)\s*|__cluster_dims__\s*\([^()]*\)\s*)*(\w+)\s*\(", text):
            at, depth = m.end(), 1
            while depth:
                depth += {"(": 1, ")": -1}.get(text[at], 0)
                at += 1
            args, at = text[m.end():at - 1], text.index("{", at) + 1
            start, depth = at, 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            yield name, m.group(1), args, text[start:at]


def test_kernels_are_found():
    assert len(list(kernels())) == sum(len(re.findall(r"__global__\s+void", t)) for t in FILES.values()) > 15


@pytest.mark.parametrize("file,name,args,body", [pytest.param(*k, id=k[1]) for k in kernels() if "grid_dep_wait" in k[3]])
def test_early_kernels_promise_nothing_about_their_arguments(file, name, args, body):
    """A kernel that waits for the launch before it starts while that launch may still write what it is going to read.
    A __restrict__ argument promises that nobody writes the data while the kernel runs: the compiler may then read it
    through the cache that is not kept coherent, and ahead of the wait."""
    assert "__restrict__" not in args and "__ldg" not in body and "ld.global.nc" not in body


def test_no_load_is_multicast_over_a_cluster():
    """The library also runs where several GPUs see one another's memory; a bulk load that lands in several CTAs is kept
    out of it.  (Commits of tensor-core work may arrive on both CTAs of a pair: they move no data.)"""
    for name, text in FILES.items():
        for m in re.finditer(r"cp\.async\.bulk[^;]*", text):
            assert "multicast" not in m.group(0), name


@pytest.mark.parametrize("file,name,args,body", [pytest.param(*k, id=k[1]) for k in kernels()
                                                 if k[0] == "fp8_linear.cu" and "tcgen05.alloc" in k[3]])
def test_commits_of_the_products_end_before_their_cta(file, name, args, body):
    """Commits of tensor-core work arrive on barriers in shared memory, whoever owns that by then: each kernel of the 8-bit
    products waits for those that no other role waits for (the stages' last ones)."""
    called = set(re.findall(r"(\w+)(?:<[^<>;]*>)?\s*\(", body))
    text = body
    for m in re.finditer(r"__device__ __forceinline__ void (\w+)\([^)]*\) \{(.*?)\n\}\n", FILES[file], flags=re.S):
        if m.group(1) in called:
            text += m.group(2)
    assert "mma_commit(" in text and "await_commits(ring" in text


def test_the_benchmark_has_the_main_pass_traffic_of_these_sources():
    """The benchmark reports the DRAM bytes of a committed profile only while it belongs to the sources, all of them."""
    import json
    import bench
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "profiles", "fwd_main_traffic.json")) as f:
        cfg = json.load(f)["config"]
    assert bench.profiled_traffic(cfg) is not None
    named = re.findall(r'#include "(\w+\.h)"', open(os.path.join(CSRC, "tc_kernel.cu")).read())
    with open(os.path.join(root, "bench.py")) as f:
        hashed = re.search(r"def kernel_hash.*?\n\n", f.read(), flags=re.S).group(0)
    assert "tc_prims.h" in named and all(n in hashed for n in named)
