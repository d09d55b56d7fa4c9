"""CPU checks of properties of the CUDA sources that a run cannot show: what they guard
against is undefined behaviour, which may pass on any one compiler."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fine_grained_fp8_persistent_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))


def _code(path):
    """The file without comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _functions(code):
    """(name, body) of the __device__ __forceinline__ functions."""
    for m in re.finditer(r"__device__ __forceinline__ [\w ]+?\b(\w+)\(([^{;]*)\) \{", code):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(code[i], 0)
            # braces of register lists inside asm strings come in pairs
            i += 1
        yield m.group(1), code[m.end():i]


def test_wrappers_converge_first():
    """The cluster barrier (it follows loops that lanes leave at different times) and the TMEM
    allocation and release, whatever stands before the call."""
    seen = set()
    for path in SOURCES:
        for name, body in _functions(_code(path)):
            if name in ("cluster_sync_all", "tc_alloc", "tc_dealloc", "tmem_alloc", "tmem_dealloc"):
                assert body.lstrip().startswith("__syncwarp();"), f"{os.path.basename(path)}: {name}"
                seen.add(name)
    assert len(seen) == 5


def test_aligned_instructions_stand_in_wrappers_only():
    for path in SOURCES:
        code = _code(path)
        inside = sum(body.count(".aligned") for _, body in _functions(code))
        assert code.count(".aligned") == inside, os.path.basename(path)


# (file, what lanes run apart, expected next): TMEM loads follow in the loop or behind it
DIVERGENT = [
    ("gemm_persistent.cuh", r"ptx::bulk_commit_group\(\);\s*\}"),                 # lane 0's store, by TMA
    ("gemm_persistent.cuh", r"store_row32\(args\.D, row_off, tl\.n_blk \* BN \+ 32 \* c, N, reinterpret_cast<const float\*>\(v\), bf16\);"),
    ("gemm_persistent.cuh", r"fused_group_out\(args, PackedBf16\{hv\}, amax, \(tl\.n_blk \* BN\) / 128 \+ g, grow, row_ok\);"),
    ("gemm_persistent.cuh", r"row_ok = false;\s*\}\s*\}"),                       # rows of another expert
    ("gated_gemm.cuh", r"ptx::bulk_commit_group\(\);\s*\}"),
    ("gated_thin.cuh", r"__nanosleep\(1000\);\s*\}"),                             # the wait after an abort
]


@pytest.mark.parametrize("name,what", DIVERGENT, ids=range(len(DIVERGENT)))
def test_lanes_meet_before_the_next_tmem_load(name, what):
    code = _code(os.path.join(CSRC, name))
    found = list(re.finditer(what, code))
    assert found
    for m in found:
        assert code[m.end():].lstrip().startswith("__syncwarp();"), code[m.start(): m.end() + 80]


def test_matrix_vector_chunks_begin_converged():
    """ldmatrix and mma.sync follow."""
    code = _code(os.path.join(CSRC, "gemv.cuh"))
    assert re.search(r"cp_wait<C::DEPTH - 2>\(\);\s*__syncwarp\(\);\s*issue\(\);", code)


def test_kernels_that_start_early_read_coherently():
    """Under a programmatic launch the kernel before may still write what this one is about to
    read: the read-only path, whose data nobody may write while the kernel runs, is not for
    it, nor for anything that the compiler may read above the wait."""
    checked = 0
    for path in SOURCES:
        code = _code(path)
        assert "ld.global.nc" not in code, os.path.basename(path)
        if "griddep_wait();" in code:
            assert "__ldg(" not in code, os.path.basename(path)
            checked += 1
    assert checked >= 5
    ptx = _code(os.path.join(CSRC, "ptx.cuh"))
    assert ptx.count('asm volatile("ld.global.') == 3
