"""The streamed norm's grid: every CTA that the plan counts as resident fits an SM beside the others."""

import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_block_sparse_attn_b200",
                    "csrc")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text("""#include "stream_plan.h"
extern "C" void plan(int resident, int threads, long long stage, long long staged, long long fixed, long long* out) {
  const qbsa::StreamPlan p = qbsa::plan_stream(resident, threads, stage, staged, fixed);
  out[0] = p.per_sm, out[1] = p.stages, out[2] = p.smem;
}
""")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(so), str(src)], check=True)
    fn = ctypes.CDLL(str(so)).plan
    fn.argtypes = [ctypes.c_int, ctypes.c_int] + [ctypes.c_longlong] * 3 + [ctypes.c_void_p]

    def call(*args):
        out = (ctypes.c_longlong * 3)()
        fn(*args, out)
        return tuple(out)
    return call


def _call(plan, width, size, residual, aligned, regs, fixed):
    """As the launch asks: rows of `width` values of `size` bytes, four 16-byte pieces per thread (two for
    unaligned rows with a residual)."""
    pieces = -(-width * size // 16)
    each = 2 if residual and not aligned and pieces <= 1024 else 4
    threads = -(-(-(-pieces // each)) // 32) * 32
    slot = pieces * 16 + (0 if aligned else 16)
    resident = 128 * min(16, 16384 // (32 * (-(-regs // 8) * 8)))
    return threads, resident, plan(resident, threads, slot * (1 + residual), 0 if aligned or not residual else 2 * slot,
                                   fixed)


@pytest.mark.parametrize("size", [2, 4])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("aligned", [False, True])
def test_what_is_planned_as_resident_fits(plan, size, residual, aligned):
    for regs in (58, 64, 72, 85, 93):
        for fixed in (384, 640):
            for width in range(128 if aligned else 257, 2560 * 16 // size + 1, 16 // size if aligned else 7):
                threads, resident, (per_sm, stages, smem) = _call(plan, width, size, residual, aligned, regs, fixed)
                if stages < 2:
                    continue
                cta = -(-(smem + fixed + 1024) // 128) * 128           # shared memory comes in units of 128 bytes
                assert per_sm >= 1 and per_sm * cta <= 233472
                assert per_sm == 1 or per_sm * threads <= resident
                assert smem <= 216 * 1024 and 2 <= stages <= 4


@pytest.mark.parametrize("width,size,residual,regs,fixed,want", [
    # as cudaOccupancyMaxActiveBlocksPerMultiprocessor counts them for these registers
    (640, 4, True, 69, 640, (13, 3)), (1024, 4, True, 69, 640, (12, 2)), (1536, 4, True, 69, 640, (8, 2)),
    (480, 4, False, 66, 384, (25, 4)), (640, 2, True, 85, 640, (19, 4)), (688, 2, True, 85, 640, (18, 4)),
    (4096, 2, True, 85, 640, (5, 2)), (5120, 2, True, 85, 640, (4, 2)), (5120, 2, False, 78, 384, (4, 4)),
])
def test_known_plans(plan, width, size, residual, regs, fixed, want):
    assert _call(plan, width, size, residual, True, regs, fixed)[2][:2] == want
