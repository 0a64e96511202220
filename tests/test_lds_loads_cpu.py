"""The loads straight to LDS in the compiler's listing of a kernel that makes them: a wait state
behind the write of M0, which holds their place, and five behind a vector instruction's write of a
scalar register that they read."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from swish_activation_backward_amd import build

SOURCE = """
#include "mma.hpp"
using namespace swg;
extern "C" __global__ void loads(const void* p, float* out, uint32_t bytes, uint32_t soff) {
  __shared__ __attribute__((aligned(1024))) uint16_t ring[8192];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const __amdgpu_buffer_rsrc_t r = make_rsrc(uniform_ptr(p), bytes);
  dma16s<0>(r, threadIdx.x * 16, soff, ring + wave * 512);
  dma16s<4096>(r, threadIdx.x * 16, soff + 64, ring + wave * 512);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  out[threadIdx.x] = ring[threadIdx.x] + ring[threadIdx.x + 2048];
}
"""


def listing(tmp_path):
    try:
        hipcc = build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc here")
    src = tmp_path / "loads.hip"
    src.write_text(SOURCE)
    cmd = [hipcc, "-O3", "-std=c++17", f"--offload-arch={build.ARCH}", *build.DEVICE_FLAGS,
           "-I", build.CSRC, "--cuda-device-only", "-S", str(src), "-o", str(tmp_path / "loads.s")]
    subprocess.run(cmd, check=True, capture_output=True, cwd=tmp_path)
    return (tmp_path / "loads.s").read_text()


def scalars(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]|s(\d+)", operand)
    if not m:
        return set()
    return {int(m[3])} if m[3] else set(range(int(m[1]), int(m[2]) + 1))


def waits(text):
    """(wait states behind the write of M0, least ones behind a vector write of an operand) of each
    load to LDS."""
    found, now, m0, written = [], 0, None, {}
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        if not line or line.startswith(".") or line.endswith(":"):
            continue
        op, _, rest = line.partition("\t" if "\t" in line else " ")
        args = [a.split()[0] for a in rest.split(",") if a.strip()]
        if op == "s_nop":
            now += int(args[0], 0) + 1
            continue
        now += 1
        if re.search(r"\blds\b", rest):
            reads = set().union(*(scalars(a) for a in args))
            found.append((now - m0 - 1, min([now - written[r] - 1 for r in reads if r in written],
                                            default=99)))
        if args and op.startswith("s_") and args[0] == "m0":
            m0 = now
        for r in scalars(args[0]) if args else ():
            if op.startswith("v_"):
                written[r] = now
            elif op.startswith("s_"):
                written.pop(r, None)
    return found


def test_wait_states(tmp_path):
    found = waits(listing(tmp_path))
    assert len(found) == 2
    for m0, scalar in found:
        assert m0 >= 1 and scalar >= 5


def test_the_reader_of_listings():
    """Planted: no wait, one instruction between, a no-operation, a fresh scalar."""
    load = "buffer_load_dwordx4 v1, s[0:3], s4 offen lds"
    assert waits(f"\ts_add_u32 m0, s7, 0\n\t{load}") == [(0, 99)]
    assert waits(f"\ts_mov_b32 m0, s7\n\tv_add_u32_e32 v2, 1, v2\n\t{load}") == [(1, 99)]
    assert waits(f"\ts_mov_b32 m0, s7\n\ts_nop 1\n\t{load}") == [(2, 99)]
    text = f"\tv_readfirstlane_b32 s4, v9\n\ts_mov_b32 m0, s7\n\ts_nop 0\n\t{load}"
    assert waits(text) == [(1, 2)]
