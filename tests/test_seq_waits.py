"""The waits inside the sequence kernels' assembly, in the listing of the
compiler that builds them (no GPU): it keeps its own instructions apart, but
does not look into assembly."""

import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "recommender_sparse_embedding_amd")

SOURCE = """
#include "rse_seqmma.h"
__global__ void by_sixteen(const uint64_t* place, const uint32_t* bytes, uint32_t* out) {
    __shared__ rse::u32x4 lds[64];
    rse::to_lds(reinterpret_cast<const void*>(place[threadIdx.x]), bytes[threadIdx.x], lds);
    rse::loads_left<0>();
    out[threadIdx.x] = lds[threadIdx.x][0];
}
__global__ void by_four(const uint64_t* place, const uint32_t* bytes, uint32_t* out) {
    __shared__ uint32_t lds[64];
    rse::to_lds4(reinterpret_cast<const void*>(place[threadIdx.x]), bytes[threadIdx.x], lds);
    rse::loads_left<0>();
    out[threadIdx.x] = lds[threadIdx.x];
}
"""


# a message's value passes through m0, as a copy's place in LDS does
MESSAGES = """
#include "rse_seqmma.h"
__global__ void between(const uint64_t* place, uint32_t* out, int value) {
    __shared__ rse::u32x4 lds[64];
    const void* p = reinterpret_cast<const void*>(place[threadIdx.x]);
    __builtin_amdgcn_s_sendmsg(1, value);
    rse::to_lds(p, lds);
    __builtin_amdgcn_s_sendmsg(1, value);
    rse::loads_left<0>();
    out[threadIdx.x] = lds[threadIdx.x][0];
}
"""


def _listing(tmp_path, source):
    spec = importlib.util.spec_from_file_location("_rse_build_flags", os.path.join(PACKAGE, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    try:
        cc = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    at = tmp_path
    (at / "waits.hip").write_text(source)
    r = subprocess.run([cc, *build.HIPCC_FLAGS, "-S", "--cuda-device-only", "-I", os.path.join(PACKAGE, "csrc"),
                        str(at / "waits.hip"), "-o", str(at / "waits.s")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return (at / "waits.s").read_text()


def _instructions(listing):
    """(operation, operands) in order; a label or the listing's own lines end a run."""
    for line in listing.splitlines():
        line = line.split(";")[0].strip()
        if line and not line.startswith((".", "#")) and not line.endswith(":"):
            op, _, rest = line.partition(" ") if " " in line else line.partition("\t")
            yield op.strip(), [x.strip() for x in rest.replace("\t", " ").split(",")]


def _scalars(operand):
    one, many = re.fullmatch(r"s(\d+)", operand), re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    return {int(one[1])} if one else set(range(int(many[1]), int(many[2]) + 1)) if many else set()


def test_scalar_addresses_wait_for_the_vector_instruction_that_wrote_them(tmp_path):
    """Five wait states from a vector instruction's write of a scalar register
    to a memory instruction that reads it."""
    run = list(_instructions(_listing(tmp_path, SOURCE)))
    loads = [i for i, (op, _) in enumerate(run) if op.startswith("global_load_lds")]
    assert len(loads) == 2
    for i in loads:
        read, waited, written = set().union(*(_scalars(x) for x in run[i][1])), 0, False
        assert read, "a scalar address"
        for op, args in reversed(run[:i]):
            if op.startswith(("v_readfirstlane", "v_readlane")) and _scalars(args[0]) & read:
                written = True
                assert waited >= 5, f"{waited} wait states before {run[i]}"
                break
            waited += 1 + (int(args[0]) if op == "s_nop" else 0)
        assert written, "the address comes from a vector register"


def test_m0_is_not_kept_over_a_copy(tmp_path):
    """What the compiler put into m0 before a copy it puts there again behind it
    (compiled only)."""
    run = list(_instructions(_listing(tmp_path, MESSAGES)))
    ops = [op if op != "s_mov_b32" else f"{op} {args[0]}" for op, args in run]
    ops = [op for op in ops if op in ("s_mov_b32 m0", "s_sendmsg") or op.startswith("global_load_lds")]
    assert ops == ["s_mov_b32 m0", "s_sendmsg", "s_mov_b32 m0", "global_load_lds_dwordx4", "s_mov_b32 m0", "s_sendmsg"]
