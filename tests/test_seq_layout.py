"""Layout of what the sequence kernels hold in LDS, by the compiler that builds
them (no GPU): structures read by 16-byte accesses have to keep them aligned in
every element of an array."""

import importlib.util
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "recommender_sparse_embedding_amd")

SOURCE = """
#include <cstddef>
#include "rse_seqmma.h"
using rse::KeySide;
template <int KT>
constexpr bool ok = alignof(KeySide<KT>) % 16 == 0 && sizeof(KeySide<KT>) % 16 == 0 &&
                    offsetof(KeySide<KT>, mask) % 16 == 0 && offsetof(KeySide<KT>, pos) % 16 == 0;
static_assert(ok<32>, "tiles of 32 keys");
static_assert(ok<64>, "tiles of 64 keys");
"""


def test_key_sides_are_aligned(tmp_path):
    spec = importlib.util.spec_from_file_location("_rse_build_flags", os.path.join(PACKAGE, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    try:
        cc = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    src = tmp_path / "layout.hip"
    src.write_text(SOURCE)
    r = subprocess.run([cc, *build.HIPCC_FLAGS, "-fsyntax-only", "-I", os.path.join(PACKAGE, "csrc"), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
