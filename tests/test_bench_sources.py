"""What the bench's hash of the step's sources covers: all of rse.h but the
declarations of the sequence operators."""

import importlib.util
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bench():
    spec = importlib.util.spec_from_file_location("_bench_sources", os.path.join(ROOT, "bench.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def header():
    with open(os.path.join(ROOT, "include", "rse.h"), "rb") as f:
        return f.read()


def _functions(text):
    return re.findall(rb"^\w+ (\w+)\(", text, re.M)


def test_all_but_the_sequence_operators_is_hashed(bench, header):
    kept, every = _functions(bench.step_header(header)), _functions(header)
    assert kept == [f for f in every if b"seq" not in f] and len(kept) < len(every)


def test_changes_of_titles_never_hide_other_text(bench, header):
    """Whatever becomes of the title lines, the hash covers every other section."""
    step = [f for f in _functions(header) if b"seq" not in f]
    titles = [m.group(0) for m in re.finditer(rb"^/\* -{2,} .* -{2,} \*/$", header, re.M)]
    assert len(titles) >= 5
    for t in titles:
        for new in (b"/* another title */", t.replace(b"--", b"-----"), t + b"\n" + t, b""):
            got = _functions(bench.step_header(header.replace(t, new)))
            assert [f for f in got if b"seq" not in f] == step, t


def test_changes_of_text_change_the_hash(bench, header):
    kept = bench.step_header(header)
    for f in _functions(header):
        changed = bench.step_header(header.replace(f + b"(", f + b"(int more, ", 1)) != kept
        assert changed == (b"seq" not in f), f


def test_a_new_section_is_hashed(bench, header):
    """Also one that stands right behind the sequence operators'."""
    for m in re.finditer(rb"^/\* -{2,} .* -{2,} \*/$", header, re.M):
        new = header[:m.start()] + b"/* ------ something else ------ */\nint other_call(int x);\n" + header[m.start():]
        assert b"other_call" in bench.step_header(new)
