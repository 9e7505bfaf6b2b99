"""Kernels that start under programmatic dependent launch run while the previous kernel still writes. What
they read must not be declared read-only: a load through the non-coherent path (__ldg) or through a
`const __restrict__` pointer may be moved above griddep_wait() and then returns what was there before
(a stale tile list sends loads out of range). Checked on the source: no function that waits, nor one
that it calls, has such a load."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_nvfp4_gemm_gb300", "csrc")
READ_ONLY = re.compile(r"__ldg\s*\(|const\s+\w+\s*\*\s*__restrict__|ld\.global\.nc")


def definitions(path):
    """Top-level definitions of a source file (they end with a brace in the first column), without comments."""
    text = re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S))
    text = re.sub(r"__launch_bounds__\s*\([^()]*\)", "", text)
    return [d for d in re.split(r"^\};?$", text, flags=re.M) if "{" in d]


def names(definition):
    """What a definition can be called by: its function's, or struct's and member functions' names."""
    struct = re.search(r"\bstruct\s+(\w+)\s*\{", definition)
    head = re.findall(r"(?:DEVI|__global__)[^;{]*?\b(\w+)\s*\([^;{]*\)\s*(?:const\s*)?\{", definition)
    return set(head) | ({struct.group(1)} if struct else set())


def offenders(files):
    defs = [(os.path.basename(f), d) for f in files for d in definitions(f)]
    # launched in the ordinary way: they start after the previous kernel has completed
    bad = {n for _, d in defs if READ_ONLY.search(d) for n in names(d)}
    found, grown = [], True
    while grown:  # callers of such functions, however deep
        more = {n for _, d in defs for n in names(d) if any(re.search(rf"\b{b}\b\s*[<(]", d) for b in bad)}
        grown = not more <= bad
        bad |= more
    for f, d in defs:
        if re.search(r"griddep_wait\s*\(\s*\)\s*;", d) and names(d) & bad:
            found += [(f, n) for n in sorted(names(d) & bad)]
    return found


def test_waiting_kernels_read_with_plain_loads():
    assert offenders(sorted(glob.glob(os.path.join(CSRC, "*.cu")))) == []


@pytest.mark.parametrize("body,bad", [
    ("DEVI int first(const int* p) {\n  return __ldg(p);\n}\n__global__ void k(const int* p) {\n  griddep_wait();\n  first(p);\n}\n", True),
    ("DEVI int first(const int* p) {\n  return p[0];\n}\n__global__ void k(const int* p) {\n  griddep_wait();\n  first(p);\n}\n", False),
    ("__global__ void k(const int* __restrict__ p) {\n  griddep_wait();\n  use(p[0]);\n}\n", True),
    ("__global__ void k(const int* __restrict__ p) {\n  use(p[0]);\n}\n", False)])
def test_the_check_itself(tmp_path, body, bad):
    f = tmp_path / "a.cu"
    f.write_text(body)
    assert bool(offenders([str(f)])) == bad
