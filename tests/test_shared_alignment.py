"""Arrays in shared memory that are read or written 16 bytes at a time: an array of words alone has an alignment of
four bytes, and where it lies is up to the compiler, so that each has to ask for its 16."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_ffn_gb300", "csrc")
WIDE = r"(?:float4|uint4|int4|double2|ulonglong2)"


def misaligned(text):
    """Names of the shared arrays that are taken as vectors of 16 bytes and do not ask for the alignment."""
    found = []
    # a declaration counts up to the next kernel or function, where the name may be another thing
    for decl in re.finditer(r"(?<!extern )__shared__\s+((?:alignas|__align__)\s*\(\s*\d+\s*\)\s*)?(\w+)\s+(\w+)\s*\[[^;]*?\];", text):
        aligned, kind, name = decl.groups()
        if re.fullmatch(WIDE, kind) or (aligned and int(re.search(r"\d+", aligned).group()) >= 16):
            continue
        body = re.split(r"__global__|\n}\n", text[decl.end():])[0]
        if re.search(r"reinterpret_cast<\s*(?:const\s+)?" + WIDE + r"\s*(?:const\s*)?\*\s*>\(\s*&?" + name + r"\b", body):
            found.append(name)
    return found


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_vectors_in_shared_memory_are_aligned(name):
    with open(os.path.join(CSRC, name)) as f:
        assert misaligned(f.read()) == []


def test_the_search_finds_them():
    bad = "__shared__ int sh;\n__shared__ float vs[128];\nfloat4 q = *reinterpret_cast<const float4 *>(vs + c);\n}\n"
    assert misaligned(bad) == ["vs"]
    assert misaligned(bad.replace("__shared__ float", "__shared__ __align__(16) float")) == []
    assert misaligned(bad.replace("__shared__ float", "__shared__ alignas(8) float")) == ["vs"]
    assert misaligned(bad.replace("(vs + c)", "(other + c)")) == []
