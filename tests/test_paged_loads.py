"""How the page-cache kernels load what kernels before them may still be
writing.  They are launched programmatically, so a kernel's life begins before
the one in front of it ends: the read-only path is not defined for such data,
and loads that the compiler takes for invariant may be moved above the wait."""
import os
import re

import pytest

from quantized_exact_attention_gb300 import build as B

SOURCES = ("sage_paged.h", "sage_paged_sched.cuh", "sage_paged.cu", "sage_paged_tiles.cu", "sage_tables.cu")


def unordered_loads(src: str) -> list:
    """Loads of global memory in src that griddepcontrol.wait does not hold back."""
    src = re.sub(r"//[^\n]*|/\*.*?\*/", "", src, flags=re.S)
    found = re.findall(r"__ld\w+|__restrict\w*|\.nc\b", src)
    # an asm statement that loads is volatile and clobbers memory
    for m in re.finditer(r"\basm\b(\s+volatile)?\s*\((.*?)\);", src, flags=re.S):
        if re.search(r"\bld\.(?!shared)", m[2]) and not (m[1] and '"memory"' in m[2]):
            found.append(m[0])
    return found


@pytest.mark.parametrize("name", SOURCES)
def test_no_load_may_pass_the_wait(name):
    with open(os.path.join(B.CSRC, name)) as f:
        assert unordered_loads(f.read()) == []


@pytest.mark.parametrize("planted", [
    "int v = __ldg(p.kv_len + b);", "float4 y = __ldcg(po);", "const int* __restrict__ t = p.table;",
    'asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(a) : "memory");',
    'asm("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(a));', 'asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(a));'])
def test_the_check_finds_what_it_looks_for(planted):
    assert unordered_loads(planted)
    assert not unordered_loads("// " + planted)
