"""Calls of the rotary and tree entries that are refused on the host, before any
CUDA call; the frequencies and their turns; how the kernels load."""
import ctypes
import math
import os
import re
import subprocess
from fractions import Fraction

import pytest
import torch

import quantized_exact_attention_gb300 as S
from quantized_exact_attention_gb300 import build as B
from tests.test_paged_loads import unordered_loads
from tests.tree_support import TWO_PI

R = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    B.build()
    return S.load_library()


def tensor(ptr=0x10000, sb=128 * 128, sh=128, sn=128 * 8):
    return S.sage_tensor(ptr, sb, sh, sn)


def cache(k=None, v=None, pages=64, page=16, heads=8, D=128):
    return S.sage_page_cache(k or tensor(), v or tensor(0x900000), pages, page, heads, D)


def rotary(turns=0x7000, dim=128, interleaved=0, amplitude=1.0):
    return S.sage_rotary(turns, dim, interleaved, amplitude)


BAD_ROTARY = [(dict(turns=None), S.SAGE_ERR_ARG), (dict(dim=0), S.SAGE_ERR_ARG), (dict(dim=-16), S.SAGE_ERR_ARG),
              (dict(dim=144), S.SAGE_ERR_UNSUPPORTED), (dict(dim=24), S.SAGE_ERR_UNSUPPORTED),
              (dict(turns=0x7008), S.SAGE_ERR_UNSUPPORTED)]


def test_rope_refuses(lib):
    def call(x=None, out=None, B=2, H=8, N=4, D=128, positions=None, stride=0, r=None):
        x, out, r = x or tensor(), out or tensor(0x90000), r or rotary()
        return lib.sage_rope(R(x), R(out), B, H, N, D, positions, stride, None, None, R(r), 0, None)

    for bad in (dict(x=tensor(ptr=0)), dict(out=tensor(ptr=0)), dict(B=0), dict(H=0), dict(N=0), dict(H=-1),
                dict(positions=0x8000, stride=-1),
                dict(out=tensor(sh=256)), dict(out=tensor(sb=1 << 20)), dict(out=tensor(sn=2048))):  # x's memory, other strides
        assert call(**bad) == S.SAGE_ERR_ARG, bad
    for bad in (dict(x=tensor(ptr=0x10008)), dict(out=tensor(ptr=0x90004)), dict(x=tensor(sn=100)), dict(x=tensor(sh=-128)),
                dict(D=96), dict(D=256), dict(out=tensor(0x90000, sh=0)), dict(out=tensor(0x90000, sb=64)),
                dict(out=tensor(0x90000, sn=0)), dict(B=1 << 16, N=1 << 15)):
        assert call(**bad) == S.SAGE_ERR_UNSUPPORTED, bad
    for bad, code in BAD_ROTARY:
        assert call(r=rotary(**bad)) == code, bad
    assert call(D=64, r=rotary(dim=80)) == S.SAGE_ERR_UNSUPPORTED
    t = tensor()
    assert lib.sage_rope(R(t), R(t), 1, 1, 1, 128, None, 0, None, None, None, 0, None) == S.SAGE_ERR_ARG
    assert lib.sage_rope(None, R(t), 1, 1, 1, 128, None, 0, None, None, R(rotary()), 0, None) == S.SAGE_ERR_ARG
    # a token of one request may share memory under any strides of axes of one
    assert call(x=tensor(sb=128), out=tensor(sb=256), B=1, N=0) == S.SAGE_ERR_ARG


def test_cache_append_rope_refuses(lib):
    def call(k=None, v=None, B=1, N=1, slots=0x20000, stride=1, positions=None, pstride=0, r=None, c=None):
        k, v, r, c = k or tensor(), v or tensor(), r or rotary(), c or cache()
        return lib.sage_cache_append_rope(R(k), R(v), B, N, slots, stride, positions, pstride, None, R(r), R(c), None)

    for bad in (dict(B=0), dict(N=0), dict(slots=None), dict(stride=-1), dict(k=tensor(ptr=0)), dict(v=tensor(ptr=0)),
                dict(positions=0x8000, pstride=-2), dict(c=cache(pages=0)), dict(c=cache(heads=0))):
        assert call(**bad) == S.SAGE_ERR_ARG, bad
    for bad in (dict(v=tensor(ptr=0x10002)), dict(B=1 << 16, N=1 << 15), dict(c=cache(page=24)), dict(c=cache(D=96)),
                dict(c=cache(k=tensor(sn=0))), dict(c=cache(D=64))):         # 128 rotated channels of 64
        assert call(**bad) == S.SAGE_ERR_UNSUPPORTED, bad
    for bad, code in BAD_ROTARY:
        assert call(r=rotary(**bad)) == code, bad
    t, r, c = tensor(), rotary(), cache()
    assert lib.sage_cache_append_rope(R(t), R(t), 1, 1, 0x20000, 1, None, 0, None, R(r), None, None) == S.SAGE_ERR_ARG
    assert lib.sage_cache_append_rope(R(t), R(t), 1, 1, 0x20000, 1, None, 0, None, None, R(c), None) == S.SAGE_ERR_ARG


def test_tree_tables_refuses(lib):
    def call(parents=0x1000, ps=8, B=2, N=8, mask=0x2000, mb=8, mn=1, depth=0x3000, ds=8):
        return lib.sage_tree_tables(parents, ps, B, N, None, mask, mb, mn, depth, ds, None)

    for bad in (dict(parents=None), dict(mask=None), dict(B=0), dict(N=0), dict(ps=-1), dict(mn=0), dict(mb=0), dict(ds=7),
                dict(N=33, mn=1, mb=66, ds=33)):
        assert call(**bad) == S.SAGE_ERR_ARG, bad
    assert call(N=4097, ps=4097, mb=4097 * 129, mn=129, ds=4097) == S.SAGE_ERR_UNSUPPORTED


def test_cache_keep_refuses(lib):
    def call(kept=0x1000, ks=4, B=2, K=4, slots=0x2000, ss=8, N=8, c=None):
        return lib.sage_cache_keep(kept, ks, B, K, slots, ss, N, R(c or cache()), None)

    for bad in (dict(kept=None), dict(slots=None), dict(B=0), dict(K=0), dict(N=3), dict(ks=-1), dict(ss=-1),
                dict(c=cache(pages=0))):
        assert call(**bad) == S.SAGE_ERR_ARG, bad
    assert call(c=cache(page=20)) == S.SAGE_ERR_UNSUPPORTED
    assert lib.sage_cache_keep(0x1000, 4, 1, 1, 0x2000, 8, 8, None, None) == S.SAGE_ERR_ARG


def test_attn_paged_tree_refuses(lib):
    def call(q=None, mask=0x30000, mb=1, mn=1, B=2, H=8, Nq=1, table=0x20000, width=8, ws=0x40000, ws_bytes=1 << 40, c=None):
        q, o, c = q or tensor(), tensor(), c or cache()
        return lib.sage_attn_paged_tree(R(q), R(o), R(c), B, H, Nq, None, table, 8, width, None, None, 0, None, mask, mb, mn,
                                        0.0, ws, ws_bytes, None)

    for bad in (dict(mask=None), dict(mb=-1), dict(mn=-1), dict(q=tensor(ptr=0)), dict(B=0), dict(Nq=0), dict(H=12),
                dict(table=None), dict(width=-1), dict(ws=None), dict(ws=0x40004), dict(ws_bytes=64)):
        assert call(**bad) == S.SAGE_ERR_ARG, bad
    for bad in (dict(q=tensor(ptr=0x10008)), dict(q=tensor(sh=0)), dict(width=1 << 28), dict(c=cache(page=8))):
        assert call(**bad) == S.SAGE_ERR_UNSUPPORTED, bad


def test_turns_hold_the_frequencies_to_the_last_bit(lib):
    """turns = f / (2 pi) modulo 1 in units of 2^-64, off by half a unit and what the double-double leaves (2^-20 units)."""
    f = S.rotary_frequencies(128, 500000.0)[0] + [0.0, 1.0, -0.25, 3.0, 6.283185307179586, 1e-12, 1e5, -77.7, 2.0 ** -60]
    turns = S.make_rotary(f, device="cpu").turns.tolist()
    for x, t in zip(f, turns):
        want = Fraction(x) / TWO_PI * 2 ** 64
        off = (t - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 2 ** 20), x


def test_turns_refuse(lib):
    out = (ctypes.c_uint64 * 2)()
    for bad in (math.nan, math.inf, -math.inf, 2.0 ** 20, -2.0 ** 21):
        assert lib.sage_rotary_turns((ctypes.c_double * 2)(1.0, bad), 2, out) == S.SAGE_ERR_ARG
    assert lib.sage_rotary_turns(None, 1, out) == S.SAGE_ERR_ARG
    assert lib.sage_rotary_turns((ctypes.c_double * 1)(1.0), 0, out) == S.SAGE_ERR_ARG
    assert lib.sage_rotary_turns((ctypes.c_double * 1)(1.0), 1, None) == S.SAGE_ERR_ARG
    with pytest.raises(S.SageError):
        S.make_rotary([], device="cpu")


def test_frequencies():
    plain, a = S.rotary_frequencies(64)
    assert a == 1.0 and plain[0] == 1.0 and len(plain) == 32 and plain[31] == pytest.approx(10000.0 ** (-62 / 64), rel=1e-15)
    f, a = S.rotary_frequencies(64, scale=4.0)
    assert a == 1.0 and f == [x / 4 for x in plain]
    f, a = S.rotary_frequencies(64, scale=4.0, method="base")       # the fastest stays, the slowest is divided by the scale
    assert a == 1.0 and f[0] == 1.0 and f[31] == pytest.approx(plain[31] / 4, rel=1e-12)
    assert all(x > y for x, y in zip(f, f[1:]))
    f, a = S.rotary_frequencies(64, scale=16.0, method="parts", trained=2048)
    assert a == pytest.approx(0.1 * math.log(16) + 1)
    for x, y in zip(plain, f):
        turns = 2048 * x / (2 * math.pi)
        want = x if turns >= 32 else x / 16 if turns <= 1 else x / 16 + (x - x / 16) * (turns - 1) / 31
        assert y == pytest.approx(want, rel=1e-13)
    assert any(1 < 2048 * x / (2 * math.pi) < 32 for x in plain)
    for method in ("linear", "base", "parts"):
        assert S.rotary_frequencies(64, method=method) == (plain, 1.0)
    for bad in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=8, base=0.0), dict(rotary_dim=8, scale=0.5),
                dict(rotary_dim=8, scale=2.0, method="other"), dict(rotary_dim=8, method="other"), dict(rotary_dim=2, scale=2.0, method="base"),
                dict(rotary_dim=8, scale=2.0, method="parts", slow=3.0, fast=3.0)):
        with pytest.raises(ValueError):
            S.rotary_frequencies(**bad)


def test_python_checks_name_the_argument():
    with pytest.raises(ValueError, match="turns"):
        S.Rotary(torch.zeros(4))
    with pytest.raises(ValueError, match="turns"):
        S.Rotary(torch.zeros(8, dtype=torch.int64)[::2])
    c = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    cache_ = S.PageCache(c, c.clone())
    r = S.make_rotary(S.rotary_frequencies(64)[0], device="cpu")
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 3), dtype=torch.int32)
    with pytest.raises(ValueError):                        # tensors of the CPU
        S.sage_rope(x, x, r)
    with pytest.raises(ValueError):
        S.sage_cache_append_rope(x, x, i, cache_, r)
    with pytest.raises(ValueError):
        S.sage_tree_tables(i, torch.zeros((1, 3, 1), dtype=torch.int32))
    with pytest.raises(ValueError):
        S.sage_cache_keep(i, i, cache_)
    with pytest.raises(ValueError):
        S.sage_attn_paged_tree(x, x.clone(), cache_, None, torch.zeros((3, 1), dtype=torch.int32), torch.zeros(16))
    with pytest.raises(ValueError, match="one shape"):
        S.sage_rope(x, x[:, :1], r)
    with pytest.raises(ValueError, match="bfloat16"):
        S.sage_rope(x.float(), x, r)


@pytest.mark.parametrize("name", ["sage_rotary.cu", "sage_tree.cu", "sage_paged_tiles_tree.cu", "sage_paged_tiles_half.cu"])
def test_no_load_may_pass_the_wait(name):
    with open(os.path.join(B.CSRC, name)) as f:
        assert unordered_loads(f.read()) == []


@pytest.mark.parametrize("name", ["sage_rotary.cu", "sage_tree.cu"])
def test_the_device_says_how_many_sms_it_has(name):
    """Rules of the host that go by the size of the GPU ask for it."""
    with open(os.path.join(B.CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"\b15[02]\b", code)
    assert "sm_count()" in code


def test_no_form_is_built_that_no_call_reaches(lib):
    """paged_tiles_kernel<channels, groups, form, tree, two lanes a row> (forms: 0 the list, 1 with the prefix's items, 2 an
    item to a CTA, 3 to a cluster), as the library's symbols name them."""
    names = subprocess.run(["nm", "-C", B.LIB], capture_output=True, text=True, check=True).stdout
    built = set(re.findall(r" t void sage::\(anonymous namespace\)::paged_tiles_kernel<(\d+), (\d), (\d), (\w+), (\w+)>\(", names))
    want = set()
    for D in ("64", "128"):
        for tree in ("false", "true"):
            want |= {(D, g, form, tree, "false") for g in "12" for form in "02"}
            want.add((D, "1", "1", tree, "false"))
        want.add((D, "2", "1", "false", "false"))          # the prefix's own list, which needs no mask
        want |= {(D, "1", "3", "true", "false"), (D, "1", "3", "true", "true")}
    want.add(("64", "1", "0", "true", "true"))
    assert built == want


@pytest.mark.parametrize("name,form", [("sage_paged_tiles_tree.cu", "1"), ("sage_paged_tiles_half.cu", "2")])
def test_units_of_the_other_forms_hold_nothing_else(name, form):
    """So the checks of sage_paged_tiles.cu's text cover what they compile."""
    with open(os.path.join(B.CSRC, name)) as f:
        code = [x for x in (re.sub(r"//.*", "", line).strip() for line in f) if x]
    assert code == [f"#define SAGE_PAGED_TILES_TREE {form}", '#include "sage_paged_tiles.cu"']


def test_angles_of_far_positions(lib):
    """The upper 32 bits of pos * turns: off by less than |pos| * 2^-64 + 2^-32 turns, which is 2^-31 at most for positions
    of 32 bits and for the sum of two."""
    f = S.rotary_frequencies(128, 500000.0)[0] + [3.0, -0.25, 1e-12, 77777.7]
    for pos in (1, -1, 12345, 10 ** 6, 2 ** 31 - 1, -2 ** 31, 2 ** 32 - 2, -2 ** 32):
        for x, t in zip(f, S.make_rotary(f, device="cpu").turns.tolist()):
            phase = (pos * t) % 2 ** 64 >> 32
            off = (Fraction(phase, 2 ** 32) - pos * Fraction(x) / TWO_PI) % 1
            off = min(off, 1 - off)
            assert off < abs(pos) * Fraction(1, 2 ** 64) + Fraction(1, 2 ** 32) <= Fraction(1, 2 ** 31), (x, pos)
