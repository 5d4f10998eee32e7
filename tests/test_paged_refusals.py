"""Calls of the page-cache entries that are refused on the host, before any
CUDA call, and the size of the workspace."""
import ctypes

import pytest
import torch

import quantized_exact_attention_gb300 as S
from quantized_exact_attention_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return S.load_library()


def tensor(ptr=0x10000, sb=128 * 128, sh=128, sn=128 * 8):
    return S.sage_tensor(ptr, sb, sh, sn)


def cache(k=None, v=None, pages=64, page=16, heads=8, D=128):
    return S.sage_page_cache(k or tensor(), v or tensor(0x900000), pages, page, heads, D)


def attn(lib, q=None, o=None, c=None, B=2, H=8, Nq=1, table=0x20000, stride=8, width=8, ptable=None, pwidth=0,
         ws=0x40000, ws_bytes=None, D=128, Hkv=8):
    q, o, c = q or tensor(), o or tensor(), c or cache()
    if ws_bytes is None:
        n = ctypes.c_size_t()
        ws_bytes = n.value if lib.sage_paged_workspace(B, H, Hkv, Nq, D, ctypes.byref(n)) else n.value
    return lib.sage_attn_paged(ctypes.byref(q), ctypes.byref(o), ctypes.byref(c), B, H, Nq, None, table, stride, width,
                               None, ptable, pwidth, None, 0.0, 1, ws, ws_bytes, None)


def test_attn_paged_refuses(lib):
    assert attn(lib, q=tensor(ptr=0)) == S.SAGE_ERR_ARG
    assert attn(lib, o=tensor(ptr=0x10008)) == S.SAGE_ERR_UNSUPPORTED
    assert attn(lib, q=tensor(sn=100)) == S.SAGE_ERR_UNSUPPORTED
    assert attn(lib, q=tensor(sb=-128)) == S.SAGE_ERR_UNSUPPORTED
    assert attn(lib, B=0) == S.SAGE_ERR_ARG
    assert attn(lib, Nq=0) == S.SAGE_ERR_ARG
    assert attn(lib, H=12) == S.SAGE_ERR_ARG                       # not a multiple of the cache's heads
    assert attn(lib, table=None) == S.SAGE_ERR_ARG
    assert attn(lib, width=-1) == S.SAGE_ERR_ARG
    assert attn(lib, stride=-1) == S.SAGE_ERR_ARG
    assert attn(lib, pwidth=3) == S.SAGE_ERR_ARG                   # a prefix without its table
    assert attn(lib, ws=None) == S.SAGE_ERR_ARG
    assert attn(lib, ws=0x40004) == S.SAGE_ERR_ARG
    assert attn(lib, ws_bytes=64) == S.SAGE_ERR_ARG
    assert attn(lib, width=1 << 28) == S.SAGE_ERR_UNSUPPORTED      # token numbers would pass 2^31
    n = ctypes.c_size_t()
    assert lib.sage_attn_paged(None, None, None, 1, 1, 1, None, None, 0, 0, None, None, 0, None, 0.0, 1, None, 0,
                               None) == S.SAGE_ERR_ARG
    assert lib.sage_paged_workspace(1, 1, 1, 1, 128, None) == S.SAGE_ERR_ARG
    assert lib.sage_paged_workspace(1, 3, 2, 1, 128, ctypes.byref(n)) == S.SAGE_ERR_ARG
    assert lib.sage_paged_workspace(1, 2, 2, 1, 96, ctypes.byref(n)) == S.SAGE_ERR_UNSUPPORTED
    assert lib.sage_paged_workspace(1, 1024, 1024, 1 << 21, 64, ctypes.byref(n)) == S.SAGE_ERR_UNSUPPORTED
    assert attn(lib, q=tensor(sh=0)) == S.SAGE_ERR_UNSUPPORTED     # a broadcast axis
    assert attn(lib, o=tensor(sb=64)) == S.SAGE_ERR_UNSUPPORTED
    assert attn(lib, c=cache(k=tensor(sn=0))) == S.SAGE_ERR_UNSUPPORTED
    assert attn(lib, c=cache(v=tensor(sb=1 << 40))) == S.SAGE_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad,code", [(dict(pages=0), S.SAGE_ERR_ARG), (dict(heads=0), S.SAGE_ERR_ARG),
                                      (dict(page=24), S.SAGE_ERR_UNSUPPORTED), (dict(page=8), S.SAGE_ERR_UNSUPPORTED),
                                      (dict(page=256), S.SAGE_ERR_UNSUPPORTED), (dict(D=96), S.SAGE_ERR_UNSUPPORTED),
                                      (dict(pages=1 << 28), S.SAGE_ERR_UNSUPPORTED),
                                      (dict(k=S.sage_tensor(0x10004, 128, 128, 128)), S.SAGE_ERR_UNSUPPORTED),
                                      (dict(v=S.sage_tensor(0x10000, 128, 100, 128)), S.SAGE_ERR_UNSUPPORTED)])
def test_a_bad_cache_is_refused(lib, bad, code):
    c, t = cache(**bad), tensor()
    assert attn(lib, c=c, ws_bytes=1 << 40) == code
    assert lib.sage_cache_append(ctypes.byref(t), ctypes.byref(t), 1, 1, 0x20000, 1, ctypes.byref(c), None) == code


def test_cache_append_refuses(lib):
    c, t = cache(), tensor()
    R = ctypes.byref
    assert lib.sage_cache_append(R(t), R(t), 0, 1, 0x20000, 1, R(c), None) == S.SAGE_ERR_ARG
    assert lib.sage_cache_append(R(t), R(t), 1, 0, 0x20000, 1, R(c), None) == S.SAGE_ERR_ARG
    assert lib.sage_cache_append(R(t), R(t), 1, 1, None, 1, R(c), None) == S.SAGE_ERR_ARG
    assert lib.sage_cache_append(None, R(t), 1, 1, 0x20000, 1, R(c), None) == S.SAGE_ERR_ARG
    assert lib.sage_cache_append(R(t), R(tensor(ptr=0x10002)), 1, 1, 0x20000, 1, R(c), None) == S.SAGE_ERR_UNSUPPORTED
    assert lib.sage_cache_append(R(t), R(t), 1, 1, 0x20000, 1, None, None) == S.SAGE_ERR_ARG
    assert lib.sage_cache_append(R(t), R(t), 1 << 16, 1 << 15, 0x20000, 1, R(c), None) == S.SAGE_ERR_UNSUPPORTED


def test_page_tables_refuses(lib):
    def call(old=None, new=0x1000, B=2, page=16, free=0x2000, n_free=4, table=0x3000, stride=8, W=8, slots=0x4000,
             sstride=4, N=4, taken=0x5000):
        return lib.sage_page_tables(old, new, B, page, free, n_free, table, stride, W, slots, sstride, N, taken, None)

    for bad in (dict(new=None), dict(B=0), dict(table=None), dict(W=0), dict(taken=None), dict(free=None),
                dict(n_free=-1), dict(slots=None), dict(N=-1), dict(stride=7), dict(sstride=3)):
        assert call(**bad) == S.SAGE_ERR_ARG, bad
    assert call(page=20) == S.SAGE_ERR_UNSUPPORTED
    assert call(W=1 << 28, stride=1 << 28) == S.SAGE_ERR_UNSUPPORTED


def test_workspace_covers_both_forms_and_grows_with_the_batch(lib):
    a = S.paged_workspace_bytes(4, 8, 8, 1)
    assert 0 < a < S.paged_workspace_bytes(512, 8, 8, 1)
    assert S.paged_workspace_bytes(4, 8, 8, 1, D=64) < a
    assert a % 16 == 0


def test_python_checks_name_the_argument():
    c = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        S.PageCache(c, c[:2])
    with pytest.raises(ValueError):
        S.PageCache(c.float(), c.float())
    with pytest.raises(ValueError):
        S.alloc_page_cache(4, 24, 2, device="cpu")
    cache_ = S.PageCache(c, c.clone())
    assert (cache_.num_pages, cache_.heads, cache_.page_size) == (4, 2, 16)
    q = torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):                        # tensors of the CPU
        S.sage_attn_paged(q, q.clone(), cache_, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(16))
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="page_size"):     # not taken modulo 2^32
        S.sage_page_tables(n, (1 << 32) + 16, n, torch.zeros((1, 1), dtype=torch.int32), taken=n)
    with pytest.raises(ValueError):                        # another head dimension than the cache's
        S.sage_attn_paged(q[..., :32], q[..., :32], cache_, None, torch.zeros(16))
    with pytest.raises(ValueError):                        # heads other than the cache's
        S.sage_cache_append(q[:, :1], q[:, :1], torch.zeros((1, 1), dtype=torch.int32), cache_)


def test_widths_whose_tiles_pass_int_are_refused(lib):
    """The bound counts tiles by the table widths, for few rows (16 keys) and for many (128)."""
    c = cache(heads=32)
    assert attn(lib, B=512, H=32, Hkv=32, c=c, width=65536, stride=65536) == S.SAGE_ERR_UNSUPPORTED
    # the same with half of the width in a shared prefix that is read with each request's keys
    assert attn(lib, B=1, H=65535, Hkv=65535, c=cache(heads=65535), width=65536, ptable=0x30000,
                pwidth=200000) == S.SAGE_ERR_UNSUPPORTED
    assert attn(lib, B=512, H=32, Hkv=32, Nq=4096, c=c, width=65536, q=tensor(sb=1 << 30, sn=4096),
                o=tensor(sb=1 << 30, sn=4096)) == S.SAGE_ERR_UNSUPPORTED
