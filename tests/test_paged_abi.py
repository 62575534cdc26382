"""The paged-cache entry points: exported as declared, and refusing bad arguments on the host."""
import ctypes
import subprocess

import pytest
import torch

from differential_attention_attn_gb300 import build as libbuild
from differential_attention_attn_gb300 import ops

FAKE = 0x10000  # never dereferenced: validation rejects or returns before any launch


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return ops.load()


def test_exports_what_the_header_declares(lib):
    import re
    text = open(ops.PAGED_HEADER_PATH).read()
    names = set(re.findall(r"\b(diffpaged_[a-z0-9_]+)\s*\(", text))
    assert names == {"diffpaged_append", "diffpaged_fwd", "diffpaged_fwd_plan", "diffpaged_evict",
                     "diffpaged_evict_plan"}
    out = subprocess.run(["nm", "-D", "--defined-only", libbuild.build()], capture_output=True,
                         text=True, check=True).stdout
    assert {x.split()[-1] for x in out.splitlines()
            if x.split()[-1].startswith("diffpaged_")} == names


def test_struct_layout_and_status(lib):
    assert ctypes.sizeof(ops.PagedCacheStruct) == 6 * 8 + 9 * 8 + 3 * 8 + 8
    assert ops.strerror(ops.ERR_PAGE) == "page number or sequence length outside the paged cache"


def _cache(heads=2, d=64, page=16, pages=8, max_pages=4, k=2, **kw):
    st = lambda w: ops.Strides(heads * page * w, page * w, w)
    c = ops.PagedCacheStruct(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, st(d), st(d), st(2 * d), pages,
                             heads, max_pages, page, 0)
    for name, x in kw.items():
        setattr(c, name, x)
    return c


def _desc(B=1, H=2, N=1, d=64, dtype=None, headnorm=1, eps=1e-5):
    return ops.make_desc(B, H, N, d, ops.BF16 if dtype is None else dtype, True, headnorm, eps, 0.0)


def _append(lib, desc, cache, ptrs=(FAKE,) * 3, strides=None):
    return lib.diffpaged_append(ctypes.byref(desc) if desc else None,
                                ctypes.byref(cache) if cache else None, *ptrs, strides, None)


def _fwd(lib, desc, cache, ptrs=(FAKE,) * 5, strides=None, acc=0, ws=FAKE, nbytes=1 << 40):
    return lib.diffpaged_fwd(ctypes.byref(desc) if desc else None,
                             ctypes.byref(cache) if cache else None, *ptrs, strides, acc, ws,
                             nbytes, None)


def _evict(lib, desc, cache, keep=8, recent=0, ws=FAKE, nbytes=1 << 40):
    return lib.diffpaged_evict(ctypes.byref(desc) if desc else None,
                               ctypes.byref(cache) if cache else None, keep, recent, ws, nbytes,
                               None)


ALL = [_append, _fwd, _evict]


@pytest.mark.parametrize("call", ALL)
def test_null_structs(lib, call):
    assert call(lib, None, _cache()) == ops.ERR_INVALID_ARG
    assert call(lib, _desc(), None) == ops.ERR_INVALID_ARG


@pytest.mark.parametrize("call", ALL)
@pytest.mark.parametrize("field,value", [
    ("k1", 0), ("k2", 0), ("v", 0), ("page_table", 0), ("kv_len", 0), ("k1", FAKE + 8),
    ("k2", FAKE + 2), ("v", FAKE + 8), ("page_table", FAKE + 2), ("kv_len", FAKE + 1),
    ("weights", FAKE + 2), ("num_pages", 0), ("num_pages", -1), ("kv_heads", 0), ("kv_heads", 3),
    ("max_pages", 0), ("page_size", 0), ("page_size", -16), ("reserved", 1),
    ("k1_strides", ops.Strides(2048, 1024, 60)), ("k2_strides", ops.Strides(2048, 0, 64)),
    ("v_strides", ops.Strides(-4096, 2048, 128)), ("v_strides", ops.Strides(1 << 39, 2048, 128))])
def test_invalid_cache(lib, call, field, value):
    assert call(lib, _desc(), _cache(**{field: value})) == ops.ERR_INVALID_ARG


@pytest.mark.parametrize("call", ALL)
def test_unsupported(lib, call):
    U = ops.ERR_UNSUPPORTED
    assert call(lib, _desc(dtype=ops.F32), _cache()) == U
    assert call(lib, _desc(d=32), _cache()) == U
    assert call(lib, _desc(), _cache(page_size=24)) == U
    assert call(lib, _desc(), _cache(page_size=8)) == U
    assert call(lib, _desc(), _cache(max_pages=1 << 26)) == U
    assert call(lib, _desc(), _cache(num_pages=1 << 31)) == U


def test_e4m3_strides_are_multiples_of_sixteen(lib):
    d = _desc(dtype=ops.E4M3_QK)
    bad = _cache(k1_strides=ops.Strides(2048, 1024, 72))
    for call in ALL:
        assert call(lib, d, bad) == ops.ERR_INVALID_ARG


def test_negative_sizes(lib):
    for call in ALL:
        assert call(lib, _desc(B=-1), _cache()) == ops.ERR_INVALID_ARG
        assert call(lib, _desc(N=-1), _cache()) == ops.ERR_INVALID_ARG
        assert call(lib, _desc(d=0), _cache()) == ops.ERR_INVALID_ARG
        assert call(lib, _desc(eps=-1.0), _cache()) == ops.ERR_INVALID_ARG


def test_heads(lib):
    assert _append(lib, _desc(H=4), _cache()) == ops.ERR_INVALID_ARG  # H = kv_heads
    assert _evict(lib, _desc(H=4), _cache()) == ops.ERR_INVALID_ARG
    assert _fwd(lib, _desc(H=3), _cache()) == ops.ERR_INVALID_ARG     # a multiple of kv_heads
    assert _fwd(lib, _desc(H=2 * 65), _cache()) == ops.ERR_UNSUPPORTED
    assert _fwd(lib, _desc(N=17), _cache()) == ops.ERR_UNSUPPORTED


def test_append_pointers(lib):
    for k in range(3):
        for x in (0, FAKE + 8):
            ptrs = [FAKE] * 3
            ptrs[k] = x
            assert _append(lib, _desc(), _cache(), ptrs) == ops.ERR_INVALID_ARG
    bad = (ops.Strides * 3)(ops.Strides(64, 64, 64), ops.Strides(64, 64, 63), ops.Strides(8, 8, 8))
    assert _append(lib, _desc(), _cache(), strides=bad) == ops.ERR_INVALID_ARG


def test_evict_arguments(lib):
    assert _evict(lib, _desc(), _cache(weights=0)) == ops.ERR_INVALID_ARG
    assert _evict(lib, _desc(), _cache(), keep=-1) == ops.ERR_INVALID_ARG
    assert _evict(lib, _desc(), _cache(), keep=8, recent=9) == ops.ERR_INVALID_ARG
    assert _evict(lib, _desc(), _cache(), keep=8, recent=-1) == ops.ERR_INVALID_ARG
    assert _evict(lib, _desc(), _cache(), ws=0) == ops.ERR_INVALID_ARG
    assert _evict(lib, _desc(), _cache(), ws=FAKE + 16) == ops.ERR_INVALID_ARG
    assert _evict(lib, _desc(), _cache(), nbytes=16) == ops.ERR_INVALID_ARG


def test_evict_plan(lib):
    n = ctypes.c_size_t(1)
    plan = lambda keep: lib.diffpaged_evict_plan(ctypes.byref(_desc()), ctypes.byref(_cache()),
                                                 keep, ctypes.byref(n))
    assert plan(8) == ops.OK and n.value > 0
    assert plan(64) == ops.OK and n.value == 0  # no sequence can be longer than 4 pages of 16
    assert plan(-1) == ops.ERR_INVALID_ARG


def test_sizes_that_do_not_fit(lib):
    """Workspaces past 64 bits and grids past 31 are refused, not wrapped."""
    n = ctypes.c_size_t(0)
    st = ops.Strides(1 << 38, 1 << 20, 128)  # (those of a contiguous pool would be past the limit)
    big = _cache(heads=1 << 14, page=1 << 29, max_pages=1, k1_strides=st, k2_strides=st,
                 v_strides=st)
    for B in (1 << 20, 1 << 16):
        desc = _desc(B=B, H=1 << 14)
        assert lib.diffpaged_evict_plan(ctypes.byref(desc), ctypes.byref(big), 1 << 28,
                                        ctypes.byref(n)) == ops.ERR_UNSUPPORTED
        assert _evict(lib, desc, big, keep=1 << 28) == ops.ERR_UNSUPPORTED


def test_nothing_to_do(lib):
    assert _append(lib, _desc(N=0), _cache()) == ops.OK
    assert _append(lib, _desc(B=0), _cache()) == ops.OK
    assert _fwd(lib, _desc(N=0), _cache()) == ops.OK
    assert _fwd(lib, _desc(B=0), _cache()) == ops.OK
    assert _evict(lib, _desc(B=0), _cache()) == ops.OK


def test_accumulate_needs_weights(lib):
    assert _fwd(lib, _desc(), _cache(weights=0), acc=1) == ops.ERR_INVALID_ARG


def test_python_checks():
    with pytest.raises(ValueError, match="k1 must be"):
        ops.PagedCache(torch.zeros(2, 2, 16), None, None, None, None)
    pool = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    v = torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="unsupported key dtype"):
        ops.PagedCache(pool.float(), pool, v, table, lens)
    with pytest.raises(ValueError, match="v must be"):
        ops.PagedCache(pool, pool, pool, table, lens)
    with pytest.raises(ValueError, match="page_table must be"):
        ops.PagedCache(pool, pool, v, table.long(), lens)
    with pytest.raises(ValueError, match="kv_len must be"):
        ops.PagedCache(pool, pool, v, table, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        ops.PagedCache(pool, pool, v, table, lens)


def test_lengths_are_not_read_through_the_read_only_path():
    """kv_len is written by diffpaged_evict while the kernels behind it may be resident already
    (dependent launch): ld.global.nc, which __ldg is, must not read it."""
    import glob
    import os
    files = glob.glob(os.path.join(libbuild.CSRC, "paged*"))
    assert len(files) >= 6
    uses = 0
    for path in files:
        text = open(path).read()
        uses += text.count("kv_len[")
        for part in text.split("__ldg(")[1:]:
            assert "kv_len" not in part[:part.index(")")], path
            assert "uint4" not in part[:part.index(")")], path  # rows: another kernel's output
    assert uses > 0
