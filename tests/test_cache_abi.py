"""Host-side argument checks of the 4-bit cache and page entry points: the documented codes come
back before anything reaches the GPU (so these run without a device)."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

import attn_fwd_05_b200 as ab
from attn_fwd_05_b200 import binding, build
from oracle import kv4

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "attn_b200.h")
OK, INVALID, UNSUPPORTED, ALIGN, CUDA, TIMEOUT, BAD_PAGE, WORKSPACE, TOO_LARGE = range(9)
FAKE, FAKE2 = 0x10000, 0x4000000  # aligned, never dereferenced: every call below ends in its checks

NAMES = ["attn_kv4_page_bytes", "attn_kv4_append", "attn_kv4_gather", "attn_decode_paged_kv4",
         "attn_decode_paged_kv4_workspace_size", "attn_pages_workspace_size", "attn_pages_fork", "attn_pages_compact"]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def test_entry_points_are_declared_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"\b(attn_[a-z_0-9]+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", binding.library_path()], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(NAMES) <= declared
    assert declared == set(binding.SIGNATURES) and declared <= exported
    for name in NAMES:
        assert callable(getattr(ab, name))


@pytest.mark.parametrize("Hkv,ps,d", [(1, 16, 64), (8, 16, 128), (3, 64, 256), (2, 32, 64)])
def test_page_bytes(lib, Hkv, ps, d):
    assert lib.attn_kv4_page_bytes(Hkv, ps, d) == kv4.page_bytes(Hkv, ps, d) == Hkv * ps * d * 9 // 8


def test_page_bytes_of_unsupported_sizes(lib):
    assert lib.attn_kv4_page_bytes(8, 24, 128) == lib.attn_kv4_page_bytes(8, 16, 96) == lib.attn_kv4_page_bytes(0, 16, 64) == 0


def append(lib, k=FAKE, v=FAKE, ks=1024, vs=1024, pool=FAKE, bt=FAKE, sl=FAKE, cu=FAKE, ps=16, ko=None, vo=None, S=4,
           T=10, Hkv=8, d=128, npages=10, maxp=8):
    return lib.attn_kv4_append(k, v, ks, vs, pool, bt, sl, cu, ps, ko, vo, S, T, Hkv, d, npages, maxp, None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), INVALID), (dict(T=-1), INVALID), (dict(S=0), INVALID), (dict(Hkv=0), INVALID), (dict(maxp=0), INVALID),
    (dict(npages=-1), INVALID), (dict(ps=48), UNSUPPORTED), (dict(ps=8), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cu=None), INVALID), (dict(pool=None), INVALID),
    (dict(bt=None), INVALID), (dict(sl=None), INVALID), (dict(ks=1016), INVALID), (dict(vs=8), INVALID),
    (dict(ks=1028), ALIGN), (dict(k=FAKE + 8), ALIGN), (dict(v=FAKE + 2), ALIGN), (dict(pool=FAKE + 8), ALIGN),
    (dict(ko=FAKE + 8), ALIGN), (dict(vo=FAKE + 4), ALIGN), (dict(bt=FAKE + 2), ALIGN), (dict(cu=FAKE + 1), ALIGN),
    (dict(maxp=1 << 28), INVALID), (dict(maxp=(1 << 26) + 1), INVALID), (dict(npages=1 << 28), INVALID),
    # outputs over inputs, other than a dense tensor over itself, or over one another
    (dict(v=FAKE2, ko=FAKE + 16), INVALID), (dict(v=FAKE2, ks=1032, ko=FAKE), INVALID), (dict(v=FAKE2, ko=FAKE2), INVALID),
    (dict(v=FAKE2, vo=FAKE2 - 16), INVALID), (dict(v=FAKE2, vo=FAKE), INVALID), (dict(v=FAKE2, vs=2048, vo=FAKE2), INVALID),
    (dict(k=FAKE, v=FAKE2, ko=FAKE2 + 65536, vo=FAKE2 + 65536 + 1024), INVALID),
])
def test_append_rejects_bad_arguments(lib, kw, code):
    assert append(lib, **kw) == code


def test_append_of_nothing_is_a_noop(lib):
    assert append(lib, T=0, k=None, v=None) == OK
    assert append(lib, S=0, T=0, bt=None, sl=None, pool=None) == OK


def gather(lib, pool=FAKE, bt=FAKE, sl=FAKE, ps=16, k=FAKE, v=FAKE, S=4, Hkv=8, N=100, d=128, npages=10, maxp=8):
    return lib.attn_kv4_gather(pool, bt, sl, ps, k, v, S, Hkv, N, d, npages, maxp, None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), INVALID), (dict(N=-1), INVALID), (dict(Hkv=0), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k=FAKE + 8), ALIGN), (dict(v=FAKE + 8), ALIGN), (dict(pool=FAKE + 4), ALIGN), (dict(d=80), UNSUPPORTED),
    (dict(ps=128), UNSUPPORTED), (dict(pool=None), INVALID), (dict(sl=None), INVALID),
    (dict(N=(1 << 30) + 1), INVALID), (dict(maxp=(1 << 26) + 1), INVALID),
])
def test_gather_rejects_bad_arguments(lib, kw, code):
    assert gather(lib, **kw) == code


def test_gather_of_nothing_is_a_noop(lib):
    assert gather(lib, S=0, k=None, v=None) == OK and gather(lib, N=0, k=None, v=None) == OK


def dec(lib, q=FAKE, pool=FAKE, bt=FAKE, sl=FAKE, ps=16, o=FAKE, lse=None, S=4, Hq=8, Hkv=2, d=128, npages=10, maxp=8,
        scale=0.1, ws=FAKE, wsb=1 << 30):
    return lib.attn_decode_paged_kv4(q, pool, bt, sl, ps, o, lse, S, Hq, Hkv, d, npages, maxp, ctypes.c_float(scale),
                                     ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), INVALID), (dict(Hq=6, Hkv=4), INVALID), (dict(Hq=0), INVALID), (dict(maxp=0), INVALID),
    (dict(npages=-1), INVALID), (dict(ps=8), UNSUPPORTED), (dict(d=80), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID),
    (dict(o=None), INVALID), (dict(bt=None), INVALID), (dict(sl=None), INVALID), (dict(pool=None), INVALID),
    (dict(q=FAKE + 8), ALIGN), (dict(o=FAKE + 4), ALIGN), (dict(pool=FAKE + 8), ALIGN), (dict(lse=FAKE + 2), ALIGN),
    (dict(ws=FAKE + 16), ALIGN), (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE),
    (dict(maxp=(1 << 26) + 1), INVALID), (dict(S=100000, maxp=1 << 20), INVALID), (dict(S=1 << 14, maxp=1 << 18), INVALID),  # 2^31 units of 32 tokens
])
def test_decode_rejects_bad_arguments(lib, kw, code):
    assert dec(lib, **kw) == code


def test_decode_of_no_sequence_is_a_noop(lib):
    assert dec(lib, S=0, q=None, o=None) == OK


def test_decode_workspace_size(lib):
    f = lib.attn_decode_paged_kv4_workspace_size
    assert f(64, 64, 8, 96) == 0 and f(64, 60, 8, 128) == 0 and f(-1, 64, 8, 128) == 0
    assert 0 < f(1, 64, 8, 128) <= f(64, 64, 8, 128) < 64 << 20  # bounded by the GPU's size, not by lengths


def fork(lib, bt=FAKE, sl=FAKE, parents=FAKE + 4096, add=None, nt=FAKE2, nl=FAKE2 + 65536, ps=16, pools=(FAKE,), n=None,
         pb=4096, S=4, cols=8, rows=6, ncols=8, npages=100, nfree=None, ws=FAKE, wsb=1 << 30):
    arr = None if pools is None else (ctypes.c_void_p * max(1, len(pools)))(*pools)
    return lib.attn_pages_fork(bt, sl, parents, add, nt, nl, ps, arr, len(pools or ()) if n is None else n, pb, S, cols,
                               rows, ncols, npages, nfree, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(ncols=7), INVALID),
    (dict(npages=-1), INVALID), (dict(ps=0), INVALID), (dict(ncols=1 << 28), INVALID), (dict(ps=(1 << 27) + 1), INVALID),
    (dict(rows=1 << 20, ncols=1 << 12), INVALID), (dict(pb=4088), INVALID),
    (dict(pools=None, n=1), INVALID), (dict(n=-1), INVALID), (dict(n=129), TOO_LARGE), (dict(pools=(FAKE, None)), INVALID),
    (dict(pools=(FAKE + 8,)), ALIGN), (dict(bt=None), INVALID), (dict(sl=None), INVALID), (dict(parents=None), INVALID),
    (dict(nt=None), INVALID), (dict(nl=None), INVALID), (dict(bt=FAKE + 2), ALIGN), (dict(nfree=FAKE + 2), ALIGN),
    (dict(nt=FAKE), INVALID), (dict(nt=FAKE + 64), INVALID), (dict(nl=FAKE + 8), INVALID), (dict(nl=FAKE + 4096), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE), (dict(ws=FAKE + 16), ALIGN),
])
def test_fork_rejects_bad_arguments(lib, kw, code):
    assert fork(lib, **kw) == code


def compact(lib, bt=FAKE, sl=FAKE, nt=FAKE2, pm=FAKE2 + 65536, ps=16, pools=(FAKE,), n=None, pb=4096, S=4, cols=8,
            npages=100, nlive=None, ws=FAKE, wsb=1 << 30):
    arr = None if pools is None else (ctypes.c_void_p * max(1, len(pools)))(*pools)
    return lib.attn_pages_compact(bt, sl, nt, pm, ps, arr, len(pools or ()) if n is None else n, pb, S, cols, npages,
                                  nlive, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), INVALID), (dict(cols=0), INVALID), (dict(npages=-1), INVALID), (dict(ps=-16), INVALID),
    (dict(pb=8), INVALID), (dict(n=129), TOO_LARGE), (dict(pools=(None,)), INVALID), (dict(pools=(FAKE + 4,)), ALIGN),
    (dict(ps=(1 << 27) + 1), INVALID), (dict(bt=None), INVALID), (dict(nt=None), INVALID), (dict(pm=None), INVALID),
    (dict(nt=FAKE + 16), INVALID),
    (dict(pm=FAKE + 2), ALIGN), (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE), (dict(ws=FAKE + 128), ALIGN),
])
def test_compact_rejects_bad_arguments(lib, kw, code):
    assert compact(lib, **kw) == code


def test_pages_workspace_size(lib):
    f = lib.attn_pages_workspace_size
    assert f(-1, 4) == 0 and f(100, -1) == 0
    assert f(100000, 64) >= 2 * 100000 * 4 + 2 * 100000 // 8 and f(0, 0) > 0


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    t = torch.zeros(1, 2, 16 * 128 * 9 // 8, dtype=torch.uint8)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        ab.attn_kv4_gather(t, i, i[0], 16, torch.zeros(1, 2, 16, 128, dtype=torch.bfloat16),
                           torch.zeros(1, 2, 16, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA device"):
        ab.attn_pages_compact(i, i[0], i, i[0], 16, [t], t)
    with pytest.raises(TypeError):
        ab.attn_kv4_append(t.float(), t.float(), t, i, i[0], i[0], 16)
