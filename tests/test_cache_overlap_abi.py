"""The 4-bit cache and page entry points refuse buffers that are written while another of the call's buffers
that shares their bytes is read or written (host checks: these run without a device)."""

import ctypes

import pytest

from attn_fwd_05_b200 import binding, build

INVALID = 1
# one buffer each, far apart and 256-byte aligned; never dereferenced, since every call below is refused
NAMES = ["k", "v", "k_out", "v_out", "pool", "pool2", "table", "lens", "cu", "q", "o", "lse", "parents", "add", "new_table",
         "new_lens", "n_free", "page_map", "n_live", "ws"]
PLACE = {name: (i + 1) << 32 for i, name in enumerate(NAMES)}


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def calls(lib, p):
    """The status of each entry point with the buffers at p."""
    pools = (ctypes.c_void_p * 2)(p["pool"], p["pool2"])
    return {
        "append": lambda: lib.attn_kv4_append(p["k"], p["v"], 1024, 1024, p["pool"], p["table"], p["lens"], p["cu"], 16,
                                              p["k_out"], p["v_out"], 4, 40, 8, 128, 64, 8, None),
        "gather": lambda: lib.attn_kv4_gather(p["pool"], p["table"], p["lens"], 16, p["k"], p["v"], 4, 8, 100, 128, 64, 8,
                                              None),
        "decode": lambda: lib.attn_decode_paged_kv4(p["q"], p["pool"], p["table"], p["lens"], 16, p["o"], p["lse"], 4, 64, 8,
                                                    128, 64, 8, ctypes.c_float(0.1), p["ws"], 1 << 30, None),
        "fork": lambda: lib.attn_pages_fork(p["table"], p["lens"], p["parents"], p["add"], p["new_table"], p["new_lens"],
                                            16, pools, 2, 4096, 4, 8, 6, 9, 64, p["n_free"], p["ws"], 1 << 30, None),
        "compact": lambda: lib.attn_pages_compact(p["table"], p["lens"], p["new_table"], p["page_map"], 16, pools, 2, 4096,
                                                  4, 8, 64, p["n_live"], p["ws"], 1 << 30, None),
    }


BYTES = {"append": dict(k=81920, v=81920, k_out=81920, v_out=81920, pool=64 * 18432, table=128, lens=16, cu=20),
         "gather": dict(k=819200, v=819200, pool=64 * 18432, table=128, lens=16),
         "decode": dict(q=65536, o=65536, lse=1024, pool=64 * 18432, table=128, lens=16, ws=1 << 20),
         "fork": dict(table=128, lens=16, parents=24, add=24, new_table=216, new_lens=24, n_free=4, ws=2048, pool=64 * 4096,
                      pool2=64 * 4096),
         "compact": dict(table=128, lens=16, new_table=128, page_map=256, n_live=4, ws=2048, pool=64 * 4096,
                         pool2=64 * 4096)}
WRITTEN = {"append": ["k_out", "v_out", "pool"], "gather": ["k", "v"], "decode": ["o", "lse", "ws"],
           "fork": ["new_table", "new_lens", "n_free", "ws", "pool"],
           "compact": ["new_table", "page_map", "n_live", "ws", "pool"]}
FREE = [("fork", "pool", "pool2"), ("compact", "pool", "pool2")]  # pools: the caller's
SAME = [("append", "k_out", "k"), ("append", "v_out", "v"), ("gather", "k", "v"), ("gather", "v", "k"),
        ("compact", "new_table", "table")]  # may be one and the same buffer
PAIRS = [(op, a, b) for op in WRITTEN for a in WRITTEN[op] for b in BYTES[op] if a != b and (op, a, b) not in FREE]


@pytest.mark.parametrize("op,a,b", PAIRS)
def test_shared_bytes_are_refused(op, a, b, lib):
    # `a` from the last bytes of `b` on, up to its first bytes, and from its first (or, where they may be one buffer,
    # from its 17th) byte on
    na, nb = BYTES[op][a], BYTES[op][b]
    for off in {(nb - 1) // 256 * 256, -((na - 1) // 256 * 256), 0} - {0} | {16 if (op, a, b) in SAME else 0}:
        p = dict(PLACE)
        p[a] = p[b] + off
        assert calls(lib, p)[op]() == INVALID, off


@pytest.mark.parametrize("op", ["fork", "compact"])
@pytest.mark.parametrize("off", [4096, -16, 63 * 4096])
def test_pools_that_overlap_in_part_are_refused(op, off, lib):
    p = dict(PLACE)
    p["pool2"] = p["pool"] + off
    assert calls(lib, p)[op]() == INVALID
