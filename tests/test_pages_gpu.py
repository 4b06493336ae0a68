"""attn_pages_fork and attn_pages_compact on the GPU against the sequential oracle: tables, lengths and
counts exactly, pool contents byte for byte (pages the operator must not touch among them)."""

import numpy as np
import pytest
import torch

import attn_fwd_05_b200 as ab
from oracle import pages

pytestmark = pytest.mark.gpu
OK, INVALID, BAD_PAGE, TOO_LARGE = 0, 1, 6, 8


def dev():
    return torch.device("cuda:0")


def ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(dev())


def make_pools(rng, num_pages, shapes):
    out = []
    for shape, dtype in shapes:
        n = int(np.prod(shape)) * dtype.itemsize
        raw = torch.from_numpy(rng.integers(0, 255, (num_pages, n), dtype=np.uint8))
        out.append(raw.to(dev()).view(dtype).view(num_pages, *shape))
    return out


def raw(p):
    return p.contiguous().view(torch.uint8).reshape(p.shape[0], -1).cpu().numpy()


def widened(table, more):
    t = np.asarray(table, dtype=np.int32)
    return np.concatenate([t, np.full((t.shape[0], more), -1, dtype=np.int32)], axis=1)


def run_fork(table, lens, parents, add, new_cols, ps, pools, n_free=True, more=0):
    """more: columns that no row fills."""
    rows = len(parents)
    table, new_cols = widened(table, more), new_cols + more
    nt = torch.full((rows, new_cols), 77, dtype=torch.int32, device=dev())
    nl = torch.full((rows,), 77, dtype=torch.int32, device=dev())
    left = ints([77]) if n_free else None
    ws = torch.full((ab.attn_pages_workspace_size(pools[0].shape[0], rows),), 0xA5, dtype=torch.uint8, device=dev())
    ab.attn_pages_fork(ints(table), ints(lens), ints(parents), None if add is None else ints(add), nt, nl, ps, pools, ws,
                       left)
    status = ab.attn_get_device_status()
    nt = nt.cpu().numpy()
    assert (nt[:, new_cols - more:] == -1).all()
    return nt[:, :new_cols - more], nl.cpu().numpy(), None if left is None else int(left), status


def random_rows(rng, S, ps, cols, extra, lo=0):
    lens = [int(rng.integers(lo, cols * ps + 1)) for _ in range(S)]
    need = [-(-n // ps) for n in lens]
    num_pages = max(1, sum(need) + extra)
    perm = rng.permutation(num_pages)
    table = np.full((S, cols), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    return table, lens, num_pages


SHAPES = [((2, 16, 64), torch.bfloat16), ((2, 16, 64), torch.bfloat16)]
LARGE = [((4, 16, 4096), torch.bfloat16)] * 4  # more to copy than the planning launch takes
PLANS = [(SHAPES, 0), (LARGE, 0), (SHAPES, 2100)]  # and more entries than one CTA plans


@pytest.mark.parametrize("S,rows,cols,new_cols,ps,extra", [
    (1, 1, 1, 1, 16, 2), (4, 4, 5, 6, 16, 9), (3, 12, 4, 4, 32, 30), (8, 3, 7, 9, 16, 0), (40, 160, 6, 7, 64, 500),
    (1500, 2500, 2, 3, 16, 6000), (5, 7, 3, 3, 1, 60),
])
def test_fork_chain_matches_oracle(S, rows, cols, new_cols, ps, extra, cuda_device):
    rng = np.random.default_rng(S + rows)
    table, lens, num_pages = random_rows(rng, S, ps, cols, extra)
    pools = make_pools(rng, num_pages, SHAPES)
    for step in range(3):  # forks of forks: rows share full pages, and truncations make shared pages part-filled
        parents = [int(x) for x in rng.integers(-1, len(lens), rows)]
        add = None if step == 1 else [int(x) for x in rng.integers(-20, 20, rows)]
        before = [raw(p) for p in pools]
        want, wl, left, copies, short = pages.fork(table, lens, parents, add, new_cols, ps, num_pages)
        legal = all(p < 0 or 0 <= lens[p] + (0 if add is None else a) <= new_cols * ps
                    for p, a in zip(parents, add or [0] * rows))
        nt, nl, got_left, status = run_fork(table, lens, parents, add, new_cols, ps, pools)
        assert status in ((OK,) if legal and not short else (INVALID, TOO_LARGE))
        assert np.array_equal(nt, want) and np.array_equal(nl, wl) and got_left == left
        for b, p in zip(before, pools):
            for src, dst in copies:
                b[dst] = b[src]
            assert np.array_equal(raw(p), b)
        table, lens, cols = nt, [int(n) for n in nl], new_cols
        if short:
            break


@pytest.mark.parametrize("shapes,more", PLANS)
def test_fork_of_a_truncated_shared_page(shapes, more, cuda_device):
    # rows 0 and 1 share pages 0 and 1, which are full; row 0 then drops half of page 1: it must not write there
    rng = np.random.default_rng(2)
    pools = make_pools(rng, 6, shapes)
    before = raw(pools[0])
    nt, nl, left, status = run_fork([[0, 1, -1], [0, 1, 2]], [32, 40], [0, 1], [-8, 0], 3, 16, pools, more=more)
    assert status == OK and nl.tolist() == [24, 40] and nt.tolist() == [[0, 3, -1], [0, 1, 2]] and left == 2
    after = raw(pools[0])
    assert np.array_equal(after[3], before[1]) and np.array_equal(np.delete(after, 3, 0), np.delete(before, 3, 0))


@pytest.mark.parametrize("shapes,more", PLANS)
def test_fork_out_of_pages(shapes, more, cuda_device):
    rng = np.random.default_rng(3)
    pools = make_pools(rng, 3, shapes)
    before = raw(pools[0])
    nt, nl, left, status = run_fork([[0, -1], [1, -1]], [16, 5], [0, 1, 1], [1, 0, 0], 2, 16, pools, more=more)
    assert status == TOO_LARGE and nt.tolist() == [[0, 2], [1, -1], [-1, -1]] and left == 0
    assert np.array_equal(raw(pools[0]), before)


@pytest.mark.parametrize("shapes,more", PLANS)
def test_fork_bad_inputs_are_latched(shapes, more, cuda_device):
    rng = np.random.default_rng(4)
    pools = make_pools(rng, 8, shapes)
    table, lens = [[0, 1], [2, 3]], [20, 32]
    nt, nl, _, status = run_fork(table, lens, [0, 2, -2, 1], None, 2, 16, pools, more=more)
    assert status == INVALID and nl.tolist() == [20, 0, 0, 32] and nt.tolist() == [[0, 1], [-1, -1], [-1, -1], [2, 3]]
    nt, nl, _, status = run_fork(table, lens, [0, 1], [-21, 1 + 16 * more], 2, 16, pools, more=more)
    assert status == INVALID and nl.tolist() == [20, 32] and nt.tolist() == [[0, 1], [2, 3]]
    nt, nl, _, status = run_fork(table, [-3, 33 + 16 * more], [0, 1], [4, 0], 2, 16, pools, more=more)
    assert status == INVALID and nl.tolist() == [4, 0] and nt.tolist() == [[0, -1], [-1, -1]]
    before = raw(pools[0])
    nt, nl, _, status = run_fork([[8, 1], [2, -1]], lens, [0, 1, 0], None, 2, 16, pools, more=more)
    assert status == BAD_PAGE and nt.tolist() == [[-1, 1], [2, -1], [-1, 0]]
    after = raw(pools[0])
    assert np.array_equal(after[0], before[1]) and np.array_equal(after[1:], before[1:])
    # a part-filled page out of range: nothing to copy
    nt, nl, _, status = run_fork([[0, 99], [2, 3]], lens, [0, 0], None, 2, 16, pools, more=more)
    assert status == BAD_PAGE and nt.tolist() == [[0, -1], [0, -1]]
    nt, nl, left, status = run_fork(table, lens, [], None, 2, 16, pools, more=more)
    assert status == OK and left == 8


@pytest.mark.parametrize("S,cols,ps,extra,shapes", [
    (1, 1, 16, 0, SHAPES[:1]), (3, 4, 16, 20, SHAPES), (9, 3, 64, 1, [((3, 16), torch.uint8)]), (3, 4, 16, 20, LARGE),
    (70, 40, 16, 3000, [((5, 48), torch.uint8)] * 4), (2000, 2, 16, 40000, [((16,), torch.uint8)]),
    (2, 3, 7, 4, [((1, 40000), torch.bfloat16)]), (4, 2, 16, 33, SHAPES),
])
def test_compact_matches_oracle(S, cols, ps, extra, shapes, cuda_device):
    rng = np.random.default_rng(S + cols)
    table, lens, num_pages = random_rows(rng, S, ps, cols, extra)
    if S > 1 and lens[0] and lens[1]:
        table[1, 0] = table[0, 0]  # a shared page
    pools = make_pools(rng, num_pages, shapes)
    before = [raw(p) for p in pools]
    want, page_map, live, moves = pages.compact(table, lens, ps, num_pages)
    ws = torch.full((ab.attn_pages_workspace_size(num_pages, S),), 0xA5, dtype=torch.uint8, device=dev())
    t, n = ints(table), ints(lens)
    nt, pm, nlive = torch.empty_like(t), torch.full((num_pages,), 77, dtype=torch.int32, device=dev()), ints([77])
    ab.attn_pages_compact(t, n, nt, pm, ps, pools, ws, nlive)
    assert ab.attn_get_device_status() == OK
    assert np.array_equal(nt.cpu().numpy(), want) and np.array_equal(pm.cpu().numpy(), page_map) and int(nlive) == live
    for b, p in zip(before, pools):
        for src, dst in moves:
            b[dst] = b[src]
        assert np.array_equal(raw(p), b)
    # in place, on the compacted table: nothing moves any more
    ab.attn_pages_compact(nt, n, nt, pm, ps, pools, ws)
    assert ab.attn_get_device_status() == OK
    assert np.array_equal(nt.cpu().numpy(), want)
    assert pm.tolist() == list(range(live)) + [-1] * (num_pages - live)
    for b, p in zip(before, pools):
        assert np.array_equal(raw(p), b)


@pytest.mark.parametrize("shapes,more", PLANS)
def test_compact_bad_inputs_are_latched(shapes, more, cuda_device):
    rng = np.random.default_rng(6)
    pools = make_pools(rng, 6, shapes)
    ws = torch.empty(ab.attn_pages_workspace_size(6, 3), dtype=torch.uint8, device=dev())
    t, n = ints(widened([[5, 9], [4, 1], [2, 3]], more)), ints([32, 20, -4])
    nt, pm, nlive = torch.empty_like(t), torch.empty(6, dtype=torch.int32, device=dev()), ints([0])
    ab.attn_pages_compact(t, n, nt, pm, 16, pools, ws, nlive)
    assert ab.attn_get_device_status() in (INVALID, BAD_PAGE)
    assert nt[:, :2].tolist() == [[2, -1], [0, 1], [-1, -1]] and (nt[:, 2:] == -1).all() and int(nlive) == 3 and pm.tolist() == [-1, 1, -1, -1, 0, 2]


def test_pages_without_rows_or_pools_of_no_pages(cuda_device):
    pools = [torch.empty((0, 64), dtype=torch.uint8, device=dev())]
    ws = torch.empty(ab.attn_pages_workspace_size(0, 2), dtype=torch.uint8, device=dev())
    t, n = ints([[-1, -1], [-1, -1]]), ints([0, 0])
    nt, nl, left = torch.empty_like(t), torch.empty_like(n), ints([5])
    ab.attn_pages_fork(t, n, ints([1, 0]), None, nt, nl, 16, pools, ws, left)
    assert ab.attn_get_device_status() == OK and nl.tolist() == [0, 0] and (nt == -1).all() and int(left) == 0
    ab.attn_pages_compact(t, n, nt, torch.empty(0, dtype=torch.int32, device=dev()), 16, pools, ws, left)
    assert ab.attn_get_device_status() == OK and (nt == -1).all() and int(left) == 0


def test_binding_refusals(cuda_device):
    pools = [torch.zeros((4, 64), dtype=torch.uint8, device=dev())]
    ws = torch.empty(ab.attn_pages_workspace_size(4, 2), dtype=torch.uint8, device=dev())
    t, n = ints([[0, 1], [2, 3]]), ints([20, 20])
    nt, nl, pm = torch.empty_like(t), torch.empty_like(n), ints([0, 0, 0, 0])
    bad = [
        lambda: ab.attn_pages_fork(t, n[:1], n, None, nt, nl, 16, pools, ws),
        lambda: ab.attn_pages_fork(t, n, n, ints([1]), nt, nl, 16, pools, ws),
        lambda: ab.attn_pages_fork(t, n, n, None, nt, nl, 16, [], ws),
        lambda: ab.attn_pages_fork(t, n, n, None, nt, nl, 16, pools + [torch.zeros((4, 32), dtype=torch.uint8, device=dev())], ws),
        lambda: ab.attn_pages_compact(t, n, nt[:1], pm, 16, pools, ws),
        lambda: ab.attn_pages_compact(t, n, nt, pm[:3], 16, pools, ws),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ab.AttnError):
        ab.attn_pages_fork(t, n, ints([0, 1]), None, t, nl, 16, pools, ws)
    with pytest.raises(ab.AttnError):
        ab.attn_pages_compact(t, n, nt, pm, 16, pools, ws[:256])
    assert ab.attn_get_device_status() == OK


@pytest.mark.parametrize("more", [0, 2100])
def test_bf16_cache_forked_compacted_and_decoded_in_a_graph(more, cuda_device):
    # K and V pools of attn_decode_paged: every row of the new table answers as its parent did, bit for bit
    rng = np.random.default_rng(31 + more)
    ps, Hkv, Hq, d = 16, 2, 8, 128
    table, lens, num_pages = random_rows(rng, 4, ps, 40, 30, lo=1)
    fill = [torch.randn((num_pages, Hkv, ps, d), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16) for i in range(2)]
    pools = [f.to(dev()) for f in fill]
    parents = [2, 0, 0, 3, 1, 0]
    q0 = torch.randn((4, Hq, d), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(dev())
    q = q0[parents].contiguous()
    t, n, cols = ints(widened(table, more)), ints(lens), 40 + more

    def decode(q, table, lens, o, lse, ws):
        ab.attn_decode_paged(q, pools[0], pools[1], table, lens, ps, o, lse, 0.09, ws)

    def outputs(rows):
        return (torch.empty((rows, Hq, d), dtype=torch.bfloat16, device=dev()),
                torch.empty((rows, Hq), dtype=torch.float32, device=dev()),
                torch.empty(ab.attn_decode_paged_workspace_size(rows, Hq, Hkv, d, cols, ps), dtype=torch.uint8, device=dev()))

    o0, l0, ws0 = outputs(4)
    decode(q0, t, n, o0, l0, ws0)
    o, lse, ws = outputs(6)
    nt, nl = torch.empty((6, cols), dtype=torch.int32, device=dev()), torch.empty(6, dtype=torch.int32, device=dev())
    pm, par = torch.empty(num_pages, dtype=torch.int32, device=dev()), ints(parents)
    pws = torch.empty(ab.attn_pages_workspace_size(num_pages, 6), dtype=torch.uint8, device=dev())

    def step():
        ab.attn_pages_fork(t, n, par, None, nt, nl, ps, pools, pws)
        ab.attn_pages_compact(nt, nl, nt, pm, ps, pools, pws)
        decode(q, nt, nl, o, lse, ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for replay in range(3):
        for p, f in zip(pools, fill):
            p.copy_(f)
        for x in (o, lse, nt, nl, pm):
            x.zero_()
        pws.fill_(0x5A)
        g.replay() if replay else step()
        assert ab.attn_get_device_status() == OK
        assert torch.equal(o, o0[parents]) and torch.equal(lse, l0[parents])
    del g
