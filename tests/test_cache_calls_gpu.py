"""Calls of the 4-bit cache and page entry points that name a buffer twice, or split one step over two calls."""

import numpy as np
import pytest
import torch

import attn_fwd_05_b200 as ab
from test_kv4_gpu import BF, dev, layout, random_pool
from test_pages_gpu import LARGE, SHAPES, ints, make_pools, random_rows, raw

pytestmark = pytest.mark.gpu


def test_gather_of_both_into_one_buffer_leaves_v(cuda_device):
    rng = np.random.default_rng(51)
    lens, Hkv, d, ps = [70, 0, 33], 2, 128, 16
    table, num_pages = layout(rng, lens, ps)
    pool = torch.from_numpy(random_pool(rng, num_pages, Hkv, ps, d)).to(dev())
    t, n = ints(table), ints(lens)
    k, v, both = (torch.full((3, Hkv, 72, d), 7.25, dtype=BF, device=dev()) for _ in range(3))
    ab.attn_kv4_gather(pool, t, n, ps, k, v)
    ab.attn_kv4_gather(pool, t, n, ps, both, both)
    assert ab.attn_get_device_status() == 0
    assert torch.equal(both, v) and not torch.equal(k, v)


@pytest.mark.parametrize("shapes", [SHAPES, LARGE])
def test_a_pool_listed_twice_is_moved_once(shapes, cuda_device):
    rng = np.random.default_rng(52)
    table, lens, num_pages = random_rows(rng, 6, 16, 8, 60, lo=1)
    pool = make_pools(rng, num_pages, shapes[:1])[0]
    parents = [0, 0, 3, 5, 5, 1]
    got = []
    for times in (1, 2):
        p = pool.clone()
        ws = torch.empty(ab.attn_pages_workspace_size(num_pages, 6), dtype=torch.uint8, device=dev())
        nt, nl = ints(np.zeros((6, 9))), ints(np.zeros(6))
        ab.attn_pages_fork(ints(table), ints(lens), ints(parents), None, nt, nl, 16, [p] * times, ws)
        ct, pm = torch.empty_like(nt), ints(np.zeros(num_pages))
        ab.attn_pages_compact(nt, nl, ct, pm, 16, [p] * times, ws)
        assert ab.attn_get_device_status() == 0
        got.append((nt.cpu().numpy(), ct.cpu().numpy(), pm.cpu().numpy(), raw(p)))
    assert not np.array_equal(got[0][0], got[0][1])
    for a, b in zip(*got):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("more", [0, 2100])
def test_many_pools_in_several_calls(more, cuda_device):
    # 160 pools that share a table, 128 and 32 a call, against all of them moved in calls of one
    rng = np.random.default_rng(53)
    table, lens, num_pages = random_rows(rng, 5, 16, 6, 40, lo=1)
    table = np.concatenate([table, np.full((5, more), -1, dtype=np.int32)], axis=1)
    fill = torch.from_numpy(rng.integers(0, 256, (160, num_pages, 48), dtype=np.uint8)).to(dev())
    parents = ints([4, 4, 0, 2, 2, 1])

    def step(pools, sizes):
        tables, at = [], 0
        ws = torch.empty(ab.attn_pages_workspace_size(num_pages, 6), dtype=torch.uint8, device=dev())
        nt, nl = torch.empty((6, 6 + more), dtype=torch.int32, device=dev()), ints(np.zeros(6))
        for n in sizes:
            ab.attn_pages_fork(ints(table), ints(lens), parents, None, nt, nl, 16, pools[at:at + n], ws)
            tables.append(nt.clone())
            at += n
        at = 0
        ct, pm = torch.empty_like(nt), ints(np.zeros(num_pages))
        for n in sizes:
            ab.attn_pages_compact(nt, nl, ct, pm, 16, pools[at:at + n], ws)
            tables.append(ct.clone())
            at += n
        assert ab.attn_get_device_status() == 0
        assert all(torch.equal(t, tables[0]) for t in tables[:len(sizes)])
        assert all(torch.equal(t, tables[-1]) for t in tables[len(sizes):])
        return tables[0], tables[-1], torch.stack(pools)

    a, b = fill.clone(), fill.clone()
    for x, y in zip(step(list(a), [128, 32]), step(list(b), [1] * 160)):
        assert torch.equal(x, y)
