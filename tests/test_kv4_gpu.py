"""GPU parity of the 4-bit paged cache (append, gather, decode) against the fp64 oracle.

Appended pools and gathered values are compared bit for bit: the quantizer's definition leaves
no freedom, and a gathered value is s * c + m rounded to fp32 and then to bf16.

Decode tolerances, per output element and derived from the roundings the kernel makes:
* p * s is rounded to fp16 (2^-11 of it) and multiplies a centred code of at most 8 in magnitude: with
  weights that sum to 1, at most 2^-11 * 8 * S, S the largest V scale of the head and group; below
  2^-14 of the scaling unit 2^e <= S fp16 loses at most 2^-25 units a token instead, at most
  n * 2^-25 * 8 * S over n tokens against a sum of at least 1;
* bf16 output: 2^-8 of the value;
* scores: products of a code and a scaled q are exact, their fp32 sums over 64 channels are off by
  at most 64 * 2^-24 of the sum of magnitudes, and the scale and minimum add four more roundings:
  E = 68 * 2^-24 * scale * sum_c |q_c| (8 s + |m + 8 s|).  A score error E moves an output by at
  most 2 E * max |V|, the exponential's own 2^-22 and fp32 sums (n * 2^-24) by as much again;
* the log-sum-exp is off by E, n * 2^-24 for the sum, and 2^-22 of its own value.
"""

import math

import numpy as np
import pytest
import torch

import attn_fwd_05_b200 as ab
from attn_fwd_05_b200 import binding
from oracle import attention, kv4

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def dev():
    return torch.device("cuda:0")


def bf16(rng, shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(BF)


def f64(t):
    return t.double().cpu().numpy()


def layout(rng, lens, page_size, spare=2, cols=None):
    """A table that deals random pages out to the rows, -1 past each row's pages."""
    need = [-(-n // page_size) for n in lens]
    cols = cols or max(1, max(need, default=1))
    num_pages = sum(need) + spare
    perm = rng.permutation(num_pages)
    table = np.full((len(lens), cols), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, num_pages


def random_pool(rng, num_pages, Hkv, page_size, d, s_lo=0.05, s_hi=0.6):
    """Random codes; scales in [s_lo, s_hi), minima about 7.5 steps below zero."""
    ng = d // 64
    rec = rng.integers(0, 256, (num_pages, Hkv, page_size // 16, kv4.record_bytes(d)), dtype=np.uint8)
    par = rec[..., 1024 * ng:].view(np.uint16)
    s = rng.uniform(s_lo, s_hi, (*par.shape[:-1], 32 * ng)).astype(np.float32)
    m = (-7.5 * s + rng.standard_normal(s.shape) * s).astype(np.float32)
    par[..., 0::2] = kv4.bf16_bits(s)
    par[..., 1::2] = kv4.bf16_bits(m)
    return rec.reshape(num_pages, Hkv, -1)


def poison_unused(pool, table, lens, page_size, d):
    """NaN parameters in every slot that no sequence uses."""
    P, H, _ = pool.shape
    used = np.zeros((P, page_size), dtype=bool)
    for row, n in zip(table, lens):
        for t in range(n):
            used[row[t // page_size], t % page_size] = True
    rec = pool.reshape(P, H, page_size // 16, -1)
    for p, t in zip(*np.nonzero(~used)):
        for v in (False, True):
            for g in range(d // 64):
                at = kv4.param_place(v, t % 16, g, d)
                rec[p, :, t // 16, at:at + 4] = 0xFF
    return pool


def run_decode(q, pool, table, lens, page_size, scale, with_lse=True, stream=None):
    S, Hq, d = q.shape
    Hkv = pool.shape[1]
    o = torch.full((S, Hq, d), float("nan"), dtype=BF, device=dev())
    lse = torch.full((S, Hq), float("nan"), dtype=torch.float32, device=dev()) if with_lse else None
    ws = torch.empty(ab.attn_decode_paged_kv4_workspace_size(S, Hq, Hkv, d), dtype=torch.uint8, device=dev())
    ws.fill_(0xFF)
    t = [torch.as_tensor(x).to(dev()) for x in (pool, table, np.asarray(lens, dtype=np.int32))]
    ab.attn_decode_paged_kv4(q.to(dev()), t[0], t[1], t[2], page_size, o, lse, scale, ws, stream)
    return o, lse, ab.attn_get_device_status(stream)


def check_decode(o, lse, q, pool, table, lens, page_size, scale):
    ref_o, ref_l = kv4.decode_paged_kv4(q, pool, table, lens, page_size, scale)
    o, lse, qf = f64(o), f64(lse), f64(q)
    S, Hq, d = qf.shape
    Hkv = pool.shape[1]
    K, V = kv4.pool_values(pool, page_size, d)
    rec = pool.reshape(*pool.shape[:2], page_size // 16, -1)
    words = rec.view(np.uint16)
    _, par = kv4.places(d)
    ks, km, vs = (kv4.bf16_value(words[..., at // 2 + w]).reshape(*pool.shape[:2], page_size, d // 64)
                  for at, w in ((par[0], 0), (par[0], 1), (par[1], 0)))
    for i, n in enumerate(lens):
        if n == 0:
            assert np.all(o[i] == 0) and np.all(np.isneginf(lse[i]))
            continue
        pages = table[i][: -(-n // page_size)]
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            cut = lambda x: x[pages, kv].reshape(-1, *x.shape[3:])[:n]  # noqa: E731
            big_s = np.repeat(cut(vs).max(0), 64)
            mag = 8 * cut(ks) + np.abs(cut(km) + 8 * cut(ks))
            e = 68 * 2.0 ** -24 * scale * float((mag @ np.abs(qf[i, h]).reshape(-1, 64).sum(-1)).max())
            rel = 2 * (e + 2.0 ** -22 + n * 2.0 ** -24)
            vmax = np.abs(cut(V)).max(0)
            tol = (2.0 ** -11 + n * 2.0 ** -25) * 8 * big_s + 2.0 ** -8 * np.abs(ref_o[i, h]) + rel * (vmax + 8 * big_s)
            err = np.abs(o[i, h] - ref_o[i, h])
            assert np.all(err <= tol), f"row {i} head {h}: {np.max(err / tol):.2f} of the tolerance"
            le = abs(lse[i, h] - ref_l[i, h])
            assert le <= e + n * 2.0 ** -24 + 2.0 ** -22 * abs(ref_l[i, h]) + 2.0 ** -21, f"row {i} head {h}: lse off by {le:.2e}"


def widen(table, page_size, tokens=20000):
    """The table with columns for rows of up to `tokens`: the host then has to expect long rows."""
    more = np.full((table.shape[0], -(-tokens // page_size)), -1, dtype=np.int32)
    return np.ascontiguousarray(np.concatenate([table, more], axis=1))


CASES = [
    # lens, Hq, Hkv, d, page_size
    ([1], 1, 1, 64, 16),
    ([1, 15, 16, 17, 1500], 8, 2, 128, 16),
    ([3000, 1024, 0, 1025, 2048], 8, 1, 128, 16),   # 8 query heads: a full tile; an empty row between
    ([0, 0, 700, 33, 64, 0], 4, 4, 64, 32),         # MHA; empty rows first and last
    ([513, 130, 65], 4, 2, 256, 64),
    ([63, 64, 65], 12, 1, 256, 16),                 # more than 8 heads at d = 256: two passes
    ([900, 77], 32, 2, 128, 16),                    # 16 per KV head: two column tiles
    ([1300, 5], 40, 2, 128, 32),                    # 20 per KV head: 16 and 4
    ([300, 40], 64, 1, 64, 16),                     # 64 per KV head
    ([2500], 3, 1, 128, 64),                        # odd group
    ([310, 4000], 27, 3, 128, 16),                  # odd head counts, group 9
    # around 64 segments: smaller clusters
    ([1, 2, 31, 0, 32, 33, 1000, 127, 128, 129, 4096], 16, 8, 128, 16),
    ([700, 64, 3, 2047, 0, 500, 12, 90], 18, 9, 256, 32),
    ([333, 100, 1], 16 * 18, 16, 64, 64),           # 18 per KV head: 96 segments
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,d,ps", CASES)
def test_decode_matches_oracle(lens, Hq, Hkv, d, ps, wide, cuda_device):
    rng = np.random.default_rng(Hq * d + len(lens))
    table, num_pages = layout(rng, lens, ps)
    pool = poison_unused(random_pool(rng, num_pages, Hkv, ps, d), table, lens, ps, d)
    table = widen(table, ps) if wide else table
    q = bf16(rng, (len(lens), Hq, d))
    scale = 1.0 / math.sqrt(d)
    o, lse, status = run_decode(q, pool, table, lens, ps, scale)
    assert status == 0, ab.attn_status_string(status)
    check_decode(o, lse, q, pool, table, lens, ps, scale)


def test_decode_of_many_rows(cuda_device):
    # more rows than the planning block has threads, most of them a tile or two long
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 40, 700)]
    table, num_pages = layout(rng, lens, 16)
    pool = random_pool(rng, num_pages, 2, 16, 64)
    q = bf16(rng, (700, 6, 64))
    o, lse, status = run_decode(q, pool, table, lens, 16, 0.125)
    assert status == 0
    check_decode(o, lse, q, pool, table, lens, 16, 0.125)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kind", ["peaked", "rising", "growing_v", "tiny_v", "huge_v", "flat", "large_q", "small_q"])
def test_decode_value_ranges(kind, wide, cuda_device):
    rng = np.random.default_rng(17)
    d, ps, lens = 128, 16, [1111, 600]
    table, num_pages = layout(rng, lens, ps)
    table = widen(table, ps) if wide else table
    pool = random_pool(rng, num_pages, 2, ps, d)
    q = bf16(rng, (2, 8, d))
    scale = 1.0 / math.sqrt(d)
    rec = pool.reshape(num_pages, 2, 1, -1)
    words = rec.view(np.uint16)
    _, par = kv4.places(d)

    def factor(which, f):  # scales s and m of every token by f(position) (a power of two)
        for i, n in enumerate(lens):
            for t in range(n):
                for at in par[which][t % 16]:
                    for w in (at // 2, at // 2 + 1):
                        x = kv4.bf16_value(words[table[i][t // ps], :, 0, w]) * f(t)
                        words[table[i][t // ps], :, 0, w] = kv4.bf16_bits(x.astype(np.float32))

    if kind == "peaked":
        scale = 4.0                      # one key takes nearly all the weight
    elif kind == "rising":
        factor(0, lambda t: 2.0 ** (t // 100 - 6))   # scores grow: the running maximum keeps rising
    elif kind == "growing_v":
        factor(1, lambda t: 2.0 ** (t // 40 - 14))   # V's scale grows by 2^27 along the row
    elif kind == "tiny_v":
        factor(1, lambda t: 2.0 ** -90)
    elif kind == "huge_v":
        factor(1, lambda t: 2.0 ** 80)
    elif kind == "flat":                 # constant groups: s = 0
        for at in par[1].ravel():
            words[..., at // 2] = 0
    elif kind == "large_q":
        q, scale = (q.float() * 2.0 ** 40).to(BF), scale * 2.0 ** -40
    elif kind == "small_q":
        q, scale = (q.float() * 2.0 ** -40).to(BF), scale * 2.0 ** 40
    o, lse, status = run_decode(q, pool, table, lens, ps, scale)
    assert status == 0
    check_decode(o, lse, q, pool, table, lens, ps, scale)


@pytest.mark.parametrize("wide", [False, True])
def test_decode_is_repeatable_and_placement_free(wide, cuda_device):
    rng = np.random.default_rng(8)
    lens = [700, 33, 2900]
    table, num_pages = layout(rng, lens, 32)
    table = widen(table, 32) if wide else table
    pool = random_pool(rng, num_pages, 2, 32, 128)
    q = bf16(rng, (3, 8, 128))
    o1, l1, _ = run_decode(q, pool, table, lens, 32, 0.09)
    o2, l2, _ = run_decode(q, pool, table, lens, 32, 0.09)
    perm = rng.permutation(num_pages)
    moved = np.empty_like(pool)
    moved[perm] = pool
    t2 = np.where(table >= 0, perm[np.maximum(table, 0)], -1).astype(np.int32)
    o3, l3, _ = run_decode(q, moved, t2, lens, 32, 0.09)
    o4, _, _ = run_decode(q, pool, table, lens, 32, 0.09, with_lse=False)
    for o, lse in ((o2, l2), (o3, l3), (o4, l1)):
        assert torch.equal(o1, o) and torch.equal(l1, lse)


@pytest.mark.parametrize("wide", [False, True])
def test_decode_nan_groups_stay_in_their_rows(wide, cuda_device):
    rng = np.random.default_rng(9)
    lens, d = [200, 200], 128
    table, num_pages = layout(rng, lens, 16)
    table = widen(table, 16) if wide else table
    pool = random_pool(rng, num_pages, 1, 16, d)
    rec = pool.reshape(num_pages, 1, 1, -1)
    # V group 1 of token 37 of row 0 is NaN; K of token 5 of row 1 too
    at = kv4.param_place(True, 37 % 16, 1, d)
    rec[table[0][37 // 16], 0, 0, at:at + 4] = np.array([0x7FC0, 0x7FC0], dtype=np.uint16).view(np.uint8)
    q = bf16(rng, (2, 4, d))
    o, lse, status = run_decode(q, pool, table, lens, 16, 0.09)
    assert status == 0
    assert torch.isnan(o[0, :, 64:]).all() and torch.isfinite(o[0, :, :64]).all() and torch.isfinite(o[1]).all()
    assert torch.isfinite(lse).all()
    at = kv4.param_place(False, 5, 0, d)
    rec[table[1][0], 0, 0, at:at + 4] = np.array([0x7FC0, 0x7FC0], dtype=np.uint16).view(np.uint8)
    o, lse, _ = run_decode(q, pool, table, lens, 16, 0.09)
    assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all() and torch.isfinite(lse[0]).all()


@pytest.mark.parametrize("wide", [False, True])
def test_decode_queries_that_are_not_finite_stay_in_their_heads(wide, cuda_device):
    rng = np.random.default_rng(12)
    lens = [500, 40]
    table, num_pages = layout(rng, lens, 16)
    pool = random_pool(rng, num_pages, 1, 16, 64)
    q = bf16(rng, (2, 5, 64))
    q[0, 1], q[1, 3, 7] = float("nan"), float("inf")
    o, lse, status = run_decode(q, pool, widen(table, 16) if wide else table, lens, 16, 0.125)
    assert status == 0
    assert torch.isnan(o[0, 1]).all() and torch.isnan(lse[0, 1]) and not torch.isfinite(o[1, 3]).any()
    for row, rest in ((0, [0, 2, 3, 4]), (1, [0, 1, 2, 4])):
        check_decode(o[row:row + 1, rest], lse[row:row + 1, rest], q[row:row + 1, rest], pool, table[row:row + 1],
                     lens[row:row + 1], 16, 0.125)


@pytest.mark.parametrize("wide", [False, True])
def test_decode_bad_pages_and_lengths_are_reported(wide, cuda_device):
    rng = np.random.default_rng(10)
    lens = [100, 50, 64]
    table, num_pages = layout(rng, lens, 16)
    table = widen(table, 16) if wide else table
    pool = random_pool(rng, num_pages, 2, 16, 128)
    q = bf16(rng, (3, 8, 128))
    t = table.copy()
    t[0, 2], t[1, 0] = num_pages + 5, -7       # in use; entries past a row's end are never read
    t[2, 4:] = 12345
    o, lse, status = run_decode(q, pool, t, lens, 16, 0.1)
    assert status == 6 and ab.attn_get_device_status() == 0
    assert torch.isfinite(o).all()
    check_decode(o[2:], lse[2:], q[2:], pool, table[2:], lens[2:], 16, 0.1)
    o, lse, status = run_decode(q, pool, table, [100, -1, 16 * table.shape[1] + 1], 16, 0.1)
    assert status == 1
    assert (o[1:] == 0).all() and torch.isneginf(lse[1:]).all()
    # every page of a row out of range: an empty row
    t[0] = -1
    o, lse, status = run_decode(q, pool, t, lens, 16, 0.1)
    assert status == 6 and (o[0] == 0).all() and torch.isneginf(lse[0]).all()


# ------------------------------------------------------------------ append


def run_append(k, v, pool, table, lens, cu, page_size, outs=True):
    p, t, n, c = (torch.as_tensor(np.asarray(x)).to(dev()) for x in
                  (pool, table, np.asarray(lens, dtype=np.int32), np.asarray(cu, dtype=np.int32)))
    ko = torch.full(k.shape, float("nan"), dtype=BF, device=dev()) if outs else None
    vo = torch.full(v.shape, float("nan"), dtype=BF, device=dev()) if outs else None
    ab.attn_kv4_append(k, v, p, t, n, c, page_size, ko, vo)
    return p.cpu().numpy(), ko, vo, ab.attn_get_device_status()


def bits(x64):
    """bf16 bits of fp64 values through fp32, as the kernels round them."""
    return kv4.bf16_bits(np.asarray(x64).astype(np.float32))


def bf16_bits_of(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def same_values(t, x64):
    got, want = bf16_bits_of(t), bits(x64)
    nan = np.isnan(x64)
    return np.array_equal(got[~nan], want[~nan]) and np.array_equal(np.isnan(f64(t)), nan)


@pytest.mark.parametrize("Hkv,d,ps,past,new", [
    (1, 64, 16, [0], [1]),
    (2, 128, 16, [0, 3, 15, 16, 17], [1, 1, 1, 1, 1]),            # one decode step at every offset of a block
    (2, 128, 32, [0, 30, 5, 0], [33, 3, 0, 70]),                  # ragged prompts, one without new tokens
    (3, 64, 64, [1, 62, 64], [1, 4, 130]),
    (1, 256, 16, [2, 0, 7], [5, 18, 9]),
])
@pytest.mark.parametrize("fused", [False, True])
def test_append_matches_oracle(Hkv, d, ps, past, new, fused, cuda_device):
    rng = np.random.default_rng(d + len(new))
    lens = [p + n for p, n in zip(past, new)]
    cu = np.concatenate([[0], np.cumsum(new)])
    table, num_pages = layout(rng, lens, ps)
    pool = rng.integers(0, 256, (num_pages, Hkv, ps * d * 9 // 8), dtype=np.uint8)
    x = bf16(rng, (int(cu[-1]), 3, Hkv, d))
    x[:, 1] += (3 * torch.randn(Hkv, d, generator=torch.Generator().manual_seed(1))).to(BF)
    x = x.to(dev())
    k, v = (x[:, 1], x[:, 2]) if fused else (x[:, 1].contiguous(), x[:, 2].contiguous())
    got, ko, vo, status = run_append(k, v, pool, table, lens, cu, ps)
    assert status == 0, ab.attn_status_string(status)
    want = kv4.append(pool, f64(k), f64(v), table, lens, cu, ps)
    assert np.array_equal(got, want)  # every byte, those of other tokens too
    assert same_values(ko, kv4.values(*kv4.quantize(f64(k)))) and same_values(vo, kv4.values(*kv4.quantize(f64(v))))
    again, _, _, _ = run_append(k, v, pool, table, lens, cu, ps, outs=False)
    assert np.array_equal(again, want)


def test_append_special_values(cuda_device):
    rng = np.random.default_rng(23)
    n, d = 24, 128
    x = torch.zeros(n, 1, d)
    x[0] = -3.5
    x[1, 0, :2] = torch.tensor([-0.0, 0.0])
    x[2, 0, 5] = float("inf")
    x[3, 0, 70] = float("nan")
    x[4, 0, :2] = torch.tensor([3.0e38, -3.0e38])
    x[5, 0, 0] = 2.0 ** -130
    x[6, 0] = torch.arange(d) / 8.0
    x[7, 0] = (torch.arange(d) % 31) / 2.0 - 4.0          # half steps of the scale 1: ties
    x[8, 0] = (torch.arange(d) % 31) / 2.0 + 96.0         # the same far from zero
    x[9, 0] = torch.randn(d, generator=torch.Generator().manual_seed(2)) * 2.0 ** -120
    x[10, 0] = torch.randn(d, generator=torch.Generator().manual_seed(3)) * 2.0 ** 120
    x[11, 0, 3] = -float("inf")
    x[12, 0, 64:] = 1.0e-30
    x[12, 0, 100] = -100.0
    x[13:] = torch.from_numpy(np.round(rng.standard_normal((n - 13, 1, d)) * 8) / 8)
    k = x.to(BF).to(dev())
    v = k.flip(-1).contiguous()
    table = np.array([[1, 0]], dtype=np.int32)
    pool = np.zeros((2, 1, 16 * d * 9 // 8), dtype=np.uint8)
    got, ko, vo, status = run_append(k, v, pool, table, [n], [0, n], 16)
    assert status == 0
    assert np.array_equal(got, kv4.append(pool, f64(k), f64(v), table, [n], [0, n], 16))
    assert same_values(ko, kv4.values(*kv4.quantize(f64(k)))) and same_values(vo, kv4.values(*kv4.quantize(f64(v))))


def test_append_in_place(cuda_device):
    # the values written back over dense k and v
    rng = np.random.default_rng(23)
    new, Hkv, d, ps = [5, 40, 1], 3, 128, 16
    table, num_pages = layout(rng, new, ps)
    cu = np.concatenate([[0], np.cumsum(new)])
    k, v = (bf16(rng, (sum(new), Hkv, d)).to(dev()) for _ in range(2))
    pool = np.zeros((num_pages, Hkv, ps * d * 9 // 8), dtype=np.uint8)
    want, ko, vo, _ = run_append(k, v, pool, table, new, cu, ps)
    p, t, n, c = (torch.as_tensor(np.asarray(x, dtype=y)).to(dev()) for x, y in
                  ((pool, np.uint8), (table, np.int32), (new, np.int32), (cu, np.int32)))
    ab.attn_kv4_append(k, v, p, t, n, c, ps, k, v)
    assert ab.attn_get_device_status() == 0
    assert torch.equal(k, ko) and torch.equal(v, vo) and np.array_equal(p.cpu().numpy(), want)


def test_append_of_a_padded_batch(cuda_device):
    # 12 rows of k and v of which three sequences have 6; the rest is padding
    rng = np.random.default_rng(25)
    Hkv, d, ps = 2, 128, 16
    lens, cu = [17, 0, 4, 9], [0, 1, 1, 5, 6]
    table, num_pages = layout(rng, lens, ps)
    k, v = (bf16(rng, (12, Hkv, d)).to(dev()) for _ in range(2))
    k[6:], v[6:] = float("nan"), float("inf")
    pool = rng.integers(0, 256, (num_pages, Hkv, ps * d * 9 // 8), dtype=np.uint8)
    got, ko, vo, status = run_append(k, v, pool, table, lens, cu, ps)
    assert status == 0
    assert np.array_equal(got, kv4.append(pool, f64(k[:6]), f64(v[:6]), table, lens, cu, ps))
    assert same_values(ko[:6], kv4.values(*kv4.quantize(f64(k[:6])))) and same_values(vo[:6], kv4.values(*kv4.quantize(f64(v[:6]))))
    untouched = bf16_bits_of(torch.full((1,), float("nan"), dtype=BF))[0]
    assert (bf16_bits_of(ko[6:]) == untouched).all() and (bf16_bits_of(vo[6:]) == untouched).all()


def test_append_looks_at_no_page_of_a_row_without_new_tokens(cuda_device):
    rng = np.random.default_rng(24)
    Hkv, d, ps = 2, 64, 16
    table = np.array([[-1, -1], [0, 1], [-1, 7]], dtype=np.int32)  # rows 0 and 2 have lengths, but no pages yet
    lens, cu = [21, 18, 30], [0, 0, 3, 3]
    k, v = (bf16(rng, (3, Hkv, d)).to(dev()) for _ in range(2))
    pool = np.zeros((2, Hkv, ps * d * 9 // 8), dtype=np.uint8)
    got, _, _, status = run_append(k, v, pool, table, lens, cu, ps)
    assert status == 0
    assert np.array_equal(got, kv4.append(pool.copy(), f64(k), f64(v), table, lens, cu, ps))


def test_append_errors_are_latched_and_write_nothing(cuda_device):
    rng = np.random.default_rng(24)
    d, lens, cu = 64, [20, 9], [0, 20, 29]
    pool = rng.integers(0, 256, (4, 1, 16 * d * 9 // 8), dtype=np.uint8)
    k, v = (bf16(rng, (29, 1, d)).to(dev()) for _ in range(2))
    table = np.array([[0, 4], [1, -1]], dtype=np.int32)      # tokens 16..19 of row 0 point past the pool
    got, ko, _, status = run_append(k, v, pool, table, lens, cu, 16)
    assert status == 6
    ok = np.array([[0, 2], [1, -1]], dtype=np.int32)
    want = kv4.append(pool, f64(k), f64(v), ok, lens, cu, 16)
    assert np.array_equal(got[:2], want[:2]) and np.array_equal(got[2:], pool[2:])
    for bad_lens, bad_cu in (([20, 8], cu), ([20, 33], cu), ([-1, 9], cu)):
        got, _, _, status = run_append(k, v, pool, ok, bad_lens, bad_cu, 16)
        assert status == 1
        good = 1 if bad_lens[0] < 0 else 0
        page = ok[good, 0]
        assert np.array_equal(got[page], want[page])
        assert np.array_equal(np.delete(got, [page, 2], 0), np.delete(pool, [page, 2], 0))
    for bad_cu in ([0, 20, 30], [1, 20, 29], [0, 30, 29], [0, -5, 29]):
        got, _, _, status = run_append(k, v, pool, ok, lens, bad_cu, 16)
        assert status == 1


# ------------------------------------------------------------------ gather


@pytest.mark.parametrize("Hkv,d,ps,lens,N", [
    (1, 64, 16, [1], 1), (2, 128, 16, [33, 0, 16, 100], 100), (3, 128, 64, [65, 130], 80), (1, 256, 32, [47, 5], 64),
    (2, 64, 32, [70], 1000),
])
def test_gather_matches_oracle_and_leaves_the_rest(Hkv, d, ps, lens, N, cuda_device):
    rng = np.random.default_rng(d + N)
    table, num_pages = layout(rng, lens, ps)
    pool = random_pool(rng, num_pages, Hkv, ps, d)
    k = torch.full((len(lens), Hkv, N, d), 7.25, dtype=BF, device=dev())
    v = torch.full_like(k, -7.25)
    p, t, n = (torch.as_tensor(x).to(dev()) for x in (pool, table, np.asarray(lens, dtype=np.int32)))
    ab.attn_kv4_gather(p, t, n, ps, k, v)
    assert ab.attn_get_device_status() == 0
    K, V = kv4.pool_values(pool, ps, d)
    for i, ln in enumerate(lens):
        m = min(ln, N)
        pages = table[i][: -(-ln // ps)]
        for got, ref, rest in ((k, K, 7.25), (v, V, -7.25)):
            want = ref[pages].transpose(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :m]
            assert same_values(got[i, :, :m], want)
            assert (got[i, :, m:] == rest).all()


def test_gather_errors_are_latched(cuda_device):
    rng = np.random.default_rng(4)
    pool = torch.from_numpy(random_pool(rng, 3, 1, 16, 64)).to(dev())
    table = torch.tensor([[0, 9], [1, 2]], dtype=torch.int32, device=dev())
    k, v = (torch.zeros(2, 1, 32, 64, dtype=BF, device=dev()) for _ in range(2))
    ab.attn_kv4_gather(pool, table, torch.tensor([32, 32], dtype=torch.int32, device=dev()), 16, k, v)
    assert ab.attn_get_device_status() == 6
    assert (k[0, 0, 16:] == 0).all() and (k[0, 0, :16] != 0).any() and (k[1] != 0).any()
    k.zero_()
    ab.attn_kv4_gather(pool, table, torch.tensor([33, -1], dtype=torch.int32, device=dev()), 16, k, v)
    assert ab.attn_get_device_status() == 1 and (k == 0).all()


# ------------------------------------------------------------------ together, streams, graphs, far offsets


def test_pages_beyond_four_gigabytes(cuda_device):
    rng = np.random.default_rng(31)
    Hkv, d, ps = 8, 256, 64
    page = ab.attn_kv4_page_bytes(Hkv, ps, d)
    num_pages = (5 << 30) // page
    pool = torch.zeros((num_pages, Hkv, page // Hkv), dtype=torch.uint8, device=dev())
    lens, cu = [100, 70], [0, 100, 170]
    table = np.array([[num_pages - 1, 0], [num_pages - 3, num_pages - 2]], dtype=np.int32)
    k, v = (bf16(rng, (170, Hkv, d)).to(dev()) for _ in range(2))
    t, n, c = (torch.as_tensor(np.asarray(x, dtype=np.int32)).to(dev()) for x in (table, lens, cu))
    ab.attn_kv4_append(k, v, pool, t, n, c, ps)
    q = bf16(rng, (2, 16, d))
    small = np.stack([pool[p].cpu().numpy() for p in (num_pages - 1, 0, num_pages - 3, num_pages - 2)])
    near = np.array([[0, 1], [2, 3]], dtype=np.int32)
    want = kv4.append(np.zeros_like(small), f64(k), f64(v), near, lens, cu, ps)
    assert np.array_equal(small, want)
    o, lse, status = run_decode(q, pool, table, lens, ps, 0.06)
    assert status == 0
    check_decode(o, lse, q, small, near, lens, ps, 0.06)
    gk, gv = (torch.zeros((2, Hkv, 100, d), dtype=BF, device=dev()) for _ in range(2))
    ab.attn_kv4_gather(pool, t, n, ps, gk, gv)
    K, _ = kv4.pool_values(small, ps, d)
    assert same_values(gk[1, :, :70], K[near[1]].transpose(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :70])
    ws = torch.empty(ab.attn_pages_workspace_size(num_pages, 2), dtype=torch.uint8, device=dev())
    nt, nl = torch.empty((3, 2), dtype=torch.int32, device=dev()), torch.empty(3, dtype=torch.int32, device=dev())
    ab.attn_pages_fork(t, n, torch.tensor([0, 1, 1], dtype=torch.int32, device=dev()), None, nt, nl, ps, [pool], ws)
    assert ab.attn_get_device_status() == 0
    assert nt.tolist() == [[num_pages - 1, 0], [num_pages - 3, num_pages - 2], [num_pages - 3, 1]]
    assert torch.equal(pool[1], pool[num_pages - 2])
    pm = torch.empty(num_pages, dtype=torch.int32, device=dev())
    ab.attn_pages_compact(nt, nl, nt, pm, ps, [pool], ws)
    assert ab.attn_get_device_status() == 0
    assert nt.tolist() == [[4, 0], [2, 3], [2, 1]]
    assert np.array_equal(pool[[4, 0, 2, 3]].cpu().numpy(), small)


def serving_state(rng):
    """Two prompts in a 4-bit cache with room for their forks; K and V as the model computed them."""
    Hkv, d, ps, lens = 2, 128, 16, [77, 160]
    num_pages, cols = 64, 16
    table = np.full((2, cols), -1, dtype=np.int32)
    perm = rng.permutation(num_pages)
    table[0, :5], table[1, :10] = perm[:5], perm[5:15]
    st = dict(Hkv=Hkv, d=d, ps=ps, lens=lens, cu=[0, 77, 237], num_pages=num_pages)
    st["k"], st["v"] = (bf16(rng, (237, Hkv, d)).to(dev()) for _ in range(2))
    st["pool"] = torch.full((num_pages, Hkv, ps * d * 9 // 8), 0xFF, dtype=torch.uint8, device=dev())
    st["table"] = torch.from_numpy(table).to(dev())
    for name, x in (("n", lens), ("c", st["cu"]), ("parents", [1, 0, 1, 0]), ("add", [1, 1, 1, 1]), ("c4", [0, 1, 2, 3, 4])):
        st[name] = torch.tensor(x, dtype=torch.int32, device=dev())
    st["k1"], st["v1"] = (bf16(rng, (4, Hkv, d)).to(dev()) for _ in range(2))
    st["q1"] = bf16(rng, (4, 8, d)).to(dev())
    st["o"] = torch.empty((4, 8, d), dtype=BF, device=dev())
    st["lse"] = torch.empty((4, 8), dtype=torch.float32, device=dev())
    st["nt"] = torch.empty((4, cols), dtype=torch.int32, device=dev())
    st["nl"] = torch.empty(4, dtype=torch.int32, device=dev())
    st["ct"] = torch.empty((4, cols), dtype=torch.int32, device=dev())
    st["pm"] = torch.empty(num_pages, dtype=torch.int32, device=dev())
    st["ko"], st["vo"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
    st["gk"], st["gv"] = (torch.zeros((4, Hkv, 161, d), dtype=BF, device=dev()) for _ in range(2))
    st["ws"] = torch.empty(ab.attn_decode_paged_kv4_workspace_size(4, 8, Hkv, d), dtype=torch.uint8, device=dev())
    st["pws"] = torch.empty(ab.attn_pages_workspace_size(num_pages, 4), dtype=torch.uint8, device=dev())
    return st


def serve(s, scale, stream=None):
    """Prompts in, fork each in two, one token more for all, decode, compact, read back."""
    ab.attn_kv4_append(s["k"], s["v"], s["pool"], s["table"], s["n"], s["c"], s["ps"], s["ko"], s["vo"], stream=stream)
    ab.attn_pages_fork(s["table"], s["n"], s["parents"], s["add"], s["nt"], s["nl"], s["ps"], [s["pool"]], s["pws"],
                       stream=stream)
    ab.attn_kv4_append(s["k1"], s["v1"], s["pool"], s["nt"], s["nl"], s["c4"], s["ps"], stream=stream)
    ab.attn_decode_paged_kv4(s["q1"], s["pool"], s["nt"], s["nl"], s["ps"], s["o"], s["lse"], scale, s["ws"],
                             stream=stream)
    ab.attn_pages_compact(s["nt"], s["nl"], s["ct"], s["pm"], s["ps"], [s["pool"]], s["pws"], stream=stream)
    ab.attn_kv4_gather(s["pool"], s["ct"], s["nl"], s["ps"], s["gk"], s["gv"], stream=stream)
    return [s[x].clone() for x in ("o", "lse", "nt", "nl", "ct", "pm", "pool", "gk", "gv", "ko", "vo")]


def test_serving_run_matches_oracle_and_prefill(cuda_device):
    rng = np.random.default_rng(41)
    s = serving_state(rng)
    scale = 1.0 / math.sqrt(s["d"])
    serve(s, scale)
    assert ab.attn_get_device_status() == 0
    assert s["nl"].tolist() == [161, 78, 161, 78]
    # the exact attention of the quantized keys and values each row has seen
    k, v, k1, v1, q1 = (f64(s[x]) for x in ("k", "v", "k1", "v1", "q1"))
    for i, p in enumerate([1, 0, 1, 0]):
        lo, hi = s["cu"][p], s["cu"][p + 1]
        K = kv4.values(*kv4.quantize(np.concatenate([k[lo:hi], k1[i:i + 1]]))).transpose(1, 0, 2)
        V = kv4.values(*kv4.quantize(np.concatenate([v[lo:hi], v1[i:i + 1]]))).transpose(1, 0, 2)
        n = hi - lo + 1
        assert same_values(s["gk"][i, :, :n], K) and same_values(s["gv"][i, :, :n], V)
        ref_o, ref_l = attention(q1[i][None, :, None], K[None], V[None], scale, False)
        # 2^-11 on each probability times a centred code of at most 8 steps of at most 0.5, and the bf16 output
        assert np.all(np.abs(f64(s["o"][i]) - ref_o[0, :, 0]) <= 2.0 ** -11 * 4 + 2.0 ** -8 * np.abs(ref_o[0, :, 0]) + 1e-4)
        assert np.all(np.abs(f64(s["lse"][i]) - ref_l[0, :, 0]) <= 1e-4)
        # prefill attention on the gathered context: its last row is this step (K and V rounded to bf16)
        Q = torch.zeros((1, 8, 1, s["d"]), dtype=BF, device=dev())
        Q[0, :, 0] = s["q1"][i]
        fo, fl = torch.empty_like(Q), torch.empty((1, 8, 1), dtype=torch.float32, device=dev())
        ab.attn_fwd(Q, s["gk"][i:i + 1, :, :n].contiguous(), s["gv"][i:i + 1, :, :n].contiguous(), fo, fl, True, scale)
        assert ab.attn_get_device_status() == 0
        assert (fo[0, :, 0].float() - s["o"][i].float()).abs().max() <= 3e-2
        assert (fl[0, :, 0] - s["lse"][i]).abs().max() <= 2e-2
    assert same_values(s["ko"], kv4.values(*kv4.quantize(k)))


def test_serving_run_in_a_graph_and_on_another_stream(cuda_device):
    s = serving_state(np.random.default_rng(42))
    pool0 = s["pool"].clone()
    eager = serve(s, 0.09)
    assert ab.attn_get_device_status() == 0
    names = ("o", "lse", "nt", "nl", "ct", "pm", "gk", "gv", "ko", "vo")

    def wipe():
        torch.cuda.synchronize()
        s["pool"].copy_(pool0)
        for x in names:
            s[x].zero_()
        for x in ("ws", "pws"):
            s[x].fill_(0xA5)
        torch.cuda.synchronize()

    def same():
        torch.cuda.synchronize()
        assert ab.attn_get_device_status() == 0
        for a, b in zip(eager, [s[x] for x in ("o", "lse", "nt", "nl", "ct", "pm", "pool", "gk", "gv", "ko", "vo")]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))

    side = torch.cuda.Stream()
    wipe()
    serve(s, 0.09, stream=side)
    side.synchronize()
    same()
    wipe()
    with torch.cuda.stream(side):
        serve(s, 0.09)
    side.synchronize()
    same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        serve(s, 0.09)
    for _ in range(2):
        wipe()
        g.replay()
        same()
    del g


@pytest.mark.parametrize("wide", [False, True])
def test_two_decodes_in_flight(wide, cuda_device):
    rng = np.random.default_rng(43)
    lens = [900, 1700]
    table, num_pages = layout(rng, lens, 16)
    table = widen(table, 16) if wide else table
    pool = random_pool(rng, num_pages, 2, 16, 128)
    q = [bf16(rng, (2, 8, 128)) for _ in range(2)]
    want = [run_decode(x, pool, table, lens, 16, 0.09)[:2] for x in q]
    p, t, n = (torch.as_tensor(x).to(dev()) for x in (pool, table, np.asarray(lens, dtype=np.int32)))
    qd = [x.to(dev()) for x in q]
    out = [(torch.empty((2, 8, 128), dtype=BF, device=dev()), torch.empty((2, 8), dtype=torch.float32, device=dev()))
           for _ in q]
    ws = [torch.empty(ab.attn_decode_paged_kv4_workspace_size(2, 8, 2, 128), dtype=torch.uint8, device=dev()) for _ in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            ab.attn_decode_paged_kv4(qd[i], p, t, n, 16, *out[i], 0.09, ws[i], stream=st)
    torch.cuda.synchronize()
    assert ab.attn_get_device_status() == 0
    for (o, lse), (ro, rl) in zip(out, want):
        assert torch.equal(o, ro) and torch.equal(lse, rl)


def test_binding_refusals(cuda_device):
    pool = torch.zeros(4, 2, 16 * 128 * 9 // 8, dtype=torch.uint8, device=dev())
    table = torch.zeros(1, 2, dtype=torch.int32, device=dev())
    n = torch.ones(1, dtype=torch.int32, device=dev())
    cu = torch.tensor([0, 1], dtype=torch.int32, device=dev())
    k = torch.zeros(1, 2, 128, dtype=BF, device=dev())
    q = torch.zeros(1, 4, 128, dtype=BF, device=dev())
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=dev())
    lse = torch.empty(1, 4, dtype=torch.float32, device=dev())
    bad = [
        lambda: ab.attn_kv4_append(k, k[:, :1], pool, table, n, cu, 16),
        lambda: ab.attn_kv4_append(k.transpose(1, 2).contiguous().transpose(1, 2), k, pool, table, n, cu, 16),
        lambda: ab.attn_kv4_append(k, k, pool, table, n, cu[:1], 16),
        lambda: ab.attn_kv4_append(k, k, pool, table, n, cu, 32),
        lambda: ab.attn_kv4_append(k, k, pool[:, :1].contiguous(), table, n, cu, 16),
        lambda: ab.attn_kv4_append(k, k, pool, table, n, cu, 16, k[..., :64].contiguous()),
        lambda: ab.attn_decode_paged_kv4(q, pool, table.repeat(2, 1), n.repeat(2), 16, q, lse, 0.1, ws),
        lambda: ab.attn_decode_paged_kv4(q, pool, table, n, 16, q[:, :2].contiguous(), lse, 0.1, ws),
        lambda: ab.attn_decode_paged_kv4(q, pool, table, n, 16, q, lse[:, :2].contiguous(), 0.1, ws),
        lambda: ab.attn_kv4_gather(pool, table, n, 16, k[None], k[None]),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ab.AttnError):
        ab.attn_decode_paged_kv4(q, pool, table, n, 16, q, lse, 0.1, ws[:256])
    with pytest.raises(ab.AttnError):
        ab.attn_decode_paged_kv4(q, pool, table, n, 16, q, lse, -0.1, ws)
    assert ab.attn_get_device_status() == 0


def test_tensors_of_another_device_are_refused(cuda_device, monkeypatch):
    # with another device current, the kernels would run there on this device's addresses
    pool = torch.zeros(4, 2, 16 * 64 * 9 // 8, dtype=torch.uint8, device=dev())
    table, n = torch.zeros(1, 2, dtype=torch.int32, device=dev()), torch.ones(1, dtype=torch.int32, device=dev())
    cu = torch.tensor([0, 1], dtype=torch.int32, device=dev())
    k, q = (torch.zeros(1, h, 64, dtype=BF, device=dev()) for h in (2, 4))
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=dev())
    pm = torch.zeros(4, dtype=torch.int32, device=dev())
    calls = [
        lambda: ab.attn_kv4_append(k, k, pool, table, n, cu, 16),
        lambda: ab.attn_kv4_gather(pool, table, n, 16, k[None].transpose(1, 2).contiguous(), k[None].transpose(1, 2).contiguous()),
        lambda: ab.attn_decode_paged_kv4(q, pool, table, n, 16, torch.empty_like(q), None, 0.1, ws),
        lambda: ab.attn_pages_fork(table, n, torch.zeros_like(n), None, torch.empty_like(table), torch.empty_like(n), 16,
                                   [pool], ws),
        lambda: ab.attn_pages_compact(table, n, torch.empty_like(table), pm, 16, [pool], ws),
    ]
    for call in calls:
        call()
    assert ab.attn_get_device_status() == 0
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("wide", [False, True])
def test_decode_does_not_depend_on_what_shared_memory_held(wide, cuda_device):
    # rows that end inside a unit of two records, after calls on other data left their records behind
    rng = np.random.default_rng(44)
    lens = [5, 16, 17, 31, 33, 200, 1000]
    table, num_pages = layout(rng, lens, 16)
    table = widen(table, 16) if wide else table
    pool = random_pool(rng, num_pages, 2, 16, 128)
    q = bf16(rng, (len(lens), 8, 128))
    o0, l0, _ = run_decode(q, pool, table, lens, 16, 0.09)
    big_table, big_pages = layout(rng, [20000] * 4, 16)
    for s_hi in (1e-3, 30.0, 3e4):
        other = random_pool(rng, big_pages, 2, 16, 128, s_lo=s_hi / 2, s_hi=s_hi)
        run_decode(bf16(rng, (4, 8, 128)), other, big_table, [20000] * 4, 16, 0.09)
        o, lse, _ = run_decode(q, pool, table, lens, 16, 0.09)
        assert torch.equal(o, o0) and torch.equal(lse, l0)
