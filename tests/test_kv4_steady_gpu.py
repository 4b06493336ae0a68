"""The 4-bit cache at sizes where a warp works long: decode ranges of many units (the record list is refilled every
16 units, segments end anywhere in it) and appends whose warps take several KV heads in turn.

Decode bounds, as in test_kv4_weights_gpu.py, with the sums' errors counted by their depth.  A warp's range has at most
U units and a row at most np partials.  The sum of exponentials passes U + 2 additions in a lane, 3 between lanes
and np + 4 in the merge, each 2^-24 of it.  A product is added up in 2 U tensor-core steps of 16 products (17 additions
of at most 2^-23 each) and the merge's np + 4: U 34 * 2^-23 + (np + 4) 2^-24; so is the sum of V's minima, with 4 U.
"""

import math

import numpy as np
import pytest
import torch

import attn_fwd_05_b200 as ab
from oracle import kv4
from test_kv4_gpu import BF, bf16, dev, f64, same_values

pytestmark = pytest.mark.gpu
UNIT, SEG_COST, MIN_UNITS, WARPS = 32, 2, 2, 4


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------ decode


def ranges(lens, Hq, Hkv, d, capacity):
    """Per warp of the two-launch form: the units (segment, place, units in it) of its range, by the cost rule."""
    group = Hq // Hkv
    nt = 2 if group > 8 and d <= 128 else 1
    c = Hkv * -(-group // (8 * nt))
    resident = sms() * (4 if d * nt <= 64 else (3 if d * nt <= 128 else 2))
    most = -(-capacity // UNIT)
    warps = max(1, min(-(-len(lens) * most * c // (WARPS * MIN_UNITS)), resident)) * WARPS
    units = np.repeat([-(-n // UNIT) for n in lens], c)
    units = units[units > 0]
    start = np.concatenate([[0], np.cumsum(units + SEG_COST)])
    per = max(-(-int(start[-1]) // warps), MIN_UNITS)
    out = []
    first = np.concatenate([[0], np.cumsum(units)])

    def unit_at(f):  # units before cost f
        if f >= start[-1]:
            return int(first[-1])
        seg = int(np.searchsorted(start, f, side="right")) - 1
        return int(first[seg]) + max(0, int(f - start[seg]) - SEG_COST)

    for w in range(warps):
        lo, hi = unit_at(w * per), unit_at((w + 1) * per)
        ends = first[1:][(first[1:] > lo) & (first[1:] < hi)] - lo  # units of the range before each new segment
        out.append((hi - lo, ends))
    return out


def gpu_pool(seed, num_pages, Hkv, page_size, d):
    """Random codes; scales in [0.05, 0.35), minima about 7.5 steps below zero."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    ng = d // 64
    pool = torch.randint(0, 256, (num_pages, Hkv, page_size // 16, kv4.record_bytes(d)), generator=g, device=dev(),
                         dtype=torch.uint8)
    par = pool[..., 1024 * ng:].view(BF)
    s = 0.05 + 0.3 * torch.rand((*par.shape[:-1], 32 * ng), generator=g, device=dev())
    par[..., 0::2] = s.to(BF)
    par[..., 1::2] = (-7.5 * s + s * torch.randn(s.shape, generator=g, device=dev())).to(BF)
    return pool.view(num_pages, Hkv, -1)


class Exact:
    """K, V and their parameters of a row and KV head, fp64 on the device, by the format's tables."""

    def __init__(self, pool, table, page_size, d):
        (kb, ks), (vb, vs) = kv4.places(d)[0]
        self.codes = [(torch.from_numpy(b).to(dev()), torch.from_numpy(s.astype(np.uint8)).to(dev()))
                      for b, s in ((kb, ks), (vb, vs))]
        self.par = [torch.from_numpy(p // 2).to(dev()) for p in kv4.places(d)[1]]
        self.pool, self.table, self.page_size, self.d = pool, table, page_size, d

    def row(self, i, h, n):
        pages = torch.as_tensor(self.table[i][: -(-n // self.page_size)]).long().clamp(0, self.pool.shape[0] - 1).to(dev())
        rec = self.pool[pages, h].reshape(-1, kv4.record_bytes(self.d))
        words = rec.view(BF)
        out = []
        for (byte, shift), at in zip(self.codes, self.par):
            c = ((rec[:, byte] >> shift) & 15).double().reshape(-1, self.d)[:n]
            s = words[:, at].double().reshape(-1, self.d // 64)[:n]
            m = words[:, at + 1].double().reshape(-1, self.d // 64)[:n]
            out.append((c * s.repeat_interleave(64, 1) + m.repeat_interleave(64, 1), s, m))
        return out


def check(o, lse, q, pool, table, lens, page_size, scale, longest, there):
    """Every row and head.  there(i, n): which tokens of row i take part."""
    S, Hq, d = q.shape
    Hkv = pool.shape[1]
    group = Hq // Hkv
    exact = Exact(pool, table, page_size, d)
    q, o, lse = q.double().to(dev()), o.double(), lse.double()
    worst = torch.zeros(2, dtype=torch.float64, device=dev())
    for i, n in enumerate(lens):
        if n == 0:
            assert (o[i] == 0).all() and torch.isneginf(lse[i]).all()
            continue
        depth = longest + -(-n // UNIT // max(1, longest // 2)) + 8
        el, eo = depth * 2.0 ** -24, (34 * longest * 2 + depth) * 2.0 ** -24
        out = ~torch.as_tensor(there(i, n)).to(dev())
        for h in range(Hkv):
            hq = slice(h * group, (h + 1) * group)
            (K, ks, km), (V, vs, vm) = exact.row(i, h, n)
            x = (q[i, hq] @ K.T) * scale
            x[:, out] = -math.inf
            ref_l = torch.logsumexp(x, -1)
            w = torch.exp(x - ref_l[:, None])
            ref = w @ V
            e = 68 * 2.0 ** -24 * scale * (q[i, hq].abs().reshape(group, -1, 64).sum(-1) @ (8 * ks + (km + 8 * ks).abs()).T)
            a = (vm + 8 * vs).abs() + 8 * vs
            A, we = w @ a, (w * e).sum(-1)
            tol = 8 * (2.0 ** -11 * (w @ vs) + n * 2.0 ** -25 * (w[:, :, None] * vs).amax(1)) + (w * e) @ a + we[:, None] * A \
                + 2 * (2.0 ** -22 + eo) * A
            tol = tol.repeat_interleave(64, 1) + 2.0 ** -8 * ref.abs()
            worst[0] = torch.maximum(worst[0], ((o[i, hq] - ref).abs() / tol).nan_to_num(math.inf).max())
            tol_l = we + el + 2.0 ** -22 * ref_l.abs() + 2.0 ** -21
            worst[1] = torch.maximum(worst[1], ((lse[i, hq] - ref_l).abs() / tol_l).nan_to_num(math.inf).max())
    assert (worst <= 1).all(), f"{worst.tolist()} of the tolerances of o and lse"


FORMS = [  # Hq, Hkv, d, page_size, tokens of the long rows
    (16, 16, 64, 32, 16000), (96, 8, 64, 16, 20000), (64, 8, 128, 16, 20000), (128, 8, 128, 64, 14000),
    (80, 4, 128, 16, 14000), (32, 8, 256, 16, 14000),
]


@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,ps,n_long", FORMS)
def test_decode_of_long_ranges(Hq, Hkv, d, ps, n_long, bad, cuda_device):
    rng = np.random.default_rng(Hq + d)
    lens = [int(x) for x in rng.integers(n_long // 2, n_long, 18)] + [int(x) for x in rng.integers(1, 1300, 90)] + [0] * 20
    lens = [lens[i] for i in rng.permutation(len(lens))]
    need = [-(-n // ps) for n in lens]
    cols, num_pages = max(need), sum(need) + 3
    table = np.full((len(lens), cols), -1, dtype=np.int32)
    perm, at = rng.permutation(num_pages), 0
    for i, n in enumerate(need):
        table[i, :n], at = perm[at:at + n], at + n
    # what the split of this batch covers: long ranges, and segments that end just before, at and just after a refill
    plan = ranges(lens, Hq, Hkv, d, cols * ps)
    longest = max(n for n, _ in plan)
    ends = {int(e) % 16 for _, es in plan for e in es if e >= 15}
    assert longest > 32 and {15, 0, 1} <= ends and sum(n for n, _ in plan) == sum(-(-n // UNIT) for n in lens) * (
        Hkv * -(-(Hq // Hkv) // (16 if Hq // Hkv > 8 and d <= 128 else 8)))
    pool = gpu_pool(d, num_pages, Hkv, ps, d)
    used = table.copy()
    gone = [np.zeros(n, dtype=bool) for n in lens]
    if bad:  # pages out of range far into the long rows, and in a unit of its own of some short ones
        for i, n in enumerate(lens):
            for page in {600 // ps, 1111 // ps, (n - 1) // ps // 2} if n > 1200 else ({n // ps // 2} if i % 5 == 0 and n else ()):
                used[i, page] = (-1, num_pages, 1 << 30)[i % 3]
                gone[i][page * ps:(page + 1) * ps] = True
    q = bf16(rng, (len(lens), Hq, d))
    scale = 1.0 / math.sqrt(d)
    o = torch.full((len(lens), Hq, d), float("nan"), dtype=BF, device=dev())
    lse = torch.full((len(lens), Hq), float("nan"), dtype=torch.float32, device=dev())
    ws = torch.full((ab.attn_decode_paged_kv4_workspace_size(len(lens), Hq, Hkv, d),), 0xFF, dtype=torch.uint8, device=dev())
    t, n = torch.from_numpy(used).to(dev()), torch.tensor(lens, dtype=torch.int32, device=dev())
    for _ in range(2):
        ab.attn_decode_paged_kv4(q.to(dev()), pool, t, n, ps, o, lse, scale, ws)
        assert ab.attn_get_device_status() == (6 if bad else 0)
    short = [i for i, n in enumerate(lens) if n and gone[i].all()]
    assert all((o[i] == 0).all() and torch.isneginf(lse[i]).all() for i in short)
    check(o, lse, q, pool, table, [0 if i in short else n for i, n in enumerate(lens)], ps, scale, longest,
          lambda i, n: ~gone[i])


# ------------------------------------------------------------------ append


def appended(pool, k, v, table, lens, cu, page_size):
    """The pool after an append, byte for byte, all tokens at once (k and v fp64 [T, Hkv, d])."""
    T, H, d = k.shape
    new = np.diff(cu)
    row = np.repeat(np.arange(len(lens)), new)
    pos = np.asarray(lens)[row] - np.asarray(cu)[row + 1] + np.arange(T)
    page, blk, tok = table[row, pos // page_size], pos % page_size // 16, pos % 16
    rec = pool.reshape(*pool.shape[:2], page_size // 16, -1)
    nib = np.stack((rec & 15, rec >> 4), -1).reshape(*rec.shape[:-1], -1)
    heads = np.arange(H)[None, :, None]
    sm = []
    for is_v, x in ((0, k), (1, v)):
        codes, s, m = kv4.quantize(x)
        byte, shift = kv4.places(d)[0][is_v]
        place = (2 * byte + shift // 4)[tok]
        nib[page[:, None, None], heads, blk[:, None, None], place[:, None, :]] = codes
        sm.append((s, m))
    out = (nib[..., 0::2] | nib[..., 1::2] << 4).astype(np.uint8)
    words = out.view(np.uint16)
    for is_v, (s, m) in enumerate(sm):
        place = (kv4.places(d)[1][is_v] // 2)[tok]
        for off, x in ((0, s), (1, m)):
            words[page[:, None, None], heads, blk[:, None, None], place[:, None, :] + off] = x
    return out.reshape(pool.shape)


@pytest.mark.parametrize("how", ["fused", "dense", "in place"])
@pytest.mark.parametrize("Hkv,d,ps,tokens,heads", [
    (3, 64, 16, 20000, 2), (5, 128, 32, 12500, 2), (5, 128, 16, 18500, 3), (5, 64, 64, 24500, 4), (3, 256, 16, 20000, 2),
])
def test_append_of_several_heads_a_warp(Hkv, d, ps, tokens, heads, how, cuda_device):
    rng = np.random.default_rng(tokens + d)
    cut = np.sort(rng.integers(0, tokens, 6))
    new = np.diff(np.concatenate([[0], cut, [tokens]]))
    new = np.insert(new, 3, 0)  # a row without new tokens
    past = rng.integers(0, 70, len(new))
    lens, cu = [int(x) for x in past + new], np.concatenate([[0], np.cumsum(new)])
    quads = tokens // 4 + 2 * len(new)
    assert min(Hkv, quads * Hkv // (48 * sms())) == heads or sms() != 148
    need = [-(-n // ps) for n in lens]
    num_pages = sum(need) + 2
    table = np.full((len(lens), max(need)), -1, dtype=np.int32)
    perm, at = rng.permutation(num_pages), 0
    for i, n in enumerate(need):
        table[i, :n], at = perm[at:at + n], at + n
    g = torch.Generator(device=dev()).manual_seed(tokens)
    x = torch.randn((tokens, 3, Hkv, d), generator=g, device=dev())
    x[:, 1] += 3 * torch.randn((Hkv, d), generator=g, device=dev())
    x = x.to(BF)
    k, v = (x[:, 1], x[:, 2]) if how == "fused" else (x[:, 1].contiguous(), x[:, 2].contiguous())
    k64, v64 = f64(k), f64(v)
    pool = rng.integers(0, 256, (num_pages, Hkv, ps * d * 9 // 8), dtype=np.uint8)
    p, t, n, c = (torch.as_tensor(np.asarray(a)).to(dev()) for a in
                  (pool, table, np.asarray(lens, dtype=np.int32), cu.astype(np.int32)))
    ko, vo = (k, v) if how == "in place" else (torch.full((tokens, Hkv, d), float("nan"), dtype=BF, device=dev()) for _ in range(2))
    ab.attn_kv4_append(k, v, p, t, n, c, ps, ko, vo)
    assert ab.attn_get_device_status() == 0
    want = appended(pool, k64, v64, table, lens, cu, ps)
    assert np.array_equal(p.cpu().numpy(), want)
    assert same_values(ko, kv4.values(*kv4.quantize(k64))) and same_values(vo, kv4.values(*kv4.quantize(v64)))


def test_the_pool_of_all_tokens_at_once_is_the_oracle_s(cuda_device):
    rng = np.random.default_rng(61)
    lens, cu, table = [20, 5, 9], [0, 7, 7, 16], np.array([[2, 0], [-1, -1], [1, -1]], dtype=np.int32)
    pool = rng.integers(0, 256, (3, 2, 16 * 128 * 9 // 8), dtype=np.uint8)
    k, v = (f64(bf16(rng, (16, 2, 128))) for _ in range(2))
    assert np.array_equal(appended(pool, k, v, table, lens, cu, 16), kv4.append(pool, k, v, table, lens, cu, 16))
