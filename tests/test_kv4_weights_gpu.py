"""Decode over the 4-bit cache where tokens of very different V scales and weights meet, and at the ends of
the range of queries, keys and scales.  The bounds follow the weights: a token that takes no part in a
row's result must not cost the others their bits.

Per output element, from the roundings the kernel makes (w_j: the row's softmax weights, s_j: V's scale):
* w_j s_j is rounded to fp16, 2^-11 of it, or 2^-25 of a power of two that is at most the largest such
  product of its run, and multiplies a centred code of at most 8 in magnitude:
      8 (2^-11 sum_j w_j s_j + n 2^-25 max_j w_j s_j);
* bf16 output: 2^-8 of the value;
* scores: exact products, fp32 sums over 64 channels and four more roundings:
      E_j = 68 * 2^-24 * scale * sum_c |q_c| (8 s + |m + 8 s|)_jc.
  With A_j = |m + 8 s|_j + 8 s_j (at least |V_j|, and what the two sums add up) and A = sum_j w_j A_j an error E_j
  moves the numerator by w_j E_j A_j and, through the denominator, the result by w_j E_j A; the
  exponential's 2^-22 and fp32 sums (n * 2^-24) move both sums, 2 (2^-22 + n * 2^-24) A;
* log-sum-exp: sum_j w_j E_j, n * 2^-24 for the sum, 2^-22 of its own value and 2^-21 for the logarithm.
"""

import math

import numpy as np
import pytest

from oracle import kv4
from test_kv4_gpu import BF, bf16, f64, layout, random_pool, run_decode, widen

pytestmark = pytest.mark.gpu


def params(pool, page_size, d, is_v):
    """s and m, fp64 [num_pages, Hkv, page_size, d / 64]."""
    at = kv4.places(d)[1][int(is_v)]
    words = pool.reshape(*pool.shape[:2], page_size // 16, -1).view(np.uint16)
    return [kv4.bf16_value(words[..., at // 2 + i]).reshape(*pool.shape[:2], page_size, -1) for i in (0, 1)]


def set_params(pool, page_size, d, is_v, table_row, tokens, s=None, m=None, factor=None):
    """Sets (or multiplies by a power of two) the parameters of tokens of a row, all heads and groups."""
    words = pool.reshape(*pool.shape[:2], page_size // 16, -1).view(np.uint16)
    for t in tokens:
        for at in kv4.places(d)[1][int(is_v)][t % 16]:
            for off, x in ((0, s), (1, m)):
                w = words[table_row[t // page_size], :, t % page_size // 16, at // 2 + off]
                if factor is not None:
                    x = kv4.bf16_value(w) * factor
                if x is not None:
                    words[table_row[t // page_size], :, t % page_size // 16, at // 2 + off] = kv4.bf16_bits(
                        np.asarray(x, dtype=np.float32))


def check_weighted(o, lse, q, pool, table, lens, page_size, scale):
    o, lse, qf = f64(o), f64(lse), f64(q)
    S, Hq, d = qf.shape
    group = Hq // pool.shape[1]
    K, V = kv4.pool_values(pool, page_size, d)
    (ks, km), (vs, vm) = params(pool, page_size, d, False), params(pool, page_size, d, True)
    worst = 0.0
    for i, n in enumerate(lens):
        pages = table[i][: -(-n // page_size)]
        for h in range(Hq):
            cut = lambda x: x[pages, h // group].reshape(-1, x.shape[-1])[:n]  # noqa: E731
            x = (cut(K) @ qf[i, h]) * scale
            ref_l = x.max() + math.log(np.exp(x - x.max()).sum())
            w = np.exp(x - ref_l)[:, None]
            ref = (w * cut(V)).sum(0)
            ws = np.repeat(w * cut(vs), 64, 1)
            mid = 8 * cut(ks) + np.abs(cut(km) + 8 * cut(ks))
            e = 68 * 2.0 ** -24 * scale * (mid * np.abs(qf[i, h]).reshape(-1, 64).sum(-1)).sum(-1, keepdims=True)
            a = np.repeat(np.abs(cut(vm) + 8 * cut(vs)) + 8 * cut(vs), 64, 1)
            A, we = (w * a).sum(0), float((w * e).sum())
            tol = 8 * (2.0 ** -11 * ws.sum(0) + n * 2.0 ** -25 * ws.max(0)) + 2.0 ** -8 * np.abs(ref) \
                + (w * e * a).sum(0) + we * A + 2 * (2.0 ** -22 + n * 2.0 ** -24) * A
            err = np.abs(o[i, h] - ref)
            assert np.all(err <= tol), f"row {i} head {h}: {np.nanmax(err / tol):.2f} of the tolerance, {np.isnan(err).sum()} NaN"
            worst = max(worst, float((err / tol).max()))
            le = abs(lse[i, h] - ref_l)
            assert le <= we + n * 2.0 ** -24 + 2.0 ** -22 * abs(ref_l) + 2.0 ** -21, f"row {i} head {h}: lse off by {le:.2e}"
    return worst


FORMS = [  # Hq, Hkv, d, page_size
    (4, 2, 64, 16), (16, 1, 64, 32), (8, 2, 128, 16), (16, 1, 128, 16), (4, 1, 256, 64),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,ps", FORMS)
@pytest.mark.parametrize("r", [18, 24, 30])
@pytest.mark.parametrize("where", ["first", "last", "second unit", "units before"])
def test_a_light_token_with_a_large_scale_costs_the_others_nothing(where, r, Hq, Hkv, d, ps, wide, cuda_device):
    # Two units (64 tokens) carry the weight.  Tokens among or before them have 2^r times the V scale; for the even
    # heads about 2^-(r + 20) of the weight, for the odd heads (the queries' signs turned) nearly all of it.
    rng = np.random.default_rng(r + d + Hq)
    lens = [2048, 1990]
    heavy = range(32, 64) if where == "units before" else range(64)
    large = {"first": [0], "last": [31], "second unit": [40], "units before": range(32)}[where]
    table, num_pages = layout(rng, lens, ps)
    pool = random_pool(rng, num_pages, Hkv, ps, d)
    q = bf16(rng, (2, Hq, d)).abs() + 0.25
    q[:, 1::2] *= -1
    scale = 1.0 / math.sqrt(d)
    drop = (r + 20) * math.log(2) / (scale * float(q[:, 0::2].float().sum(-1).mean()))  # in every channel of K
    for i, n in enumerate(lens):
        set_params(pool, ps, d, False, table[i], range(n), s=0.0, m=-drop)
        set_params(pool, ps, d, False, table[i], heavy, m=0.0)
        set_params(pool, ps, d, False, table[i], large, m=-drop)
        set_params(pool, ps, d, True, table[i], large, factor=2.0 ** r)
    o, lse, status = run_decode(q, pool, widen(table, ps) if wide else table, lens, ps, scale)
    assert status == 0
    check_weighted(o, lse, q, pool, table, lens, ps, scale)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,ps", FORMS)
def test_scales_and_weights_that_run_against_one_another(Hq, Hkv, d, ps, wide, cuda_device):
    # along the row V's scale falls by 2^-1 every 16 tokens and the weight rises by 2^1 (even heads) or falls by
    # 2^-1 (odd heads), there and back every 512 tokens
    rng = np.random.default_rng(d + Hq)
    lens = [1500, 777]
    table, num_pages = layout(rng, lens, ps)
    pool = random_pool(rng, num_pages, Hkv, ps, d)
    q = bf16(rng, (2, Hq, d)).abs() + 0.25
    q[:, 1::2] *= -1
    scale = 1.0 / math.sqrt(d)
    step = math.log(2) / (scale * float(q[:, 0::2].float().sum(-1).mean()))
    for i, n in enumerate(lens):
        for t in range(n):
            k = t % 512 // 16 if t // 512 % 2 == 0 else 32 - t % 512 // 16
            set_params(pool, ps, d, False, table[i], [t], s=0.0, m=step * k)
            set_params(pool, ps, d, True, table[i], [t], factor=2.0 ** -k)
    o, lse, status = run_decode(q, pool, widen(table, ps) if wide else table, lens, ps, scale)
    assert status == 0
    check_weighted(o, lse, q, pool, table, lens, ps, scale)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,ps", FORMS)
@pytest.mark.parametrize("scale", [1e-13, 1e-30, 1e-44])
def test_zero_and_tiny_queries_at_a_tiny_scale(scale, Hq, Hkv, d, ps, wide, cuda_device):
    # scores of 0: the mean of V, in rows that end inside a unit
    rng = np.random.default_rng(d)
    lens = [45, 700, 1]
    table, num_pages = layout(rng, lens, ps)
    pool = random_pool(rng, num_pages, Hkv, ps, d)
    q = bf16(rng, (3, Hq, d))
    q[:, 0] = 0
    q[:, 1] *= 2.0 ** -110
    o, lse, status = run_decode(q, pool, widen(table, ps) if wide else table, lens, ps, scale)
    assert status == 0
    check_weighted(o, lse, q, pool, table, lens, ps, scale)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,ps", FORMS)
@pytest.mark.parametrize("q_exp,k_exp,scale_exp", [
    (0, 112, -112),     # products of the unscaled query reach 2^124
    (0, 112, -120), (-100, 112, -12), (100, 10, -110),
    (120, -120, 0),
    (125, -121, 5),     # the scale times the largest query is past fp32
])
def test_far_queries_keys_and_scales(q_exp, k_exp, scale_exp, Hq, Hkv, d, ps, wide, cuda_device):
    rng = np.random.default_rng(abs(d + k_exp))
    lens = [600, 33]
    table, num_pages = layout(rng, lens, ps)
    pool = random_pool(rng, num_pages, Hkv, ps, d)
    for i, n in enumerate(lens):
        set_params(pool, ps, d, False, table[i], range(n), factor=2.0 ** k_exp)
    q = (bf16(rng, (2, Hq, d)).float() * 2.0 ** q_exp).to(BF)
    scale = 2.0 ** scale_exp / math.sqrt(d)
    o, lse, status = run_decode(q, pool, widen(table, ps) if wide else table, lens, ps, scale)
    assert status == 0
    check_weighted(o, lse, q, pool, table, lens, ps, scale)


@pytest.mark.parametrize("exponent", [-100, 100])
@pytest.mark.parametrize("wide", [False, True])
def test_values_near_the_ends_of_the_range(wide, exponent, cuda_device):
    # the sums of V stay finite in fp32; scales of 2^-104 are still normal numbers
    rng = np.random.default_rng(5)
    lens, d, ps = [300, 64], 128, 16
    table, num_pages = layout(rng, lens, ps)
    pool = random_pool(rng, num_pages, 2, ps, d)
    for i, n in enumerate(lens):
        set_params(pool, ps, d, True, table[i], range(n), factor=2.0 ** exponent)
    q = bf16(rng, (2, 8, d))
    o, lse, status = run_decode(q, pool, widen(table, ps) if wide else table, lens, ps, 0.09)
    assert status == 0
    check_weighted(o, lse, q, pool, table, lens, ps, 0.09)
