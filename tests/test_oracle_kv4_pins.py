"""Pins of the 4-bit cache's oracle and of the page oracle, against independent statements of the
same things (exact fractions, set arithmetic, a simulation of what pages hold).  CPU only."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import kv4, pages
from oracle.attention import attention


@pytest.mark.parametrize("d", [64, 128, 256])
def test_record_places_are_a_partition(d):
    ng = d // 64
    nibbles = set()
    for place in (kv4.k_code_place, kv4.v_code_place):
        for t in range(16):
            for c in range(d):
                w, n = place(t, c, d)
                assert w % 4 == 0 and 0 <= n < 8
                nibbles.add(2 * w + n)
    assert nibbles == set(range(2 * 1024 * ng))  # every nibble of the code part, once
    params = [kv4.param_place(v, t, g, d) for v in (False, True) for t in range(16) for g in range(ng)]
    assert sorted(params) == list(range(1024 * ng, 1152 * ng, 4))
    assert kv4.record_bytes(d) == 1152 * ng == 16 * d * 9 // 8


def bf16_fraction(x: Fraction) -> Fraction:
    """Round a positive fraction to bf16's 8-bit significand, ties to even (no subnormals here)."""
    e = 0
    while x >= 2 ** (e + 1):
        e += 1
    while x < Fraction(2) ** e:
        e -= 1
    ulp = Fraction(2) ** (e - 7)
    n = x / ulp
    f = n.numerator // n.denominator
    r = n - f
    if r > Fraction(1, 2) or (r == Fraction(1, 2) and f % 2):
        f += 1
    return f * ulp


def nearest(q: Fraction) -> int:
    f = q.numerator // q.denominator
    r = q - f
    if r > Fraction(1, 2) or (r == Fraction(1, 2) and f % 2):
        f += 1
    return min(f, 15)


def test_quantizer_against_exact_fractions():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 64)).astype(np.float32) * 2.0 ** rng.integers(-6, 7, (40, 1)).astype(np.float32)
    x[10:20] = np.round(x[10:20] * 4) / 4  # coarse values: quotients on and next to the borders
    x[20:24] += 100.0
    x[24, 1:] = 0.0
    x[25] = np.arange(64) / 8.0  # span 63/8
    x[26:30] = rng.integers(0, 31, (4, 64)) / 2.0 - 4.0  # half steps of the scale 1: ties
    x[26:30, :2] = [-4.0, 11.0]
    x = kv4.bf16_value(kv4.bf16_bits(x))
    codes, s, m = kv4.quantize(x)
    ties = 0
    for r in range(x.shape[0]):
        f = [Fraction(float(v)) for v in x[r]]
        lo, hi = min(f), max(f)
        if lo == hi:  # covered by the special groups
            continue
        # the span of bf16 values of one scale is exact in fp32; its 15th part rounds to fp32 first
        span32 = Fraction(float(np.float32(float(hi - lo)) / np.float32(15)))
        scale = bf16_fraction(span32)
        assert Fraction(float(kv4.bf16_value(s[r, 0]))) == scale
        assert Fraction(float(kv4.bf16_value(m[r, 0]))) == lo
        for c in range(64):
            q = (f[c] - lo) / scale
            assert codes[r, c] == nearest(q)
            ties += q.denominator == 2
    assert ties > 5  # the borders were met


def test_quantizer_special_groups():
    x = np.zeros((6, 64))
    x[0] = -3.5                       # constant: every code stands for the minimum
    x[1, :2] = [-0.0, 0.0]
    x[2, 5] = np.inf
    x[3, 7] = np.nan
    x[4, :2] = [3.0e38, -3.0e38]      # the range overflows fp32
    x[5, 0] = 2.0 ** -130             # a scale below bf16's normal numbers
    codes, s, m = kv4.quantize(x)
    v = kv4.values(codes, s, m)
    assert s[0, 0] == 0 and np.all(codes[0] == 0) and np.all(v[0] == -3.5)
    assert m[1, 0] == 0 and s[1, 0] == 0
    for r in (2, 3, 4):
        assert s[r, 0] == m[r, 0] == 0x7FC0 and np.all(codes[r] == 0) and np.all(np.isnan(v[r]))
    # 2^-130 / 15 = 1.07 * 2^-134 rounds to bf16's smallest subnormal 2^-133; 2^-130 / 2^-133 = 8
    assert kv4.bf16_value(s[5, 0]) == 2.0 ** -133 and codes[5, 0] == 8 and np.all(codes[5, 1:] == 0)


def test_error_of_a_value_is_half_a_step():
    rng = np.random.default_rng(6)
    x = kv4.bf16_value(kv4.bf16_bits(rng.standard_normal((200, 128)).astype(np.float32)))
    codes, s, m = kv4.quantize(x)
    step = np.repeat(kv4.bf16_value(s), 64, axis=-1)
    # half a step, and at the top what the scale's rounding (2^-8 at most) takes off 15 steps
    assert np.all(np.abs(kv4.values(codes, s, m) - x) <= step * (0.5 + 15 * 2.0 ** -8))


@pytest.mark.parametrize("d,page_size", [(64, 16), (128, 32), (256, 64)])
def test_append_then_read_back_and_attend(d, page_size):
    rng = np.random.default_rng(d)
    lens, cu = [page_size + 5, 3], [0, page_size + 5, page_size + 8]
    table = np.array([[2, 0], [3, -1]])
    k = kv4.bf16_value(kv4.bf16_bits(rng.standard_normal((cu[-1], 2, d)).astype(np.float32)))
    v = kv4.bf16_value(kv4.bf16_bits(rng.standard_normal((cu[-1], 2, d)).astype(np.float32)))
    pool = rng.integers(0, 256, (4, 2, page_size * d * 9 // 8), dtype=np.uint8)
    before = pool.copy()
    pool = kv4.append(pool, k, v, table, lens, cu, page_size)
    assert np.array_equal(pool[1], before[1])  # a page of no row
    K, V = kv4.pool_values(pool, page_size, d)
    q = rng.standard_normal((2, 4, d))
    o, lse = kv4.decode_paged_kv4(q, pool, table, lens, page_size, 0.1)
    for i in range(2):
        rows = [(table[i][t // page_size], t % page_size) for t in range(lens[i])]
        got_k = np.stack([K[p, :, t] for p, t in rows], 1)
        got_v = np.stack([V[p, :, t] for p, t in rows], 1)
        want_k = kv4.values(*kv4.quantize(k[cu[i]:cu[i + 1]])).transpose(1, 0, 2)
        want_v = kv4.values(*kv4.quantize(v[cu[i]:cu[i + 1]])).transpose(1, 0, 2)
        assert np.array_equal(got_k, want_k) and np.array_equal(got_v, want_v)
        ro, rl = attention(q[i][None, :, None], want_k[None], want_v[None], 0.1, False)
        np.testing.assert_allclose(o[i], ro[0, :, 0], rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(lse[i], rl[0, :, 0], rtol=1e-12)


def random_rows(rng, S, page_size, cols, extra):
    lens = [int(rng.integers(0, cols * page_size + 1)) for _ in range(S)]
    need = [-(-n // page_size) for n in lens]
    num_pages = sum(need) + extra
    perm = rng.permutation(num_pages)
    table = np.full((S, cols), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    return table, lens, num_pages


def read_tokens(content, row, n, page_size):
    return [content[int(row[t // page_size])][t % page_size] for t in range(n)]


def test_fork_keeps_every_row_and_isolates_its_tail():
    rng = np.random.default_rng(11)
    for trial in range(60):
        ps, cols = int(rng.choice([16, 32])), int(rng.integers(1, 5))
        S = int(rng.integers(1, 6))
        table, lens, num_pages = random_rows(rng, S, ps, cols, extra=40)
        content = {p: [(p, t) for t in range(ps)] for p in range(num_pages)}
        for step in range(3):  # forks of forks: rows then share full pages
            rows = int(rng.integers(1, 8))
            parents = [int(rng.integers(-1, len(lens))) for _ in range(rows)]
            add = [int(rng.integers(-20, 25)) for _ in range(rows)]
            out, new_lens, left, copies, short = pages.fork(table, lens, parents, add, cols, ps, num_pages)
            assert not short
            sources, targets = {c[0] for c in copies}, [c[1] for c in copies]
            assert len(set(targets)) == len(targets) and not sources & set(targets)
            old = [read_tokens(content, table[p], lens[p], ps) if p >= 0 else [] for p in parents]
            for src, dst in copies:
                content[dst] = list(content[src])
            for i in range(rows):
                kept = min(len(old[i]), int(new_lens[i]))
                assert read_tokens(content, out[i], kept, ps) == old[i][:kept]
                n = -(-int(new_lens[i]) // ps)
                assert np.all(out[i, :n] >= 0) and np.all(out[i, n:] == -1)
            # the pages a row may write (from its kept end on) are in no other row
            uses = {}
            for i in range(rows):
                for e in out[i, : -(-int(new_lens[i]) // ps)]:
                    uses.setdefault(int(e), []).append(i)
            for i in range(rows):
                kept = min(len(old[i]), int(new_lens[i]))
                for j in range(kept // ps, -(-int(new_lens[i]) // ps)):
                    assert uses[int(out[i, j])] == [i]
            assert left == num_pages - len(uses)
            for i in range(rows):  # writing the new tokens disturbs nobody
                for t in range(min(len(old[i]), int(new_lens[i])), int(new_lens[i])):
                    content[int(out[i, t // ps])][t % ps] = ("new", trial, step, i, t)
            table, lens = out, [int(n) for n in new_lens]


def test_fork_without_enough_pages():
    table, lens = np.array([[0, -1], [1, -1]]), [16, 5]
    out, new_lens, left, copies, short = pages.fork(table, lens, [0, 1, 1], [1, 0, 0], 2, 16, 3)
    assert short and left == 0 and out.tolist() == [[0, 2], [1, -1], [-1, -1]] and copies == []


def test_compact_moves_every_page_once():
    rng = np.random.default_rng(12)
    for _ in range(60):
        ps, cols = 16, int(rng.integers(1, 6))
        table, lens, num_pages = random_rows(rng, int(rng.integers(1, 6)), ps, cols, extra=int(rng.integers(0, 30)))
        if len(lens) > 1 and lens[0] >= ps and lens[1] >= ps:
            table[1, 0] = table[0, 0]  # a shared page
        content = {p: [(p, t) for t in range(ps)] for p in range(num_pages)}
        old = [read_tokens(content, r, n, ps) for r, n in zip(table, lens)]
        out, page_map, live, moves = pages.compact(table, lens, ps, num_pages)
        moved = {dst: list(content[src]) for src, dst in moves}
        content.update(moved)
        assert [read_tokens(content, r, n, ps) for r, n in zip(out, lens)] == old
        assert sorted(p for p in page_map if p >= 0) == list(range(live))
        assert all(src >= live > dst for src, dst in moves)
