"""The 4-bit paged cache: its values, its record layout and the quantizer, in fp64.

TEST INFRASTRUCTURE ONLY, like the rest of this package.

Format (a reading of this project; the pages fix none): a value is s * c + m with a 4-bit code c
and, per token and group of 64 channels, a bf16 scale s and a bf16 minimum m.

* m is the group's smallest value (a zero as +0); s = bf16((max - min) / 15), the subtraction and the
  division in fp32 with round-to-nearest, then bf16 with ties to even;
* c is the integer nearest to the exact quotient (x - m) / s, ties to even, at most 15; where s is 0
  the quotient is 0/0 (code 0) or infinite (code 15), and every code stands for m;
* a group whose fp32 range is not finite has s = m = NaN (bits 0x7fc0) and codes 0.

Attention over the cache is the exact attention (``attention.py``) of these values.
"""

from __future__ import annotations

import numpy as np

from .attention import decode_paged

TOK = 16
GROUP = 64


def record_bytes(d: int) -> int:
    return 1152 * (d // GROUP)


def page_bytes(Hkv: int, page_size: int, d: int) -> int:
    return Hkv * (page_size // TOK) * record_bytes(d)


def k_code_place(token: int, channel: int, d: int) -> tuple[int, int]:
    """(byte of the 32-bit word, nibble in it) of a key's code in its record."""
    a, b1, b0 = token // 4, token // 2 % 2, token % 2
    y, x = divmod(channel, GROUP)
    word = 512 * y + 16 * ((2 * a + b0) * 4 + x // 16) + 8 * b1 + 4 * (x // 8 % 2)
    j = x % 8
    return word, j // 2 + 4 * (j % 2)


def v_code_place(token: int, channel: int, d: int) -> tuple[int, int]:
    a, b1, b0 = token // 4, token // 2 % 2, token % 2
    y, x = divmod(channel, GROUP)
    word = 512 * (d // GROUP) + 512 * y + 128 * a + 16 * ((x // 8) ^ (2 * a)) + 8 * b1 + 4 * (x // 4 % 2)
    return word, 4 * b0 + x % 4


def param_place(is_v: bool, token: int, group: int, d: int) -> int:
    """Byte of the (s, m) word."""
    ng = d // GROUP
    a, b1, b0 = token // 4, token // 2 % 2, token % 2
    return (1088 if is_v else 1024) * ng + 4 * (((2 * a + b0) * 2 + b1) * ng + group)


def _places(d: int):
    """Index arrays [16, d]: byte and shift of K's and V's codes; [16, d/64]: bytes of the parameters."""
    out = []
    for place in (k_code_place, v_code_place):
        byte = np.empty((TOK, d), dtype=np.int64)
        shift = np.empty((TOK, d), dtype=np.int64)
        for t in range(TOK):
            for c in range(d):
                w, n = place(t, c, d)
                byte[t, c], shift[t, c] = w + n // 2, 4 * (n % 2)
        out.append((byte, shift))
    par = [np.array([[param_place(v, t, g, d) for g in range(d // GROUP)] for t in range(TOK)]) for v in (False, True)]
    return out, par


_PLACES: dict[int, tuple] = {}


def places(d: int):
    if d not in _PLACES:
        _PLACES[d] = _places(d)
    return _PLACES[d]


def bf16_bits(x) -> np.ndarray:
    """fp32 values to bf16 bits, round to nearest even; NaN as 0x7fc0."""
    x = np.asarray(x, dtype=np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16_value(bits) -> np.ndarray:
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantize(x) -> tuple[np.ndarray, np.ndarray, np.ndarray]:
    """fp64 values (bf16 ones) [..., d] -> codes uint8 [..., d], s and m bits uint16 [..., d/64]."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1) + 0.0, g.max(-1) + 0.0  # NaN propagates, zeros become +0
        span = hi.astype(np.float32) - lo.astype(np.float32)
        fine = np.isfinite(span)
        s_bits = np.where(fine, bf16_bits(span / np.float32(15)), np.uint16(0x7FC0))
        m_bits = np.where(fine, bf16_bits(lo.astype(np.float32)), np.uint16(0x7FC0))
        s, m = bf16_value(s_bits)[..., None], bf16_value(m_bits)[..., None]
        c = np.minimum(np.rint((g - m) / s), 15.0)
        c = np.where(np.isnan(c), 0.0, c)
    return c.astype(np.uint8).reshape(x.shape), s_bits.astype(np.uint16), m_bits.astype(np.uint16)


def values(codes, s_bits, m_bits) -> np.ndarray:
    """The exact values s * c + m, fp64."""
    c = np.asarray(codes).reshape(*np.shape(codes)[:-1], -1, GROUP).astype(np.float64)
    with np.errstate(all="ignore"):
        v = bf16_value(s_bits)[..., None] * c + bf16_value(m_bits)[..., None]
    return v.reshape(np.shape(codes))


def write_token(record: np.ndarray, token: int, is_v: bool, codes, s_bits, m_bits) -> None:
    """Writes one token's K (or V) into a record (uint8 view, in place)."""
    d = len(codes)
    coded, par = places(d)
    byte, shift = coded[int(is_v)]
    for c in range(d):
        b, sh = byte[token, c], shift[token, c]
        record[b] = (int(record[b]) & (0xF0 if sh == 0 else 0x0F)) | (int(codes[c]) << int(sh))
    for g in range(d // GROUP):
        p = par[int(is_v)][token, g]
        record[p:p + 4] = np.array([s_bits[g], m_bits[g]], dtype=np.uint16).view(np.uint8)


def pool_values(pool, page_size: int, d: int) -> tuple[np.ndarray, np.ndarray]:
    """K and V values fp64 [num_pages, Hkv, page_size, d] of a pool uint8 [num_pages, Hkv, bytes]."""
    pool = np.asarray(pool)
    P, H, _ = pool.shape
    rec = pool.reshape(P, H, page_size // TOK, record_bytes(d))
    coded, par = places(d)
    words = rec.view(np.uint16)
    out = []
    for (byte, shift), at in zip(coded, par):
        codes = (rec[..., byte] >> shift.astype(np.uint8)) & 15
        out.append(values(codes, words[..., at // 2], words[..., at // 2 + 1]).reshape(P, H, page_size, d))
    return out[0], out[1]


def append(pool, k, v, block_table, seq_lens, cu_new, page_size: int) -> np.ndarray:
    """The pool after appending k and v [T, Hkv, d]."""
    pool = np.array(pool)
    P, H, _ = pool.shape
    d = k.shape[-1]
    rec = pool.reshape(P, H, page_size // TOK, record_bytes(d))
    for is_v, x in ((False, k), (True, v)):
        codes, s, m = quantize(x)
        for i, n in enumerate(seq_lens):
            lo, hi = int(cu_new[i]), int(cu_new[i + 1])
            for t in range(lo, hi):
                pos = int(n) - (hi - t)
                page = int(block_table[i][pos // page_size])
                for h in range(H):
                    write_token(rec[page, h, pos % page_size // TOK], pos % TOK, is_v, codes[t, h], s[t, h], m[t, h])
    return pool


def decode_paged_kv4(q, pool, block_table, seq_lens, page_size: int, scale: float):
    """(O, LSE) of one decode step over the 4-bit pool, fp64."""
    k, v = pool_values(pool, page_size, q.shape[-1])
    # slots past a sequence's end, and pages of no sequence, may hold anything
    return decode_paged(q, np.nan_to_num(k, posinf=0, neginf=0), np.nan_to_num(v, posinf=0, neginf=0), block_table,
                        seq_lens, page_size, scale)
