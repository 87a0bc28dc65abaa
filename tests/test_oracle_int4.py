"""Pins of the 4-bit cache's CPU definitions: closed forms and brute force, no GPU."""
import numpy as np
import pytest
import torch

from oracle import int4 as Q
from oracle import serving as S


def test_bf16_rounding_is_torchs():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(10000) * 10.0 ** rng.uniform(-38, 37, 10000)).astype(np.float32)
    x = np.concatenate([x, np.float32([0, 1, 1 + 2 ** -8, 1 + 3 * 2 ** -8, np.inf, 2.0 ** -133, 2.0 ** -140])])
    np.testing.assert_array_equal(Q.to_bf16(x), torch.from_numpy(x).to(torch.bfloat16).float().numpy())


@pytest.mark.parametrize("d", [32, 64, 256])
def test_codes_are_the_nearest(d):
    rng = np.random.default_rng(d)
    x = (rng.standard_normal((50, d)) * 10.0 ** rng.uniform(-6, 6, (50, 1))).astype(np.float32)
    c, s = Q.quant4(x)
    assert s.shape == (50, d // 32) and np.abs(c).max() == 7
    step = np.repeat(s.astype(np.float64), 32, -1)
    grid = np.arange(-7, 8) * step[..., None]
    best = np.abs(grid - x[..., None].astype(np.float64)).min(-1)
    assert (np.abs(c * step - x) <= best * (1 + 1e-12)).all()
    np.testing.assert_array_equal(s, torch.from_numpy(np.abs(x).reshape(50, -1, 32).max(-1) / np.float32(7)).to(torch.bfloat16).float().numpy())


def test_ties_go_to_even_and_rows_that_are_special():
    x = np.zeros((6, 32), np.float32)
    x[0, :6] = [7, 0.5, 1.5, 2.5, -0.5, -1.5]
    x[1] = 0
    x[2, 3] = np.inf
    x[3, :2] = [np.nan, 14]
    x[4, :3] = [2.0 ** -131, 2.0 ** -140, 0]     # s = bf16(2^-131 / 7) is one step of 2^-133
    x[5, 0] = 2.0 ** -136                        # rounds to a scale of 0
    c, s = Q.quant4(x)
    assert c[0, :6].tolist() == [7, 0, 2, 2, 0, -2] and s[0] == 1
    assert (c[1] == 0).all() and s[1] == 0
    assert (c[2] == 0).all() and np.isinf(s[2])
    assert c[3, :2].tolist() == [0, 7] and s[3] == 2
    assert s[4] == 2.0 ** -133 and c[4, :3].tolist() == [4, 0, 0]
    assert s[5] == 0 and (c[5] == 0).all()


def test_bytes():
    c = np.arange(32) % 15 - 7
    p = Q.pack(c)
    assert p.shape == (16,) and p[0] == (c[0] + 8) | (c[1] + 8) << 4
    np.testing.assert_array_equal(Q.unpack(p), c)
    assert Q.unpack(np.uint8([0])).tolist() == [-8, -8]
    np.testing.assert_array_equal(Q.values(p, np.float32([0.5])), c * 0.5)


def test_visible():
    assert Q.visible(5, 1, 0) == [0, 1, 2, 3, 4] and Q.visible(5, 3, 0) == [0, 1, 2] and Q.visible(5, 3, 2) == [0, 1, 2, 3, 4]
    assert Q.visible(5, 3, 1, 0b101) == [0, 1, 2, 4] and Q.visible(5, 3, 0, 0) == [0, 1]
    assert Q.visible(2, 3, 0) == [] and Q.visible(2, 3, 1) == [0] and Q.visible(2, 3, 0, 0b111) == [0, 1]


def test_attention_against_the_int8_definition():
    """Rows whose groups share a scale are int8 rows of the same codes."""
    rng = np.random.default_rng(3)
    B, T, hq, hkv, d, page, nb = 2, 1, 4, 2, 64, 16, 3
    kc, vc = (rng.integers(-8, 8, (7, hkv, page, d)) for _ in range(2))
    ks, vs = (Q.to_bf16(rng.uniform(0.1, 0.3, (7, hkv, page))) for _ in range(2))
    tables, lens = rng.permutation(7)[:6].reshape(B, nb), np.array([40, 17])
    q = rng.standard_normal((B, T, hq, d)).astype(np.float32)
    out, lse = Q.attention(q, Q.pack(kc), np.repeat(ks[..., None], 2, -1), Q.pack(vc), np.repeat(vs[..., None], 2, -1), tables, lens)
    want, wlse = S.sparse_attention(q[:, 0], kc.astype(np.int8), ks, vc.astype(np.int8), vs, np.repeat(tables[:, None], hkv, 1),
                                    np.repeat(lens[:, None], hkv, 1))
    np.testing.assert_allclose(out[:, 0], want, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(lse[:, 0], wlse, rtol=1e-12)


def test_drafts_are_single_queries_of_shorter_sequences():
    rng = np.random.default_rng(4)
    T, hq, hkv, d, page = 3, 4, 1, 32, 16
    kc, vc = (Q.pack(rng.integers(-7, 8, (4, hkv, page, d))) for _ in range(2))
    ks, vs = (Q.to_bf16(rng.uniform(0.1, 0.3, (4, hkv, page, 1))) for _ in range(2))
    q = rng.standard_normal((1, T, hq, d)).astype(np.float32)
    out, lse = Q.attention(q, kc, ks, vc, vs, [[2, 0, 3]], [37])
    for t in range(T):
        one, olse = Q.attention(q[:, t:t + 1], kc, ks, vc, vs, [[2, 0, 3]], [37 - T + 1 + t])
        np.testing.assert_allclose(out[:, t], one[:, 0], rtol=1e-12)
        np.testing.assert_allclose(lse[:, t], olse[:, 0], rtol=1e-12)
    full = [[0b111] * T]
    every, _ = Q.attention(q, kc, ks, vc, vs, [[2, 0, 3]], [37], full)
    np.testing.assert_allclose(every[:, 2], out[:, 2], rtol=1e-12)


def test_the_scale_s_quotient_without_a_division():
    """group_scale of csrc/cache4.cuh forms m / 7 as q + (m - 7 q) c, q = RN(m c) and c = RN(1 / 7), each sum fused: the quotient's
    own rounding for every significand m of 24 bits, in whole numbers.  A power of two scales all of it alike."""
    c = int(np.float32(1 / 7) * 2.0 ** 26)  # of 2^-26
    assert 1 << 23 <= c < 1 << 24 and c == float(np.float32(1) / np.float32(7)) * 2.0 ** 26

    def rounded(x):  # to 24 significant bits, ties to even; frexp is exact for x < 2^53
        drop = np.frexp(x.astype(np.float64))[1] - 24
        low, half, kept = x & ((1 << drop) - 1), np.int64(1) << (drop - 1), x >> drop
        return (kept + ((low > half) | ((low == half) & (kept & 1 == 1)))) << drop

    for first in range(1 << 23, 1 << 24, 1 << 20):
        m = np.arange(first, first + (1 << 20), dtype=np.int64)
        q = rounded(m * c)  # of 2^-26
        rest = (m << 26) - 7 * q
        assert np.all(rest % (1 << 22) == 0) and np.all(np.abs(rest) >> 22 < 1 << 24)  # exact in fp32
        got = rounded((q << 4) + (rest >> 22) * c)  # of 2^-30
        whole, left = np.divmod(m << 30, 7)
        want = rounded(2 * whole + (left > 0)) >> 1  # the last bit says that something is left
        np.testing.assert_array_equal(got, want)
