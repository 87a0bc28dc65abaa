"""Pins of the serving operators' CPU definitions: cases worked by hand and invariants."""
import numpy as np
import pytest

from oracle import serving as S


def test_page_plan_by_hand():
    # pages of 4 tokens; slot 1 has ended and gives back pages 7, 8; slot 0 opens one page,
    # slot 2 stays inside its page, slot 3 asks for more than is left
    table = [[5, -1, -1], [7, 8, -1], [9, -1, -1], [-1, -1, -1]]
    r = S.paged_assign([4, 6, 1, 0], [2, 0, 2, 9], [0, 1, 0, 0], table, [3, -1, -1, -1, -1], 1, 4, 16)
    assert r["free_count"] == 2 and list(r["free_pages"][:3]) == [3, 7, 8]
    assert r["block_table"].tolist() == [[5, 8, -1], [7, 8, -1], [9, -1, -1], [-1, -1, -1]]
    assert list(r["seqlens"]) == [6, 0, 3, 0] and list(r["granted"]) == [2, 0, 2, 0]
    assert list(r["cu_new"]) == [0, 2, 2, 4, 13]
    assert list(r["slot_map"]) == [32, 33, 37, 38] + [-1] * 12
    assert list(r["token_pos"]) == [4, 5, 1, 2] + list(range(9)) + [0] * 3


def test_page_plan_keeps_every_page_once():
    rng = np.random.default_rng(3)
    for _ in range(50):
        B, nb, page = int(rng.integers(1, 12)), 6, int(rng.integers(1, 5))
        ctx = rng.integers(0, nb * page + 1, B)
        held = -(-ctx // page)
        total = int(held.sum()) + int(rng.integers(0, 12))
        perm = rng.permutation(total)
        table, at = np.full((B, nb), -1), 0
        for b in range(B):
            table[b, :held[b]] = perm[at:at + held[b]]
            at += held[b]
        free = np.full(total, -1)
        free[:total - at] = perm[at:]
        release = rng.integers(0, 2, B)
        new = rng.integers(0, 2 * page, B)
        r = S.paged_assign(ctx, new, release, table, free, total - at, page, 64)
        used = [int(p) for b in range(B) for p in r["block_table"][b, :-(-r["seqlens"][b] // page)]]
        assert sorted(used + list(r["free_pages"][:r["free_count"]])) == list(range(total))


def test_rope_quarter_turns_and_norms():
    x = np.arange(8, dtype=np.float64).reshape(1, 1, 8)
    quarter = np.float32(np.pi / 2)
    y = S.rope(x, [[1]], [quarter, 0.0], adjacent=False)  # pairs (0, 2), (1, 3); 4.. pass
    np.testing.assert_allclose(y[0, 0], [-2, 1, 0, 3, 4, 5, 6, 7], atol=1e-6)
    y = S.rope(x, [[0], [1]], [quarter, quarter], pair_axis=[0, 1], adjacent=True)  # pair 1 turns
    np.testing.assert_allclose(y[0, 0], [0, 1, -3, 2, 4, 5, 6, 7], atol=1e-6)
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 2, 16))
    y = S.rope(x, rng.integers(0, 1000, (3, 5)), rng.random(8), pair_axis=[0, 1, 2] * 2 + [0, 1])
    np.testing.assert_allclose(np.linalg.norm(x, axis=-1), np.linalg.norm(y, axis=-1))


def test_bounds_enclose_the_keys_and_the_score_the_logits():
    rng = np.random.default_rng(2)
    for n in (1, 3, 16):
        codes = rng.integers(-127, 128, (n, 32)).astype(np.int8)
        scales = rng.random(n).astype(np.float32)
        lo, hi, s = S.page_bounds(codes, scales)
        k = codes.astype(np.float64) * scales[:, None]
        assert np.all(lo * float(s) <= k.min(0) + 1e-5) and np.all(hi * float(s) >= k.max(0) - 1e-5)
        assert np.all(k.min(0) - lo * float(s) < float(s)) and np.all(hi * float(s) - k.max(0) < float(s))
        q = rng.standard_normal((4, 32)).astype(np.float32)
        qc, qs = S._quant(q)
        best = (qc.astype(np.float64) * qs[:, None] @ k.T).max()
        score = S.page_scores(q, lo[None], hi[None], np.array([s]))[0]
        assert score >= best - 1e-4 * abs(best)
        if n == 1:  # a single row is its own bound: the score is the logit
            assert np.array_equal(lo, codes[0]) and np.array_equal(hi, codes[0])
            assert abs(score - best) <= 1e-5 * abs(best)
    lo, hi, s = S.page_bounds(np.zeros((4, 32), np.int8), np.zeros(4, np.float32))
    assert s == 0 and not lo.any() and not hi.any()


def test_select_ties_and_forced_blocks():
    assert S.select([1, 5, 5, 5, 0, 2], 4, 1, 1) == [0, 1, 2, 5]
    assert S.select([1, 5, 5, 5, 0, 2], 4, 0, 0) == [1, 2, 3, 5]
    assert S.select([0, 0, 0], 4, 2, 2) == [0, 1, 2]
    assert S.select([9, 8, 7, 6, 5], 3, 1, 2) == [0, 3, 4]


def test_sparse_attention_is_softmax_over_the_listed_tokens():
    rng = np.random.default_rng(4)
    k = rng.integers(-127, 128, (5, 1, 4, 32)).astype(np.int8)
    v = rng.integers(-127, 128, (5, 1, 4, 32)).astype(np.int8)
    ks, vs = (rng.random((5, 1, 4)).astype(np.float32) * 0.02 for _ in range(2))
    q = np.zeros((1, 2, 32), np.float32)  # equal weights: the mean of the values
    out, lse = S.sparse_attention(q, k, ks, v, vs, np.array([[[3, 1]]]), np.array([[6]]))
    rows = np.concatenate([v[3, 0] * vs[3, 0][:, None], (v[1, 0] * vs[1, 0][:, None])[:2]])
    np.testing.assert_allclose(out[0], np.broadcast_to(rows.mean(0), (2, 32)), rtol=1e-6, atol=1e-9)
    np.testing.assert_allclose(lse, np.log(6))
    out, lse = S.sparse_attention(q, k, ks, v, vs, np.array([[[3, 1]]]), np.array([[0]]))
    assert not out.any() and np.all(lse == -np.inf)


@pytest.mark.parametrize("sections,inter,want", [((2, 1, 1), False, [0, 0, 1, 2]), ((3, 1, 2), True, [0, 1, 2, 0, 2, 0])])
def test_pair_axis(sections, inter, want):
    import w8a8_int8_flashattention_gb300 as sl8
    assert list(sl8.rope_pair_axis(sections, inter)) == want
