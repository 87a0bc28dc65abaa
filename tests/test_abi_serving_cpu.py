"""Refusals of the serving entry points (no GPU needed): every argument error returns its
status before anything is launched, and the binding refuses what the ABI cannot see."""
import ctypes

import pytest
import torch

import w8a8_int8_flashattention_gb300 as sl8
from w8a8_int8_flashattention_gb300 import build as sl8_build

INVALID, UNSUPPORTED, WORKSPACE, OK = sl8.SL8_ERR_INVALID_ARG, sl8.SL8_ERR_UNSUPPORTED, sl8.SL8_ERR_WORKSPACE, sl8.SL8_OK


@pytest.fixture(scope="module")
def lib():
    sl8_build.build()
    return sl8.lib()


@pytest.fixture(scope="module")
def p():
    buf = ctypes.create_string_buffer(1 << 12)
    at = (ctypes.addressof(buf) + 15) // 16 * 16
    yield at
    del buf


def _changed(args, changes):
    a = list(args)
    for i, v in changes.items():
        a[i] = v
    return a


def test_paged_assign(lib, p):
    f = lib.sl8_paged_assign
    #      ctx new rel B  page nb tab free cap cnt out  T   seq gr cu slot pos stream
    ok = [p, p, None, 4, 16, 8, p, p, 32, p, p, 64, p, p, p, p, None, None]
    for i in (0, 1, 6, 7, 9, 10, 12, 13, 14, 15):
        assert f(*_changed(ok, {i: None})) == INVALID, i
    for i, v in ((3, -1), (4, 0), (5, 0), (8, -1), (11, -1)):
        assert f(*_changed(ok, {i: v})) == INVALID, (i, v)
    assert f(*_changed(ok, {4: 1 << 16, 5: 1 << 15})) == UNSUPPORTED


def test_rope_append(lib, p):
    f = lib.sl8_rope_append
    axis = bytes([0] * 32 + [1] * 32)
    #    0  1  2  3             4     5    6    7  8  9  10   11 12 13   14 15    16 17 18   19 20 21 22 23 24 25  26
    ok = [p, p, p, sl8.SL8_BF16, 4096, 512, 512, 4, 8, 4, 128, p, 2, 128, p, axis, 0, p, 1024, p, p, p, p, p, 16, 16, None]
    assert f(*_changed(ok, {7: 0})) == OK                       # nothing to do
    for i in (0, 1, 2, 11, 14, 17, 19, 20, 21, 22, 23):
        assert f(*_changed(ok, {i: None})) == INVALID, i
    for i, v in ((3, sl8.SL8_I8), (4, 1000), (5, 511), (6, 508), (18, 1020), (7, -1), (8, -1), (9, 0), (24, 0), (25, 0),
                 (13, 136), (0, p + 8), (20, p + 4), (15, None), (15, bytes([2] * 64)), (12, 0)):
        assert f(*_changed(ok, {i: v})) == INVALID, (i, v)
    for change in ({10: 96, 13: 96}, {13: 100}, {12: 5}, {24: 1 << 20, 25: 1 << 12}):
        assert f(*_changed(ok, change)) == UNSUPPORTED, change
    # fp32 rows advance in 16 bytes: 4 elements
    assert f(*_changed(ok, {3: sl8.SL8_F32, 5: 514})) == INVALID


def test_page_bounds(lib, p):
    f = lib.sl8_page_bounds
    #    0  1  2   3   4  5  6  7  8  9  10 11   12 13 14
    ok = [p, p, 16, 16, p, 8, p, p, 4, 2, 2, 128, p, p, None]
    assert f(*_changed(ok, {9: 0})) == OK and f(*_changed(ok, {8: 0})) == OK
    for i in (0, 1, 4, 6, 12, 13):
        assert f(*_changed(ok, {i: None})) == INVALID, i
    for i, v in ((2, 0), (3, 0), (5, 0), (8, -1), (9, -1), (10, 0), (0, p + 8), (12, p + 8)):
        assert f(*_changed(ok, {i: v})) == INVALID, (i, v)
    assert f(*_changed(ok, {11: 96})) == UNSUPPORTED


def test_page_select(lib, p):
    f = lib.sl8_page_select
    #    0  1             2  3  4   5   6  7   8  9  10 11 12 13   14 15 16 17 18 19 20    21
    ok = [p, sl8.SL8_BF16, p, p, 16, 16, p, 64, p, 2, 1, 8, 2, 128, 8, 1, 2, p, p, p, None, None]
    assert f(*_changed(ok, {9: 0})) == OK and f(*_changed(ok, {10: 0})) == OK
    for i in (0, 2, 3, 6, 8, 17, 18, 19):
        assert f(*_changed(ok, {i: None})) == INVALID, i
    for change in ({1: sl8.SL8_I8}, {4: 0}, {5: 0}, {7: 0}, {9: -1}, {10: -1}, {11: 7}, {12: 0}, {14: 0}, {15: -1},
                   {15: 7}, {16: 9}, {0: p + 8}, {2: p + 8}):
        assert f(*_changed(ok, change)) == INVALID, change
    assert f(*_changed(ok, {7: 4097})) == INVALID               # a wide table needs the scores
    assert f(*_changed(ok, {2: p | 16})) == INVALID              # bounds are read 32 bytes at a time
    for change in ({13: 96}, {11: 130}, {5: 1 << 16, 7: 1 << 15}, {9: 1 << 20, 10: 1 << 10}):
        assert f(*_changed(ok, change)) == UNSUPPORTED, change


def test_sparse_decode(lib, p):
    f = lib.sl8_attn_int8_sparse_decode
    #    0  1             2  3  4  5  6   7   8  9  10 11 12 13 14   15 16 17            18    19 20       21
    ok = [p, sl8.SL8_BF16, p, p, p, p, 16, 16, p, p, 8, 2, 8, 2, 128, 0, p, sl8.SL8_BF16, None, p, 1 << 30, None]
    assert f(*_changed(ok, {11: 0})) == OK
    for i in (0, 2, 3, 4, 5, 8, 9, 16):
        assert f(*_changed(ok, {i: None})) == INVALID, i
    for change in ({1: sl8.SL8_I8}, {17: sl8.SL8_I8}, {6: 0}, {7: 0}, {10: 0}, {11: -1}, {12: 7}, {15: -1}, {0: p + 4},
                   {3: p + 4}):
        assert f(*_changed(ok, change)) == INVALID, change
    for change in ({14: 96}, {7: 24}, {6: 1 << 20, 7: 1 << 11}):
        assert f(*_changed(ok, change)) == UNSUPPORTED, change
    assert sl8.sparse_decode_workspace_bytes(2, 8, 2, 8, 16, 128) == 16  # one launch, nothing kept
    long = _changed(ok, {10: 64, 15: 20})  # 20 splits of 1,024 tokens
    need = sl8.sparse_decode_workspace_bytes(2, 8, 2, 64, 16, 128, 20)
    assert need >= 2 * 8 * 129 * 4 * 16
    for change in ({20: need - 1}, {19: None}, {19: p + 8}):
        assert f(*_changed(long, change)) == WORKSPACE, change
    size = lib.sl8_attn_int8_sparse_decode_workspace_size
    assert size(2, 8, 2, 8, 24, 128, 0) == 0 and size(0, 8, 2, 8, 16, 128, 0) == 0 and size(2, 7, 2, 8, 16, 128, 0) == 0
    assert size(1, 8, 1, 1 << 22, 16, 128, 1 << 21) == 0  # more than 65,535 splits
    # more splits need more room
    assert size(1, 8, 1, 512, 64, 128, 64) > size(1, 8, 1, 512, 64, 128, 9) > 16


def test_binding_refuses_cpu_tensors(lib):
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        sl8.paged_assign(i, i, i.view(4, 1), i, i[:1], 16, 8)
    k = torch.zeros(2, 1, 64)
    pages, scales = torch.zeros(1, 1, 16, 64, dtype=torch.int8), torch.zeros(1, 1, 16)
    with pytest.raises(ValueError):
        sl8.rope_append(None, k, k, None, None, i[:2], pages, scales, pages, scales)
    with pytest.raises(ValueError):
        sl8.page_bounds(pages, scales, i.view(1, 4), i[:1], torch.zeros(1, 1, 2, 64, dtype=torch.int8), torch.zeros(1, 1))
    with pytest.raises(ValueError):
        sl8.attn_int8_sparse_decode(k, pages, scales, pages, scales, i.view(2, 1, 2), i[:2].view(2, 1))


def test_tables_and_lists_of_almost_2_31_tokens_are_refused(lib, p):
    """Counters that step past the last token stay below 2^31."""
    full, fits = (1 << 27) - 8, (1 << 27) - 16  # pages of 16 tokens: 2^31 - 128 and 2^31 - 256
    assign = [p, p, None, 0, 16, fits, p, p, 8, p, p, 8, p, p, p, p, None, None]
    bounds = [p, p, 16, 16, p, fits, p, p, 4, 0, 1, 32, p, p, None]
    select = [p, sl8.SL8_BF16, p, p, 16, 16, p, fits, p, 0, 1, 1, 1, 32, 8, 1, 2, p, p, p, p, None]
    size = lib.sl8_attn_int8_sparse_decode_workspace_size
    assert lib.sl8_paged_assign(*_changed(assign, {5: full})) == UNSUPPORTED
    assert lib.sl8_page_bounds(*bounds) == OK and lib.sl8_page_bounds(*_changed(bounds, {5: full})) == UNSUPPORTED
    assert lib.sl8_page_select(*select) == OK
    for i in (7, 14):
        assert lib.sl8_page_select(*_changed(select, {i: full})) == UNSUPPORTED
    assert size(1, 1, 1, fits, 16, 32, 1) == 16 and size(1, 1, 1, full, 16, 32, 1) == 0


def test_the_longest_lists_have_a_split_plan(lib):
    """Lists up to the limit are split as shorter ones are, for every number of splits."""
    size = lib.sl8_attn_int8_sparse_decode_workspace_size
    fits = (1 << 27) - 16  # pages of 16 tokens: 2^31 - 256
    assert size(1, 1, 1, fits, 16, 32, 0) >= 16
    for splits in (9, 64, 300, 4096, 65535):
        assert size(1, 1, 1, fits, 16, 32, splits) > 16, splits
        n = lib.sl8_attn_decode_num_splits(1, 1, fits * 16, 32, splits)
        ss = lib.sl8_attn_decode_split_size(1, 1, fits * 16, 32, splits)
        assert n > 0 and (n - 1) * ss < fits * 16 <= n * ss and ss % 16 == 0
    # the arithmetic of lengths that never came near 2^31 is what it was
    for L in (1, 15, 16, 17, 159, 160, 161, 4096, 100000, 1 << 20):
        for splits in (1, 2, 7, 64, 1000):
            n = lib.sl8_attn_decode_num_splits(3, 2, L, 64, splits)
            ss = lib.sl8_attn_decode_split_size(3, 2, L, 64, splits)
            assert 1 <= n <= splits and (n - 1) * ss < L <= n * ss
