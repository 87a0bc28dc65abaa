"""Refusals of the 4-bit cache's entry points (no GPU needed): every argument error returns its
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


def test_rope_append(lib, p):
    f = lib.sl8_rope_append_int4
    axis = bytes([0] * 32 + [1] * 32)
    #    0  1  2  3             4     5    6    7  8  9  10   11 12 13   14 15    16 17 18   19 20    21 22 23 24 25  26  27
    ok = [p, p, p, sl8.SL8_BF16, 4096, 512, 512, 4, 8, 4, 128, p, 2, 128, p, axis, 0, p, 1024, p, None, p, p, p, p, 16, 16, None]
    assert f(*_changed(ok, {7: 0})) == OK                       # nothing to do
    for i in (0, 1, 2, 11, 14, 17, 19, 21, 22, 23, 24):
        assert f(*_changed(ok, {i: None})) == INVALID, i
    for i, v in ((3, sl8.SL8_I8), (4, 1000), (5, 511), (6, 508), (18, 1020), (7, -1), (8, -1), (9, 0), (25, 0), (26, 0),
                 (13, 136), (0, p + 8), (21, p + 4), (22, p + 2), (24, p + 8), (20, p + 4), (15, None), (15, bytes([2] * 64)),
                 (12, 0)):
        assert f(*_changed(ok, {i: v})) == INVALID, (i, v)
    for change in ({10: 96, 13: 96}, {13: 100}, {12: 5}, {25: 1 << 20, 26: 1 << 12}):
        assert f(*_changed(ok, change)) == UNSUPPORTED, change
    # fp32 rows advance in 16 bytes: 4 elements
    assert f(*_changed(ok, {3: sl8.SL8_F32, 5: 514})) == INVALID


def test_paged_read(lib, p):
    f = lib.sl8_paged_read_int4
    #    0  1  2  3  4   5   6  7  8  9     10 11 12 13   14 15    16 17 18            19
    ok = [p, p, p, p, 16, 16, p, 8, p, None, 4, 2, 64, 128, 0, None, p, p, sl8.SL8_BF16, None]
    for change in ({10: 0}, {12: 0}, {9: p, 14: 0}):
        assert f(*_changed(ok, change)) == OK, change
    for i in (0, 1, 2, 3, 6, 8):
        assert f(*_changed(ok, {i: None})) == INVALID, i
    assert f(*_changed(ok, {16: None, 17: None})) == INVALID
    for change in ({4: 0}, {5: 0}, {7: 0}, {10: -1}, {11: 0}, {12: -1}, {9: p, 14: -1}, {18: sl8.SL8_I8}, {0: p + 4}, {1: p + 2},
                   {2: p + 8}, {3: p + 8}, {15: p + 4}, {16: p + 8}, {17: p + 2}):
        assert f(*_changed(ok, change)) == INVALID, change
    for change in ({13: 96}, {5: 1 << 16, 7: 1 << 15}, {4: 1 << 20, 5: 1 << 12}, {12: (1 << 31) - 128}, {10: 1 << 20, 11: 64, 12: 4096}):
        assert f(*_changed(ok, change)) == UNSUPPORTED, change


def test_paged_decode(lib, p):
    f = lib.sl8_attn_int4_paged_decode
    #    0  1             2  3  4  5  6   7   8  9  10 11   12 13 14 15 16   17 18 19            20    21 22       23
    ok = [p, sl8.SL8_BF16, p, p, p, p, 16, 16, p, 8, p, None, 1, 2, 8, 2, 128, 0, p, sl8.SL8_BF16, None, p, 1 << 30, None]
    assert f(*_changed(ok, {13: 0})) == OK
    for i in (0, 2, 3, 4, 5, 8, 10, 18):
        assert f(*_changed(ok, {i: None})) == INVALID, i
    for change in ({1: sl8.SL8_I8}, {19: sl8.SL8_I8}, {6: 0}, {7: 0}, {9: 0}, {12: 0}, {13: -1}, {14: 7}, {15: 0}, {17: -1}, {0: p + 4},
                   {2: p + 4}, {3: p + 2}, {4: p + 8}, {5: p + 8}):
        assert f(*_changed(ok, change)) == INVALID, change
    for change in ({16: 96}, {7: 24}, {12: 33}, {6: 1 << 20, 7: 1 << 12}, {7: 16, 9: (1 << 27) - 8}, {13: 1 << 24, 12: 32}):
        assert f(*_changed(ok, change)) == UNSUPPORTED, change
    size = lib.sl8_attn_int4_paged_decode_workspace_size
    assert size(2, 1, 8, 2, 8, 16, 128, 8) == 16  # one launch, nothing kept
    long = _changed(ok, {9: 64, 17: 20})
    need = size(2, 1, 8, 2, 64, 16, 128, 20)
    assert need > 2 * 8 * 130 * 4 * 2  # two parts of eight columns for several CTAs at least
    for change in ({22: need - 1}, {21: None}, {21: p + 8}):
        assert f(*_changed(long, change)) == WORKSPACE, change
    for args in ((2, 1, 8, 2, 8, 24, 128, 0), (0, 1, 8, 2, 8, 16, 128, 0), (2, 1, 7, 2, 8, 16, 128, 0), (2, 33, 8, 2, 8, 16, 128, 0),
                 (2, 0, 8, 2, 8, 16, 128, 0), (2, 1, 8, 2, 0, 16, 128, 0), (2, 1, 8, 2, 8, 16, 96, 0), (2, 1, 8, 2, 8, 16, 128, -1),
                 (1, 1, 1, 1, (1 << 27) - 8, 16, 32, 1)):
        assert size(*args) == 0, args
    assert size(1, 1, 1, 1, (1 << 27) - 16, 16, 32, 1) == 16
    # more splits need more room, up to a few CTAs for each place on the device
    assert size(1, 1, 8, 1, 512, 64, 128, 1 << 30) >= size(1, 1, 8, 1, 512, 64, 128, 12) > size(1, 1, 8, 1, 512, 64, 128, 9) > 16
    assert size(1, 1, 8, 1, 512, 64, 128, 1 << 30) == size(1, 1, 8, 1, 512, 64, 128, 1 << 29)
    assert size(1, 1, 16, 1, 512, 64, 128, 9) > size(1, 1, 8, 1, 512, 64, 128, 9)  # 16 columns a part instead of 8


def _pool(d=64, page=16):
    codes, scales = torch.zeros((1, 1, page, d // 2), dtype=torch.uint8), torch.zeros((1, 1, page, d // 32), dtype=torch.bfloat16)
    return codes, scales, codes.clone(), scales.clone()


def test_binding_refuses_cpu_tensors(lib):
    i = torch.zeros(4, dtype=torch.int32)
    k = torch.zeros(2, 1, 64)
    with pytest.raises(ValueError):
        sl8.rope_append_int4(None, k, k, None, None, i[:2], *_pool())
    with pytest.raises(ValueError):
        sl8.paged_read_int4(*_pool(), i.view(1, 4), i[:1])
    with pytest.raises(ValueError):
        sl8.attn_int4_paged_decode(torch.zeros(1, 2, 64), *_pool(), i.view(1, 4), i[:1])
