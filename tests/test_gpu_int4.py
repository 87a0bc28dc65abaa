"""The paged 4-bit cache on the GPU, against its CPU definitions: the rotary append, reading it back
and decode attention over its pages, alone and as one serving step.

Tolerances.  Codes and scales of rows that do not turn are fixed bit for bit.  Rotations are within
2e-6 of a pair's length (the append's bound, as for the int8 pages), so a scale is a bf16 rounding
of something that near, and a stored value within half a step of it.  Values read back take one fma
and one rounding to their type.

Attention, for n tokens and kN = d / 32 groups (2^-24 is half a step of fp32):
  a logit takes kN fused sums, the scale of q and log2 e, and the reference comes off: (kN + 4) 2^-24 of
  sum |q k| / sqrt(d), in units of log2 1.45 times that; exponentials are good to 2^-22; so each p to
    ep = 1.45 (kN + 4) 2^-24 reach + 2^-22, and the quotient by their sum to twice that;
  weights p s_v of fp32 outputs are off by 2^-23 of themselves (three bf16 terms, the product's rounding); those of
  16-bit outputs are fp16 numbers of the product in fp32: 2^-11 + 2^-23 of themselves, or half of 2^-24 on a scale on
  which the largest of the query is at least 1/2: 2^-24 of that one, times |code| <= 8, for each token;
  sums: each MMA's addition may truncate (2^-23 of the partial sum), at most 3 an m16n8k16 step and 16 tokens,
  and some thirty in merges: (3 n / 16 + 32) 2^-23.
All of these are relative to sum_t p_t |v_t|; probabilities below 2^-126 of the largest may be 0; then half a
step of the output's type.
"""
import numpy as np
import pytest
import torch

import oracle
import w8a8_int8_flashattention_gb300 as sl8
from _parity import check_f32
from oracle import int4 as Q
from oracle import serving as S

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from w8a8_int8_flashattention_gb300 import build
    build.build()
    sl8.lib()


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    st, site = sl8.last_device_status()
    assert st == sl8.SL8_OK, (st, site)


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)


def np64(t):
    return t.detach().double().cpu().numpy()


def f32(t):
    return t.detach().float().cpu().numpy()


def _pool(num_pages, hkv, page, d, fill=True):
    """k_pages, k_scale_pages, v_pages, v_scale_pages; filled with bytes that no test writes."""
    p = sl8.int4_pages(num_pages, hkv, page, d, DEV)
    if fill:
        p[0].fill_(0x5a), p[2].fill_(0x5a), p[1].fill_(-7.0), p[3].fill_(-7.0)
    return p


# ------------------------------------------------------------------ rotary append

def _pair_length(x, rot, adjacent):
    """Each rotated channel's pair length; 0 for the others."""
    t = np.zeros_like(x)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if adjacent else (slice(0, rot // 2), slice(rot // 2, rot))
    t[..., a] = t[..., b] = np.hypot(x[..., a], x[..., b])
    return t


def _check_keys(codes, scales, want, tol, tag=""):
    """Stored rows [n, d] against exact keys that the kernel knows to within tol."""
    lo = np.maximum(np.abs(want) - tol, 0).reshape(*want.shape[:-1], -1, 32).max(-1)
    hi = (np.abs(want) + tol).reshape(*want.shape[:-1], -1, 32).max(-1)
    # two roundings to fp32 (the maximum, the division) before the one to bf16
    assert np.all(Q.to_bf16((lo / 7 * (1 - 2.0 ** -22)).astype(np.float32)) <= scales), tag
    assert np.all(scales <= Q.to_bf16((hi / 7 * (1 + 2.0 ** -22)).astype(np.float32))), tag
    step = np.repeat(scales.astype(np.float64), 32, -1)
    assert np.abs(codes).max() <= 7
    assert np.all(np.abs(codes * step - want) <= step * 0.5 + tol), tag


@pytest.mark.parametrize("d,rot,axes,adjacent,hq,hkv,dtype,T,page,mean", [
    (128, 128, 1, False, 32, 8, torch.bfloat16, 1, 16, False), (128, 96, 3, False, 5, 1, torch.float16, 37, 16, True),
    (64, 64, 1, True, 7, 3, torch.bfloat16, 130, 7, True), (32, 8, 2, False, 3, 3, torch.float32, 65, 32, False),
    (256, 256, 4, True, 2, 2, torch.float32, 9, 16, True), (256, 64, 1, False, 16, 8, torch.float16, 700, 64, False),
    (256, 256, 1, False, 2, 1, torch.bfloat16, 33, 16, False), (256, 208, 2, False, 2, 3, torch.float32, 33, 16, True),
    (64, 56, 1, False, 1, 5, torch.float32, 40, 16, False), (64, 24, 1, False, 2, 2, torch.bfloat16, 40, 16, True),
    (32, 32, 1, False, 4, 9, torch.float32, 21, 5, True), (32, 32, 1, True, 1, 1, torch.float16, 2000, 1000, False),
    (64, 0, 0, False, 2, 2, torch.bfloat16, 20, 16, False), (128, 128, 1, False, 0, 2, torch.bfloat16, 20, 16, True)])
def test_rope_append(d, rot, axes, adjacent, hq, hkv, dtype, T, page, mean):
    g = torch.Generator().manual_seed(T + d)
    rng = np.random.default_rng(T)
    qkv = torch.randn((T, (hq + 2 * hkv) * d + 16), generator=g).to(dtype)
    qkv[T // 2, -1 - 16 - d:-16] = 0  # part of a row of zeros
    qkv[:, hq * d:(hq + 1) * d] *= 30
    dq = qkv.to(DEV)
    view = lambda x, a, n: x[:, a * d:(a + n) * d].unflatten(1, (n, d)) if n else None  # noqa: E731
    q, k, v = view(dq, 0, hq), view(dq, hq, hkv), view(dq, hq + hkv, hkv)
    pos = rng.integers(0, 1 << 20, (max(axes, 1), T))
    pos[:, -1] = (1 << 31) - 1 - np.arange(max(axes, 1))
    pos[:, 0] = -5 if T > 1 else 3
    inv = (10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)
    axis = rng.integers(0, max(axes, 1), rot // 2).tolist()
    num_pages = -(-T // page) + 1
    slots = rng.permutation(num_pages * page)[:T]
    if T > 4:
        slots[[1, 3]] = -1
    off = rng.standard_normal((hkv, d)).astype(np.float32) * 2 if mean else np.zeros((hkv, d), np.float32)
    pool = _pool(num_pages, hkv, page, d)
    out = sl8.rope_append_int4(q, k, v, i32(pos if axes > 1 else pos[0]) if rot else None,
                               torch.from_numpy(inv).to(DEV) if rot else None, i32(slots), *pool,
                               pair_axis=axis if axes > 1 else None, adjacent=adjacent,
                               k_mean=torch.from_numpy(off).to(DEV) if mean else None)
    host = qkv.double().numpy()
    eps = torch.finfo(dtype).eps / 2
    used = axis if axes > 1 else None
    if hq:
        x = host[:, :hq * d].reshape(T, hq, d)
        want = S.rope(x, pos, inv, used, adjacent)
        # a value rounds from within the rotation's error; tiny fp16 results round to 2^-25
        assert np.all(np.abs(np64(out) - want) <= 2e-6 * _pair_length(x, rot, adjacent) * (1 + eps) + eps * np.abs(want) + 2.0 ** -25)
    kx = host[:, hq * d:(hq + hkv) * d].reshape(T, hkv, d)
    turned = S.rope(kx, pos, inv, used, adjacent)
    tol = 2e-6 * _pair_length(kx, rot, adjacent) + (2.0 ** -24 * (np.abs(turned) + np.abs(off)) if mean else 0.0)
    want = turned - off
    vc, vs = Q.quant4(host[:, (hq + hkv) * d:(hq + 2 * hkv) * d].reshape(T, hkv, d).astype(np.float32))
    gk, gv = (Q.unpack(pool[i].cpu().numpy()) for i in (0, 2))
    ks, gs = f32(pool[1]), f32(pool[3])
    touched = np.zeros((num_pages, page), bool)
    for t in range(T):
        if slots[t] < 0:
            continue
        at = slots[t] // page, slice(None), slots[t] % page
        touched[at[0], at[2]] = True
        np.testing.assert_array_equal(gv[at], vc[t])
        np.testing.assert_array_equal(gs[at], vs[t])
        _check_keys(gk[at], ks[at], want[t], tol[t], t)
    # rows without a slot stay as they were
    for x, was in zip(pool, (0x5a, -7.0, 0x5a, -7.0)):
        assert bool((x.transpose(1, 2)[torch.from_numpy(~touched).to(DEV)] == was).all())


def test_stored_rows_are_the_definitions():
    """The bits of the definition on values that sit on rounding borders, on tiny and huge rows and
    groups; a group with an infinity gets the scale inf and codes 0, a NaN the code 0."""
    g = torch.Generator().manual_seed(9)
    T, hkv, d = 512, 4, 64
    v = torch.randn((T, hkv, d), generator=g)
    v[0:64] = torch.randint(-14, 15, (64, hkv, d), generator=g).float() / 2  # halves of a step of 1
    v[0:64, :, 0] = v[0:64, :, 40] = 7.0
    v[64:128] *= torch.logspace(-44, 37, 64)[:, None, None]
    v[128:192] = torch.randint(-14, 15, (64, hkv, d), generator=g).float() / 2 * (1 + 2.0 ** -23)
    v[128:192, :, 1] = v[128:192, :, 33] = -7.0
    v[192, :, 3], v[193, :, 3], v[194, :, 3] = float("inf"), float("-inf"), float("nan")
    v[195, :, 3], v[195, :, 9] = float("nan"), float("inf")
    v[196] = float("nan")
    v[197] = 0
    v[198:262, :, :32] *= torch.logspace(-38, 30, 64)[:, None, None]  # groups of one row far apart
    v[262:290] = torch.randn((28, hkv, d), generator=g) * (2.0 ** -torch.arange(120.0, 148.0))[:, None, None]
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        x = v.to(dtype).to(DEV)
        pool = _pool(1, hkv, T, d)
        sl8.rope_append_int4(None, x, x, None, None, i32(np.arange(T)), *pool)
        want, s = Q.quant4(x.float().cpu().numpy())
        for i in (0, 2):
            np.testing.assert_array_equal(Q.unpack(pool[i][0].transpose(0, 1).cpu().numpy()), want)
            np.testing.assert_array_equal(f32(pool[i + 1][0].transpose(0, 1)), s)


def test_append_in_place_and_a_bad_slot():
    T, hq, hkv, d = 6, 4, 2, 64
    qkv = torch.randn((T, (hq + 2 * hkv) * d), device=DEV).half()
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    pos, inv = torch.arange(T, dtype=torch.int32, device=DEV), torch.rand(d // 2, device=DEV)
    pool = sl8.int4_pages(2, hkv, 4, d, DEV)
    want = sl8.rope_append_int4(q, k, v, pos, inv, i32([0, 1, 2, 8, -3, 5]), *pool)  # slot 8 lies past the two pages
    assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
    kept = k.clone()
    got = sl8.rope_append_int4(q, k, v, pos, inv, i32([0, 1, 2, -1, -3, 5]), *pool, q_out=q)
    assert got.data_ptr() == qkv.data_ptr() and torch.equal(got, want) and torch.equal(k, kept)
    assert int((pool[1][..., 0] != 0).sum()) == 4 * hkv
    # both appends turn q alike
    codes, scales = torch.zeros((2, 2, hkv, 4, d), dtype=torch.int8, device=DEV), torch.zeros((2, 2, hkv, 4), device=DEV)
    q8 = torch.randn((T, hq, d), device=DEV)
    a = sl8.rope_append(q8, k.float(), v.float(), pos, inv, i32([0, 1, 2, -1, -3, 5]), codes[0], scales[0], codes[1], scales[1])
    b = sl8.rope_append_int4(q8, k.float(), v.float(), pos, inv, i32([0, 1, 2, -1, -3, 5]), *pool)
    assert torch.equal(a, b)


# ------------------------------------------------------------------ reading back

def _filled(rng, num_pages, hkv, page, d, spread=1.0):
    """A pool of random codes (-8 among them) and scales up to `spread` powers of ten apart."""
    pool = _pool(num_pages, hkv, page, d)
    host = []
    for i in (0, 2):
        c = rng.integers(0, 256, tuple(pool[i].shape)).astype(np.uint8)
        s = Q.to_bf16((10.0 ** rng.uniform(-spread, 0, tuple(pool[i + 1].shape))).astype(np.float32))
        pool[i].copy_(torch.from_numpy(c))
        pool[i + 1].copy_(torch.from_numpy(s))
        host += [c, s]
    return pool, host


def _tables(rng, lens, nb, page, num_pages):
    """Block tables of distinct pages; entries past a sequence's last block name no page."""
    perm, tables, at = rng.permutation(num_pages), np.full((len(lens), nb), -9), 0
    for b, n in enumerate(lens):
        k = -(-n // page)
        tables[b, :k] = perm[at:at + k]
        at += k
    return tables


@pytest.mark.parametrize("d,hkv,page,lens,dtype,mean", [
    (32, 1, 16, [1], torch.float32, False), (64, 3, 7, [50, 0, 13, 64], torch.float16, True),
    (128, 2, 64, [130, 1, 65], torch.bfloat16, True), (256, 8, 16, [33, 70], torch.float32, True),
    (128, 1, 300, [299, 300, 301], torch.bfloat16, False), (256, 2, 1, [5, 3], torch.float16, False)])
def test_read(d, hkv, page, lens, dtype, mean):
    rng = np.random.default_rng(d + page)
    B, nb = len(lens), -(-max(lens) // page) + 1
    num_pages = sum(-(-n // page) for n in lens) + 2
    pool, (kc, ks, vc, vs) = _filled(rng, num_pages, hkv, page, d)
    tables = _tables(rng, lens, nb, page, num_pages)
    off = rng.standard_normal((hkv, d)).astype(np.float32) if mean else np.zeros((hkv, d), np.float32)
    km = torch.from_numpy(off).to(DEV) if mean else None
    N = max(lens) + 3
    ko, vo = (torch.full((B, hkv, N, d), 5.0, dtype=dtype, device=DEV) for _ in range(2))
    got = sl8.paged_read_int4(*pool, i32(tables), i32(lens), max_seqlen=N, k_mean=km, k_out=ko, v_out=vo)
    assert got[0] is ko and got[1] is vo
    room = 4
    cu = np.concatenate([[0], np.cumsum(np.array(lens) + room)])
    pk, pv = sl8.paged_read_int4(*pool, i32(tables), i32(lens), cu_seqlens=i32(cu), max_seqlen=N, total_tokens=int(cu[-1]) + 2,
                                 k_mean=km, out_dtype=dtype)
    eps = torch.finfo(dtype).eps / 2
    for b, n in enumerate(lens):
        for dense, packed, c, s, o in ((ko, pk, kc, ks, off), (vo, pv, vc, vs, np.zeros_like(off))):
            want = Q.values(Q.gather(c, tables[b], n), Q.gather(s, tables[b], n)) + o[:, None]
            # the fma's rounding to fp32, then the type's; fp16 below 2^-14 rounds to 2^-25
            tol = np.abs(want) * (2.0 ** -24 * (1 + eps) + eps) + (2.0 ** -25 if dtype == torch.float16 else 0)
            assert np.all(np.abs(np64(dense[b, :, :n]) - want) <= tol), b
            assert bool((dense[b, :, n:] == 5.0).all())
            rows = packed[cu[b]:cu[b + 1]].transpose(0, 1)
            assert torch.equal(rows[:, :n], dense[b, :, :n]) and bool((rows[:, n:] == 0).all())
    # without a length bound the table's width counts
    wide, _ = sl8.paged_read_int4(*pool, i32(tables), i32(lens), k_mean=km, out_dtype=dtype)
    assert wide.shape == (B, hkv, nb * page, d) and torch.equal(wide[:, :, :min(N, nb * page)][:, :, :max(lens)][0, :, :lens[0]], ko[0, :, :lens[0]])


def test_read_reports_what_is_out_of_range():
    rng = np.random.default_rng(1)
    pool, (kc, ks, _, _) = _filled(rng, 4, 1, 16, 32)
    bad = lambda: sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG  # noqa: E731
    out = lambda n: torch.full((1, 1, n, 32), 9.0, device=DEV)  # noqa: E731
    table = i32([[2, 1]])
    for n, N, rows in ((-1, 20, 0), (33, 40, 32), (25, 20, 20)):
        k, v = out(N), out(N)
        sl8.paged_read_int4(*pool, table, i32([n]), max_seqlen=N, k_out=k, v_out=v)
        assert bad()
        assert bool((k[:, :, rows:] == 9).all())
        np.testing.assert_array_equal(f32(k[0, :, :rows]), Q.values(Q.gather(kc, [2, 1], rows), Q.gather(ks, [2, 1], rows)).astype(np.float32))
    for page in (-1, 4):  # read as page 0
        k, _ = sl8.paged_read_int4(*pool, i32([[2, page]]), i32([20]), out_dtype=torch.float32)
        assert bad()
        np.testing.assert_array_equal(f32(k[0, :, 16:20]), Q.values(kc[0, :, :4], ks[0, :, :4]).astype(np.float32))
    for cu, rows in (([0, 10], 10), ([3, 30], 9), ([-1, 30], 0), ([0, -5], 0), ([12, 30], 0)):
        k, v = (torch.full((12, 1, 32), 9.0, device=DEV) for _ in range(2))
        sl8.paged_read_int4(*pool, table, i32([20]), cu_seqlens=i32(cu), max_seqlen=32, k_out=k, v_out=v)
        assert bad(), cu
        first = max(cu[0], 0)
        assert bool((k[:first] == 9).all()) and bool((k[first + rows:] == 9).all()), cu
        np.testing.assert_array_equal(f32(k[first:first + rows, 0]), Q.values(Q.gather(kc, [2, 1], rows), Q.gather(ks, [2, 1], rows))[0].astype(np.float32))


def test_read_of_infinite_groups_and_what_was_appended():
    T, hkv, d = 20, 2, 64
    x = torch.randn((T, hkv, d), device=DEV)
    x[3, 0, 5], x[4, 1, 40] = float("inf"), float("nan")
    pool = sl8.int4_pages(2, hkv, 16, d, DEV)
    sl8.rope_append_int4(None, x, x, None, None, i32(np.arange(T)), *pool)
    k, v = sl8.paged_read_int4(*pool, i32([[0, 1]]), i32([T]), max_seqlen=T, out_dtype=torch.float32)
    assert torch.equal(torch.isnan(k[0, 0, 3]), torch.arange(d, device=DEV) < 32) and k[0, 1, 4, 40] == 0
    ok = torch.isfinite(k[0].transpose(0, 1)) & torch.isfinite(x)
    step = x.unflatten(-1, (-1, 32)).nan_to_num(0.0, 0.0, 0.0).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2) / 7 * (1 + 2.0 ** -8)
    assert bool(((k[0].transpose(0, 1) - x).abs() <= step * 0.5)[ok].all()) and torch.equal(k.nan_to_num(), v.nan_to_num())


# ------------------------------------------------------------------ decode attention

def _check_attention(out, lse, q, host, tables, lens, masks=None, tag=""):
    """out [B,T,Hq,d], lse [B,T,Hq] against the definition with the bounds above."""
    want, wlse, size, reach, heavy = Q.attention(f32(q), *host, tables, lens, masks, bounds=True)
    n, groups = max(int(np.max(lens)), 1), q.shape[-1] // 32
    ep = 1.45 * (groups + 4) * 2.0 ** -24 * reach + 2.0 ** -22
    ew, floor = (2.0 ** -23, 0.0) if out.dtype == torch.float32 else (2.0 ** -11 + 2.0 ** -23, 2.0 ** -24 * 8 * n)
    rel = 2 * ep[..., None] + ew + (3 * n / 16 + 32) * 2.0 ** -23
    eps = torch.finfo(out.dtype).eps / 2
    got = np64(out)
    assert np.all(np.isfinite(got)), tag
    gone = 2.0 ** -126 * 8 * n * np.max(np.where(np.isfinite(host[3]), np.abs(host[3]), 0))
    tol = (size * rel + floor * heavy[..., None] + gone) * (1 + eps) + eps * np.abs(want) + (2.0 ** -25 if out.dtype == torch.float16 else 0)
    worst = np.max((np.abs(got - want) - tol))
    assert worst <= 0, (tag, worst, np.max(np.abs(got - want) / np.maximum(tol, 1e-30)))
    empty = np.isinf(wlse)
    gl = np64(lse)
    assert np.all(np.isneginf(gl[empty])), tag
    tl = 2 * ep + (n / 16 + 32) * 2.0 ** -24 + 2.0 ** -23 * (1 + np.abs(np.where(empty, 0, wlse)))
    assert np.all(np.abs(gl[~empty] - wlse[~empty]) <= tl[~empty]), tag


def _attend(B, T, hq, hkv, d, page, lens, qdt, odt, splits=0, tree=False, spread=1.0, seed=0, workspace=None, nb=None):
    rng = np.random.default_rng(seed + d + 7 * T)
    nb = nb or -(-max(max(lens), 1) // page) + 1
    num_pages = sum(-(-n // page) for n in lens) + 2
    pool, host = _filled(rng, num_pages, hkv, page, d, spread)
    tables = _tables(rng, lens, nb, page, num_pages)
    q = torch.from_numpy(rng.standard_normal((B, T, hq, d)).astype(np.float32)).to(qdt).to(DEV)
    masks = rng.integers(0, 1 << T, (B, T)) if tree else None
    mask = None
    if tree:
        mask = torch.from_numpy(masks.astype(np.uint32).view(np.int32).copy() if T == 32 else masks.astype(np.int32)).to(DEV)
    out, lse = sl8.attn_int4_paged_decode(q if T > 1 else q[:, 0], *pool, i32(tables), i32(lens), tree_mask=mask, num_splits=splits,
                                          out_dtype=odt, return_lse=True, workspace=workspace)
    assert out.dtype == odt and out.shape == (q.shape if T > 1 else q[:, 0].shape)
    _check_attention(out.view(q.shape), lse.view(q.shape[:-1]), q, host, tables, lens, masks, (d, T, splits))


F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("G,hkv,splits,qdt,odt", [
    (1, 1, 0, BF16, BF16), (4, 2, 1, BF16, F32), (8, 1, 2, F16, F16), (16, 2, 3, F32, BF16), (11, 1, 8, BF16, F32), (3, 3, 9, F32, F32),
    (40, 1, 20, F16, F32), (17, 2, 0, BF16, F16)])
def test_decode(d, G, hkv, splits, qdt, odt):
    """Lengths of zero and one, around units and pages, and some hundred tokens."""
    for page, lens in ((16, [0, 1, 15, 16, 17]), (64, [63, 64, 65, 500]), (48, [331, 2])):
        _attend(len(lens), 1, G * hkv, hkv, d, page, lens, qdt, odt, splits, seed=page)


@pytest.mark.parametrize("T,G,hkv,d,splits,tree,odt", [
    (2, 4, 2, 128, 0, False, BF16), (5, 4, 2, 128, 1, True, F32), (7, 1, 2, 64, 3, True, F16), (32, 2, 1, 32, 2, True, F32),
    (32, 1, 1, 256, 12, False, BF16), (31, 3, 1, 64, 0, True, BF16), (4, 16, 1, 128, 5, False, F32), (3, 5, 2, 256, 1, True, F16)])
def test_drafts(T, G, hkv, d, splits, tree, odt):
    """Causal drafts and random trees, among them queries that see nothing; sequences shorter than
    their drafts."""
    lens = [0, 1, T, T + 1, 16, 33, 200 + T]
    _attend(len(lens), T, G * hkv, hkv, d, 16, lens, BF16, odt, splits, tree)


@pytest.mark.parametrize("splits", [0, 1, 5, 64])
def test_a_long_sequence(splits):
    _attend(1, 1, 8, 2, 128, 32, [20011], BF16, F32, splits, spread=0.3)


@pytest.mark.parametrize("d,G", [(32, 4), (64, 16), (128, 2), (256, 8)])
def test_scales_far_apart(d, G):
    """Groups and rows whose scales are far apart: in fp32 each keeps its own relative accuracy, up to 10^12
    apart; 16-bit outputs have the weights' accuracy of the largest."""
    for splits in (1, 4, 10):
        _attend(3, 1, G, 1, d, 16, [90, 7, 300], BF16, F32, splits, spread=12.0)
        _attend(3, 1, G, 1, d, 16, [90, 7, 300], BF16, F16, splits, spread=4.0)


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("splits", [1, 3, 12])
@pytest.mark.parametrize("odt", [BF16, F32])
def test_a_huge_value_row_of_no_weight(odt, splits, d):
    """Rows whose V scales are 2^18 to 2^60 times the others' and whose keys have no probability, first, last and
    in between, and the reverse, a row that has all of it and the least scale: the other weights keep their bits."""
    rng = np.random.default_rng(d + splits)
    L, page, hkv, G = 300, 16, 1, 4
    for factor, kept in ((2.0 ** 18, False), (2.0 ** 60, False), (2.0 ** -40, True)):
        pool, (kc, ks, vc, vs) = _filled(rng, 20, hkv, page, d, 0.3)
        tables = np.arange(20)[None]
        q = torch.from_numpy(np.abs(rng.standard_normal((1, 1, G, d)).astype(np.float32)) + 0.5).to(DEV)
        for row in (0, 97, 160, L - 1) if not kept else (150,):
            at = row // page, 0, row % page
            kc[at] = 0xff if kept else 0x11  # codes 7 or -7 against positive queries
            ks[at] = 4.0 if kept else 16.0
            vs[at] *= factor
        for i, x in enumerate((kc, ks, vc, vs)):
            pool[i].copy_(torch.from_numpy(x))
        out, lse = sl8.attn_int4_paged_decode(q[:, 0], *pool, i32(tables), i32([L]), num_splits=splits, out_dtype=odt, return_lse=True)
        _check_attention(out[:, None], lse[:, None], q, (kc, ks, vc, vs), tables, [L], tag=(factor, kept))


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("splits", [1, 3, 9])
def test_what_lies_past_a_sequence_does_not_matter(d, splits):
    """Infinities and NaN in the scales of rows that a query does not see: past the length, or of a
    draft that its mask hides.  -8 codes and all bytes are codes."""
    rng = np.random.default_rng(5)
    T, hkv, G, page, L = 3, 2, 3, 16, 70
    pool, host = _filled(rng, 8, hkv, page, d)
    tables = _tables(rng, [L], 6, page, 8)
    bad = [float("nan"), float("inf")]
    for row in range(L - 2, 80):  # drafts 1 and 2 and what lies behind them in the last page
        for i, val in ((1, bad[row % 2]), (3, bad[(row + 1) % 2])):
            pool[i][tables[0][row // page], :, row % page] = val
    q = torch.from_numpy(rng.standard_normal((1, T, hkv * G, d)).astype(np.float32)).to(DEV)
    masks = [[0b001, 0b001, 0b000]]
    out, lse = sl8.attn_int4_paged_decode(q, *pool, i32(tables), i32([L]), tree_mask=i32(masks), num_splits=splits, return_lse=True)
    clean = [h.copy() for h in host]
    _check_attention(out, lse, q, clean, tables, [L], masks)
    # a query that sees the NaN scales has no other value
    seen, sl = sl8.attn_int4_paged_decode(q, *pool, i32(tables), i32([L]), tree_mask=i32([[1, 3, 2]]), num_splits=splits, return_lse=True)
    assert torch.equal(seen[:, 0], out[:, 0]) and torch.isnan(sl[:, 1:]).all() and torch.isnan(seen[:, 1:]).all()


def test_infinite_value_groups_reach_their_channels():
    rng = np.random.default_rng(6)
    d, hkv, page, L = 128, 2, 16, 40
    pool, host = _filled(rng, 4, hkv, page, d)
    tables = _tables(rng, [L], 3, page, 4)
    pool[2][tables[0][1], 1, 3, 16:32] = 0x88  # row 19 of head 1, group 1: codes 0 with the scale inf
    pool[3][tables[0][1], 1, 3, 1] = float("inf")
    q = torch.randn((1, 4, d), device=DEV)
    out, lse = sl8.attn_int4_paged_decode(q, *pool, i32(tables), i32([L]), return_lse=True)
    nan = torch.isnan(out[0])
    assert not nan[:2].any() and nan[2:, 32:64].all() and not nan[2:, :32].any() and not nan[2:, 64:].any()
    assert torch.isfinite(lse).all()
    # and a query row with an infinity is NaN, alone
    q[0, 1, 7] = float("inf")
    out2, lse2 = sl8.attn_int4_paged_decode(q, *pool, i32(tables), i32([L]), return_lse=True)
    assert torch.isnan(out2[0, 1]).all() and torch.isnan(lse2[0, 1]) and torch.equal(out2[0, 0], out[0, 0])


@pytest.mark.parametrize("splits", [0, 1, 3, 8, 9, 40])
@pytest.mark.parametrize("d,odt", [(32, F32), (64, BF16), (128, F16), (256, F32)])
def test_nan_logits_reach_the_output(d, odt, splits):
    """A query row with an infinity, whose logits are all NaN, and keys whose scales are NaN in every row, in all but
    the first, or in the last alone: NaN for the queries that see them; the others as ever (not to the bit: 16-bit outputs' columns
    that share a warp move their references together)."""
    rng = np.random.default_rng(d)
    for L in (30, 2000):
        nb = -(-L // 16)
        pool, host = _filled(rng, 2 * nb, 2, 16, d)
        tables, lens = i32(rng.permutation(2 * nb).reshape(2, nb)), i32([L, L - 3])
        q = torch.randn((2, 6, d), device=DEV)
        call = lambda: sl8.attn_int4_paged_decode(q, *pool, tables, lens, num_splits=splits, out_dtype=odt, return_lse=True)  # noqa: E731
        want, wl = call()
        assert torch.isfinite(want).all() and torch.isfinite(wl).all()
        kept = q[0, 4].clone()
        q[0, 4, d // 2] = float("-inf")
        out, lse = call()
        q[0, 4] = kept
        hit = torch.zeros((2, 6), dtype=torch.bool, device=DEV)
        hit[0, 4] = True
        for rows in (None, slice(None), slice(1, None), slice(L - 4, L - 3)):
            if rows is not None:  # head 1 of the second sequence
                at = torch.arange(nb * 16, device=DEV)[rows]
                scales = pool[1].clone()
                pool[1][tables[1][at // 16].long(), 1, at % 16, -1] = float("nan")
                out, lse = call()
                pool[1].copy_(scales)
                hit = torch.zeros((2, 6), dtype=torch.bool, device=DEV)
                hit[1, 3:] = True
            assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all(), (L, rows)
            rest = torch.where(hit[..., None], want, out), torch.where(hit, wl, lse)
            _check_attention(rest[0][:, None], rest[1][:, None], q[:, None], host, tables.cpu().numpy(), lens.tolist(), tag=(L, rows))


@pytest.mark.parametrize("d,splits", [(32, 1), (64, 0), (128, 1), (128, 8), (256, 2), (128, 12)])
def test_every_row_and_channel_counts(d, splits):
    """Value rows one by one: with the others zero, a row's weight comes out of each of its channels;
    key channels one by one: each moves the logits by its own q."""
    rng = np.random.default_rng(d)
    L, page, hkv, hq = 150, 16, 1, 5
    pool, (kc, ks, vc, vs) = _filled(rng, 10, hkv, page, d)
    tables = np.arange(10)[None]
    q = torch.from_numpy(rng.standard_normal((1, hq, d)).astype(np.float32)).to(DEV)
    for row in (0, 1, 2, 3, 15, 16, 63, 64, 97, 148, 149):
        pool[2].fill_(0x88)
        c = rng.integers(0, 256, d // 2).astype(np.uint8)
        pool[2][row // page, 0, row % page] = torch.from_numpy(c).to(DEV)
        v = np.full_like(vc, 0x88)
        v[row // page, 0, row % page] = c
        out, lse = sl8.attn_int4_paged_decode(q, *pool, i32(tables), i32([L]), num_splits=splits, return_lse=True)
        _check_attention(out[:, None], lse[:, None], q[:, None], (kc, ks, v, vs), tables, [L], tag=row)
    pool[2].copy_(torch.from_numpy(vc))
    for ch in range(0, d, 3):
        one = torch.zeros((1, hq, d), device=DEV)
        one[..., ch] = torch.tensor([3.0, -2.0, 1.0, 0.5, 0.0], device=DEV)
        out, lse = sl8.attn_int4_paged_decode(one, *pool, i32(tables), i32([L]), num_splits=splits, return_lse=True)
        _check_attention(out[:, None], lse[:, None], one[:, None], (kc, ks, vc, vs), tables, [L], tag=ch)


def test_decode_reports_bad_pages_and_lengths():
    rng = np.random.default_rng(8)
    pool, host = _filled(rng, 4, 1, 16, 64)
    q = torch.randn((1, 1, 2, 64), device=DEV)
    for tables, lens, as_tables, as_lens in (([[2, 7]], [30], [[2, 0]], [30]), ([[2, -1]], [30], [[2, 0]], [30]), ([[2, 1]], [33], [[2, 1]], [32]),
                                             ([[2, 1]], [-4], [[2, 1]], [0])):
        for splits in (1, 4, 9):
            out, lse = sl8.attn_int4_paged_decode(q, *pool, i32(tables), i32(lens), num_splits=splits, return_lse=True)
            assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
            _check_attention(out, lse, q, host, as_tables, as_lens)


def test_the_same_bits_every_time_and_shared_pages():
    rng = np.random.default_rng(9)
    pool, host = _filled(rng, 6, 2, 32, 128)
    tables, lens = [[1, 2, 3], [1, 2, 5], [4, 4, 4]], [90, 70, 96]
    q = torch.randn((3, 8, 128), device=DEV).bfloat16()
    for splits in (0, 2, 12):
        a = sl8.attn_int4_paged_decode(q, *pool, i32(tables), i32(lens), num_splits=splits, return_lse=True)
        for _ in range(3):
            b = sl8.attn_int4_paged_decode(q, *pool, i32(tables), i32(lens), num_splits=splits, return_lse=True)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        _check_attention(a[0][:, None], a[1][:, None], q[:, None], host, tables, lens)


@pytest.mark.parametrize("splits", [0, 1, 9])
@pytest.mark.parametrize("d,cols", [(32, 7), (32, 9), (32, 24), (32, 25), (32, 64), (64, 8), (64, 17), (64, 23), (64, 49), (128, 15), (128, 16),
                                    (128, 25), (128, 33), (128, 48), (256, 9), (256, 17)])
def test_columns_of_heads_and_drafts(d, cols, splits):
    """Drafts times query heads around what a tile and a CTA take, with one draft or one head, or both."""
    for T, G in ((1, cols), (cols, 1)) + (((cols // 3, 3),) if cols % 3 == 0 else ()) + (((cols // 8, 8),) if cols % 8 == 0 else ()):
        if T <= 32:
            _attend(2, T, 2 * G, 2, d, 16, [T + 40, 9], BF16, F32 if cols % 2 else BF16, splits, tree=T > 1, seed=cols)


@pytest.mark.parametrize("B,T,G,hkv,d,width,odt", [
    (64, 1, 4, 2, 128, 16384, BF16), (700, 1, 3, 1, 64, 8192, F32), (5000, 1, 1, 1, 32, 1024, F16), (130, 1, 20, 1, 64, 8192, BF16),
    (257, 4, 2, 1, 128, 8192, F32), (129, 1, 2, 2, 256, 4096, BF16), (40, 32, 1, 1, 32, 32768, BF16)])
def test_many_sequences_of_uneven_lengths_in_a_wide_table(B, T, G, hkv, d, width, odt):
    """The work cut evenly among CTAs, where most sequences are empty or short and one is long: shares that hold
    many sequences, a part of one, the end of one and the start of another; then none with a token."""
    assert sl8.int4_decode_workspace_bytes(B, T, G * hkv, hkv, width // 16, 16, d) > 16  # the shares' parts
    rng = np.random.default_rng(B)
    lens = rng.choice([0, 0, 0, 1, 2, 15, 16, 17, 33, 70], B)
    lens[rng.integers(0, B, 3)] = 200
    lens[B // 2] = min(width, 3001)
    lens[-1] = 5
    _attend(B, T, G * hkv, hkv, d, 16, lens.tolist(), BF16, odt, nb=width // 16)
    _attend(B, T, G * hkv, hkv, d, 16, [0] * B, BF16, odt, nb=width // 16)
    _attend(B, T, G * hkv, hkv, d, 16, [0] * (B - 1) + [width], BF16, odt, nb=width // 16) if width <= 4096 else None


def test_rows_and_columns_of_the_workspace_are_not_read_before_they_are_written():
    """A workspace of NaN, and one that a call of another shape has left: the same bits."""
    rng = np.random.default_rng(12)
    pool, host = _filled(rng, 80, 2, 16, 64)
    tables, lens = i32(rng.permutation(80).reshape(4, 20)), i32([320, 0, 17, 150])
    q = torch.randn((4, 6, 64), device=DEV).bfloat16()
    for splits in (9, 40, 1 << 20):
        n = sl8.int4_decode_workspace_bytes(4, 1, 6, 2, 20, 16, 64, splits)
        ws = torch.full((n // 4 + 1,), float("nan"), device=DEV).view(torch.uint8)
        a = sl8.attn_int4_paged_decode(q, *pool, tables, lens, num_splits=splits, return_lse=True, workspace=ws)
        ws.view(torch.int32).fill_(7)
        b = sl8.attn_int4_paged_decode(q, *pool, tables, lens, num_splits=splits, return_lse=True, workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        _check_attention(a[0][:, None], a[1][:, None], q[:, None], host, tables.cpu().numpy(), lens.tolist())


def test_offsets_past_32_bits():
    """A pool whose codes pass 2^32 bytes many times, and whose scales do too: its last pages through every operator."""
    hq, hkv, d, page = 8, 8, 128, 64
    num_pages = (1 << 32) // (hkv * page * (d // 32) * 2) + 9
    codes, scales = (num_pages, hkv, page, d // 2), (num_pages, hkv, page, d // 32)
    pool = [torch.empty(s, dtype=t, device=DEV) for _ in range(2) for s, t in ((codes, torch.uint8), (scales, torch.bfloat16))]
    assert pool[1].numel() * 2 > 1 << 32
    ids, n = np.array([num_pages - 1, 3, num_pages - 2, num_pages // 2]), 3 * page + 21
    slots = (ids[:, None] * page + np.arange(page)).reshape(-1)[:n]
    g = torch.Generator().manual_seed(3)
    x = torch.randn((n, 2 * hkv, d), generator=g).bfloat16()
    xd = x.to(DEV)
    sl8.rope_append_int4(None, xd[:, :hkv], xd[:, hkv:], None, None, i32(slots), *pool)
    small = [np.zeros((4, hkv, page, c), t) for _ in range(2) for c, t in ((d // 2, np.uint8), (d // 32, np.float32))]
    c, s = Q.quant4(x.float().numpy())
    for t in range(n):
        for i in range(2):
            small[2 * i][t // page, :, t % page], small[2 * i + 1][t // page, :, t % page] = Q.pack(c[t, i * hkv:(i + 1) * hkv]), s[t, i * hkv:(i + 1) * hkv]
    k, v = sl8.paged_read_int4(*pool, i32(ids[None]), i32([n]), max_seqlen=n, out_dtype=F32)
    for got, i in ((k, 0), (v, 2)):
        np.testing.assert_array_equal(f32(got[0]), Q.values(Q.gather(small[i], range(4), n), Q.gather(small[i + 1], range(4), n)).astype(np.float32))
    q = torch.randn((1, 1, hq, d), generator=g).bfloat16()
    for splits in (1, 9):
        out, lse = sl8.attn_int4_paged_decode(q.to(DEV), *pool, i32(ids[None]), i32([n]), num_splits=splits, out_dtype=F32, return_lse=True)
        _check_attention(out, lse, q, small, [range(4)], [n])


# ------------------------------------------------------------------ one step

def _state(B, hq, hkv, d, page, nb, num_pages, T, mean):
    z = lambda *n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(seq=z(B), new=z(B), release=z(B), table=z(B, nb) - 1, free=torch.arange(num_pages, dtype=torch.int32, device=DEV),
                count=i32([num_pages]), pool=sl8.int4_pages(num_pages, hkv, page, d, DEV), mean=mean,
                qkv=torch.zeros((T, (hq + 2 * hkv) * d), dtype=BF16, device=DEV), dims=(B, hq, hkv, d, page, T))


def _step(s, inv, new, splits=0, plan=None, out=None, workspace=None):
    """One step of one layer: plan, rotary append, attention; with `new` tokens of every sequence as drafts, or, new = 0,
    of its last token."""
    B, hq, hkv, d, page, T = s["dims"]
    plan = sl8.paged_assign(s["seq"], s["new"], s["table"], s["free"], s["count"], page, T, release=s["release"], out=plan)
    s["seq"].copy_(plan["seqlens"])
    s["count"].copy_(plan["free_count"])
    q, k, v = (x.unflatten(1, (-1, d)) for x in s["qkv"].split([hq * d, hkv * d, hkv * d], 1))
    q = sl8.rope_append_int4(q, k, v, plan["token_pos"], inv, plan["slot_map"], *s["pool"], k_mean=s["mean"])
    q = q[:B * new].view(B, new, hq, d) if new else q[(plan["cu_new"][1:] - 1).clamp(min=0).long()][:, None]
    out = sl8.attn_int4_paged_decode(q, *s["pool"], s["table"], s["seq"], num_splits=splits, return_lse=True, workspace=workspace,
                                     out=out and out[0], lse=out and out[1])
    return plan, q, out


@pytest.mark.parametrize("hq,hkv,d,page,splits,with_mean", [(8, 2, 64, 16, 0, True), (12, 2, 128, 32, 9, False), (3, 1, 256, 16, 3, True),
                                                            (25, 1, 32, 48, 0, False)])
def test_a_serving_loop(hq, hkv, d, page, splits, with_mean):
    """Prompts, decode steps, drafts, a release and a new request in its slot.  Each step's attention is the definition's over
    the cache as it stands; what is read back is the tokens' keys and values to half a step of 4 bits; and a prompt's chunk
    and a ragged batch attend over it."""
    B, nb, T = 5, 200 // page + 1, 256
    rng = np.random.default_rng(d)
    mean = rng.standard_normal((hkv, d)).astype(np.float32) if with_mean else np.zeros((hkv, d), np.float32)
    s = _state(B, hq, hkv, d, page, nb, B * nb, T, torch.from_numpy(mean).to(DEV) if with_mean else None)
    freq = (10000.0 ** (-np.arange(0, d, 2) / d)).astype(np.float32)
    inv = torch.from_numpy(freq).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(d)
    rows = [[] for _ in range(B)]  # of each sequence: exact keys, their error, values
    steps = [([60, 33, 1, 100, 0], [0] * 5, 0)] + [([1, 1, 1, 1, 0], [0] * 5, 0)] * 5 + [([1, 20, 1, 1, 16], [0, 1, 0, 0, 0], 0)] + \
            [([1] * 5, [0] * 5, 1)] * 3 + [([4] * 5, [0] * 5, 4)] * 2
    for new, release, drafts in steps:
        s["new"].copy_(i32(new)), s["release"].copy_(i32(release))
        s["qkv"].copy_(torch.randn(s["qkv"].shape, generator=g, device=DEV))
        plan, q, out = _step(s, inv, drafts, splits)
        kv = np64(s["qkv"])[:, hq * d:].reshape(T, 2 * hkv, d)
        at = 0
        for b in range(B):
            if release[b]:
                rows[b] = []
            for _ in range(new[b]):
                x = kv[at:at + 1, :hkv]
                k = S.rope(x, np.array([[len(rows[b])]]), freq)
                err = 2e-6 * _pair_length(x, d, False) + (2.0 ** -24 * (np.abs(k) + np.abs(mean)) if with_mean else 0)
                rows[b].append((k[0], err[0], kv[at, hkv:]))
                at += 1
        lens = s["seq"].tolist()
        assert lens == [len(r) for r in rows]
        host = [s["pool"][0].cpu().numpy(), f32(s["pool"][1]), s["pool"][2].cpu().numpy(), f32(s["pool"][3])]
        _check_attention(*out, q, host, s["table"].cpu().numpy(), lens, tag=lens)
    keys, values = sl8.paged_read_int4(*s["pool"], s["table"], s["seq"], k_mean=s["mean"], out_dtype=F32)
    for b in range(B):
        k, err, v = (np.stack([r[i] for r in rows[b]], 1) for i in range(3))
        for got, want, off, tol in ((keys, k, mean[:, None], err), (values, v, 0.0, np.zeros_like(err))):
            most = (np.abs(want - off) + tol).reshape(*want.shape[:-1], -1, 32).max(-1)
            half = np.repeat(most / 7 * (1 + 2.0 ** -8) * (1 + 2.0 ** -22), 32, -1) / 2
            x = np64(got[b, :, :lens[b]])
            assert np.all(np.abs(x - want) <= half + tol + 2.0 ** -24 * np.abs(x)), b
    # the last 7 tokens of a sequence as a prompt's chunk
    b, n = 3, lens[3]
    k, v = sl8.paged_read_int4(*s["pool"], s["table"][b:b + 1], s["seq"][b:b + 1], max_seqlen=n, k_mean=s["mean"])
    qc = torch.randn((1, hq, 7, d), generator=g, device=DEV).bfloat16()
    o = sl8.attn_int8_fwd_chunk(qc, k, v, out_dtype=F32)
    check_f32(f32(o), oracle.attn_prefill(f32(qc), f32(k), f32(v), causal=True, smooth_k=True)["out"], "chunk")
    # the sequences side by side
    cu = np.concatenate([[0], np.cumsum(lens)])
    k, v = sl8.paged_read_int4(*s["pool"], s["table"], s["seq"], cu_seqlens=i32(cu), max_seqlen=max(lens), total_tokens=int(cu[-1]),
                               k_mean=s["mean"])
    qp = torch.randn((int(cu[-1]), hq, d), generator=g, device=DEV).bfloat16()
    o = sl8.attn_int8_fwd(qp, k, v, cu_seqlens=i32(cu), max_seqlen=max(lens), out_dtype=F32)
    for b in range(B):
        part = [f32(x[cu[b]:cu[b + 1]].transpose(0, 1)[None]) for x in (qp, k, v, o)]
        check_f32(part[3], oracle.attn_prefill(*part[:3], causal=True, smooth_k=True)["out"], "ragged")


@pytest.mark.parametrize("splits", [0, 4, 12])
def test_two_captured_steps_and_an_eager_one(splits):
    """Two graphs of a step, each with its state and workspace, replayed at the same time on two streams, do what eager
    calls do."""
    B, hq, hkv, d, page, nb, T = 3, 8, 2, 64, 16, 20, 8
    inv = (10000.0 ** (-torch.arange(0, d, 2, device=DEV) / d)).float()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    runs = []
    for seed in (1, 2, 3):
        s = _state(B, hq, hkv, d, page, nb, 60, T, torch.ones((hkv, d), device=DEV))
        s["new"].fill_(2)
        _step(s, inv, 2, splits)  # warms up what a capture may not do
        sl8.paged_read_int4(*s["pool"], s["table"], s["seq"], out_dtype=BF16)
        torch.cuda.synchronize()
        s["seq"].zero_(), s["table"].fill_(-1), s["count"].fill_(60)
        s["free"].copy_(torch.arange(60)), s["pool"][0].fill_(0x88), s["pool"][2].fill_(0x88), s["pool"][1].zero_(), s["pool"][3].zero_()
        ws = torch.empty(max(16, sl8.int4_decode_workspace_bytes(B, 2, hq, hkv, nb, page, d, splits)), dtype=torch.uint8, device=DEV)
        dense = [torch.zeros((B, hkv, nb * page, d), dtype=BF16, device=DEV) for _ in range(2)]

        def step(s=s, ws=ws, dense=dense):
            res = _step(s, inv, 2, splits, workspace=ws)
            sl8.paged_read_int4(*s["pool"], s["table"], s["seq"], k_mean=s["mean"], k_out=dense[0], v_out=dense[1])
            return res[2] + tuple(dense) + s["pool"]
        g, res = torch.cuda.CUDAGraph(), None
        if seed < 3:
            with torch.cuda.graph(g):
                res = step()
        runs.append([s, g, res, step])
    for n in range(40):
        x = torch.randn(runs[0][0]["qkv"].shape, generator=torch.Generator(device=DEV).manual_seed(n), device=DEV)
        for run in runs:
            run[0]["qkv"].copy_(x)
        for st in (side, other):
            st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            runs[0][1].replay()
        with torch.cuda.stream(other):
            runs[1][1].replay()
        want = runs[2][3]()
        for st in (side, other):
            torch.cuda.current_stream().wait_stream(st)
        for run in runs[:2]:
            for a, b in zip(run[2], want):
                assert torch.equal(a, b), n
    assert runs[0][0]["seq"].tolist() == [80] * 3


def test_side_stream_and_refusals():
    rng = np.random.default_rng(2)
    pool, _ = _filled(rng, 6, 2, 16, 64)
    table, lens = i32([[0, 1, 2], [3, 4, 5]]), i32([40, 20])
    q = torch.randn((2, 4, 64), device=DEV).half()
    want = sl8.attn_int4_paged_decode(q, *pool, table, lens, num_splits=12), *sl8.paged_read_int4(*pool, table, lens)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = sl8.attn_int4_paged_decode(q, *pool, table, lens, num_splits=12), *sl8.paged_read_int4(*pool, table, lens)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # out, lse and workspace of the caller's
    out, lse = torch.empty((2, 4, 64), device=DEV), torch.empty((2, 4), device=DEV)
    a, b = sl8.attn_int4_paged_decode(q, *pool, table, lens, return_lse=True, out=out, lse=lse,
                                      workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert a is out and b is lse
    decode = lambda *x, **kw: sl8.attn_int4_paged_decode(*x, **kw)  # noqa: E731
    bad = [(ValueError, lambda: decode(q.transpose(0, 1), *pool, table, lens)), (ValueError, lambda: decode(q[:1], *pool, table, lens)),
           (TypeError, lambda: decode(q, *pool, table.long(), lens)), (ValueError, lambda: decode(q, *pool, table, lens[:1])),
           (ValueError, lambda: decode(q, *pool, table.t().contiguous().t(), lens)), (TypeError, lambda: decode(q.double(), *pool, table, lens)),
           (ValueError, lambda: decode(q, *pool, table, lens, tree_mask=i32([1]))), (ValueError, lambda: decode(q, *pool, table, lens, out=out[:1])),
           (ValueError, lambda: decode(q, *pool, table, lens, return_lse=True, lse=lse[:1])), (ValueError, lambda: decode(q[0], *pool, table, lens)),
           (TypeError, lambda: decode(q, pool[0].view(torch.int8), *pool[1:], table, lens)),
           (TypeError, lambda: decode(q, pool[0], pool[1].half(), *pool[2:], table, lens)),
           (ValueError, lambda: decode(q, pool[0], pool[1][:5], *pool[2:], table, lens)),
           (ValueError, lambda: decode(q, *pool[:2], pool[2][:5], pool[3], table, lens)),
           (sl8.SL8Error, lambda: decode(q, *pool, table, lens, num_splits=12, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))),
           (ValueError, lambda: decode(q.cpu(), *pool, table, lens))]
    k = torch.randn((4, 2, 64), device=DEV).half()
    slots = i32([0, 1, 2, 3])
    append = sl8.rope_append_int4
    bad += [(ValueError, lambda: append(None, k[..., ::2], k[..., ::2], None, None, slots, *pool)),
            (TypeError, lambda: append(None, k, k.float(), None, None, slots, *pool)),
            (ValueError, lambda: append(None, k, k, slots, None, slots, *pool)), (ValueError, lambda: append(None, k, k, None, None, slots[:3], *pool)),
            (ValueError, lambda: append(None, k, k, None, None, slots, *pool, k_mean=torch.zeros(64, device=DEV))),
            (TypeError, lambda: append(None, k, k, None, None, slots, *pool, k_mean=torch.zeros((2, 64), device=DEV).half()))]
    read = sl8.paged_read_int4
    bad += [(ValueError, lambda: read(*pool, table, lens[:1])), (ValueError, lambda: read(*pool, table, lens, cu_seqlens=i32([0, 40, 60]))),
            (ValueError, lambda: read(*pool, table, lens, cu_seqlens=i32([0, 40]), total_tokens=60)),
            (TypeError, lambda: read(*pool, table, lens, out_dtype=torch.float64)),
            (ValueError, lambda: read(*pool, table, lens, max_seqlen=40, k_out=torch.empty((2, 2, 39, 64), device=DEV))),
            (TypeError, lambda: read(*pool, table, lens, max_seqlen=8, k_out=torch.empty((2, 2, 8, 64), device=DEV), out_dtype=BF16)),
            (ValueError, lambda: read(*pool, table, lens, k_mean=torch.zeros((1, 64), device=DEV)))]
    for i, (error, call) in enumerate(bad):
        try:
            call()
        except error:
            continue
        pytest.fail(f"call {i} was not refused with {error}")


def test_a_sequence_of_almost_2_31_tokens():
    """Positions, steps and block numbers near their limits: one token outweighs all others by 2^80 (they come to 2^-49 of it),
    and the output is its value row, wherever it lies."""
    d, page = 32, 1 << 20
    nb = (1 << 31) // page - 1
    pool = sl8.int4_pages(2, 1, page, d, DEV)  # page 0: keys and values of 0
    row = page - 1
    pool[0][1, 0, row], pool[1][1, 0, row] = 0xff, 1.0  # codes 7
    c = torch.arange(16, dtype=torch.uint8) * 17
    pool[2][1, 0, row], pool[3][1, 0, row] = c.to(DEV), 0.5
    want = Q.values(c.numpy()[None], np.array([[0.5]]))[0]
    q = torch.ones((1, 2, d), device=DEV)
    q *= 80 * np.log(2) * np.sqrt(d) / (7 * d)  # codes 127 of the scale's own: a logit of 80 log 2
    for block in (0, 1024, nb - 1):
        table = torch.zeros((1, nb), dtype=torch.int32, device=DEV)
        table[0, block] = 1
        for splits, odt in ((0, F32), (1 << 20, F16)):
            out, lse = sl8.attn_int4_paged_decode(q, *pool, table, i32([nb * page]), num_splits=splits, out_dtype=odt, return_lse=True)
            # the weight's roundings (2^-23, or 2^-11 + 2^-17), those of the merges and the output's
            tol = np.abs(want) * (2.0 ** -18 if odt == F32 else 2.0 ** -11 + 2.0 ** -16 + 2.0 ** -11)
            assert np.all(np.abs(np64(out[0]) - want) <= tol), (block, splits)
            assert np.all(np.abs(np64(lse[0]) - 80 * np.log(2)) <= 80 * 2.0 ** -20)
        # cut before that token, all logits are 0: the mean of values of 0; each lane's sum of ones is whole, and a few dozen merges
        # of 4 x 2,432 parts at most round by 2^-24 each
        if block == nb - 1:
            out, lse = sl8.attn_int4_paged_decode(q, *pool, table, i32([nb * page - 1]), return_lse=True)
            assert not out.any() and np.all(np.abs(np64(lse) - np.log(nb * page - 1)) <= 2.0 ** -10)


def test_nothing_to_do():
    """No sequences, no tokens, no room: nothing is written and nothing refused."""
    pool = sl8.int4_pages(2, 2, 16, 64, DEV)
    before = [x.clone() for x in pool]
    k = torch.zeros((0, 2, 64), device=DEV)
    assert sl8.rope_append_int4(k, k, k, i32([]), torch.ones(32, device=DEV), i32([]), *pool).shape == (0, 2, 64)
    out = sl8.attn_int4_paged_decode(torch.zeros((0, 4, 64), device=DEV), *pool, i32(np.zeros((0, 3))), i32([]))
    assert out.shape == (0, 4, 64)
    k, v = sl8.paged_read_int4(*pool, i32(np.zeros((0, 3))), i32([]))
    assert k.shape == v.shape == (0, 2, 48, 64)
    k, v = sl8.paged_read_int4(*pool, i32([[0, 1]]), i32([0]), max_seqlen=0)
    assert k.shape == (1, 2, 0, 64)
    k, v = sl8.paged_read_int4(*pool, i32([[0, 1]]), i32([0]), cu_seqlens=i32([0, 0]), total_tokens=0)
    assert k.shape == (0, 2, 64)
    assert all(torch.equal(a, b) for a, b in zip(pool, before))


# ------------------------------------------------------------------ groups and rows that are not numbers, scales far apart

def test_groups_of_nan_alone_are_zeros():
    """A group whose 32 values are all NaN has the codes 0 and the scale +0, bit for bit, where pairs turn (halves or adjacent)
    and where they do not; what its row's other groups hold comes out of a 16-bit attention, alone or with most of the weight."""
    T, hkv, d = 9, 2, 64
    for dtype in (F32, F16, BF16):
        for adjacent, rot in ((False, 0), (True, 32), (False, 32)):
            x = torch.randn((T, hkv, d), device=DEV).to(dtype)
            x[2, 0, :32], x[5, 1], x[7, :, 32:] = float("nan"), float("nan"), float("nan")
            pool = _pool(1, hkv, 16, d)
            pos, inv = (torch.arange(T, dtype=torch.int32, device=DEV), torch.rand(rot // 2, device=DEV)) if rot else (None, None)
            sl8.rope_append_int4(None, x, x, pos, inv, i32(np.arange(T)), *pool, adjacent=adjacent)
            for i in (0, 2):
                bits = pool[i + 1][0].transpose(0, 1)[:T].view(torch.int16)  # [T, hkv, 2]
                nan = torch.isnan(x).unflatten(-1, (2, 32)).all(-1)
                assert bool((bits[nan] == 0).all()) and bool((bits[~nan] > 0).all()), (dtype, adjacent, rot, i)
                assert bool((pool[i][0].transpose(0, 1)[:T].unflatten(-1, (2, 16))[nan] == 0x88).all())
    for d, odt in ((64, F16), (128, BF16), (256, F16), (32, BF16)):
        d2 = max(d, 64)
        for L in (1, 40):
            k = torch.zeros((L, 1, d2), device=DEV)
            v = torch.randn((L, 1, d2), device=DEV)
            k[L // 2], v[L // 2, :, 32:] = 30.0, float("nan")  # almost all of the weight
            v[L // 2, :, :32] = torch.linspace(-3.5, 3.5, 32, device=DEV)
            q = torch.ones((1, 1, 4, d2), device=DEV)
            pool = sl8.int4_pages(3, 1, 16, d2, DEV)
            sl8.rope_append_int4(None, k, v, None, None, i32(np.arange(L)), *pool)
            host = [x.float().cpu().numpy() if x.dtype == BF16 else x.cpu().numpy() for x in pool]
            for splits in (1, 3, 12):
                out, lse = sl8.attn_int4_paged_decode(q, *pool, i32([[0, 1, 2]]), i32([L]), num_splits=splits, out_dtype=odt, return_lse=True)
                _check_attention(out, lse, q, host, [[0, 1, 2]], [L], tag=(d2, L, splits))


@pytest.mark.parametrize("splits", [1, 3, 12])
@pytest.mark.parametrize("d,odt", [(64, F16), (64, BF16), (128, F16), (128, BF16), (256, BF16), (128, F32)])
def test_infinite_value_groups_leave_the_others_their_values(d, odt, splits):
    """An infinite V scale (codes 0, as the append stores it), a NaN one, and scales of -0 and below, in rows of ordinary, most and
    hardly any weight: the group's own channels are NaN where the scale is, all others and the lse the definition's."""
    rng = np.random.default_rng(d + splits)
    hkv, G, page, L = 1, 3, 16, 300
    q = torch.from_numpy(np.abs(rng.standard_normal((1, 1, G, d)).astype(np.float32)) + 0.5).to(DEV)
    for value in (float("inf"), float("nan"), -0.0, -0.5):
        for row, key in ((0, None), (19, None), (L - 1, None), (131, 0xff), (44, 0x11)):
            for n in (L, row + 1) if row == 0 else (L,):
                pool, (kc, ks, vc, vs) = _filled(rng, 20, hkv, page, d, 0.5)
                at = row // page, 0, row % page
                if key is not None:  # codes 7 or -7 against positive queries
                    kc[at], ks[at] = key, 2.0
                if not np.isfinite(value):
                    vc[at][16:32] = 0x88
                vs[at][1] = value
                for i, x in enumerate((kc, ks, vc, vs)):
                    pool[i].copy_(torch.from_numpy(x))
                out, lse = sl8.attn_int4_paged_decode(q, *pool, i32(np.arange(20)[None]), i32([n]), num_splits=splits, out_dtype=odt,
                                                      return_lse=True)
                if not np.isfinite(value):
                    assert torch.isnan(out[..., 32:64]).all(), (value, row)
                    vs[at][1] = 0
                    want = Q.attention(f32(q), kc, ks, vc, vs, [np.arange(20)], [n])[0]
                    out[..., 32:64] = torch.from_numpy(want[..., 32:64]).to(out)
                _check_attention(out, lse, q, (kc, ks, vc, np.abs(vs)) if value != -0.5 else (kc, ks, vc, vs), [np.arange(20)], [n],
                                 tag=(value, row, n))


@pytest.mark.parametrize("splits", [1, 3, 12])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_probabilities_do_not_depend_on_value_scales(d, splits):
    """The sum of the probabilities, and with it out and lse, whatever the V scales: rows of zero or the least scale beside one
    of a large one, equal logits or far apart, in one warp, in several and in several parts; scales of both ends of the stated range."""
    rng = np.random.default_rng(d)
    hkv, G, page, L = 1, 4, 16, 300
    tables = [np.arange(20)]
    q = torch.ones((1, 1, G, d), device=DEV)
    unit = 7 * np.sqrt(d)  # the logit of a row of codes 7 and the scale 1
    for most, least, row, x in ((60, None, 150, 0.0), (60, None, 299, 0.0), (60, None, 1, 0.0), (47, None, 131, 0.0), (112, -94, 40, 0.0),
                                (112, -94, 200, -50.0), (112, -94, 3, -20.0), (100, None, 257, -50.0), (0, 112, 64, 17.0), (112, 0, 5, 17.0),
                                (-94, None, 290, 3.0), (20, -20, 33, 30.0), (124, -94, 77, 30.0), (124, -94, 77, 0.0), (-94, 124, 291, 9.0)):
        pool, (kc, ks, vc, vs) = _filled(rng, 20, hkv, page, d)
        kc[:], ks[:] = 0x88, 1.0
        vs[:] = 0.0 if least is None else 2.0 ** least
        at = row // page, 0, row % page
        kc[at] = 0xff if x >= 0 else 0x11
        ks[at] = Q.to_bf16(np.float32(abs(x) * np.log(2) / unit))
        vs[at] = 2.0 ** most
        for i, a in enumerate((kc, ks, vc, vs)):
            pool[i].copy_(torch.from_numpy(a))
        for odt in (BF16, F32) if 124 not in (most, least) else (BF16,):  # fp32 outputs take up to 2^117 over the length
            out, lse = sl8.attn_int4_paged_decode(q, *pool, i32(tables), i32([L]), num_splits=splits, out_dtype=odt, return_lse=True)
            _check_attention(out, lse, q, (kc, ks, vc, vs), tables, [L], tag=(most, least, row, x, odt))


@pytest.mark.parametrize("splits", [1, 8, 40])
def test_many_small_probabilities_beside_a_large_scale(splits):
    """20,000 tokens of 2^-17 of the largest probability each come to 15 % of the sum, beside a row of the scale 2^110."""
    d, page, L = 64, 16, 20001
    nb = -(-L // page)
    tables = [np.arange(nb)]
    kc, ks = np.full((nb, 1, page, d // 2), 0x88, np.uint8), np.ones((nb, 1, page, d // 32), np.float32)
    vc, vs = np.full((nb, 1, page, d // 2), 0x9d, np.uint8), np.ones((nb, 1, page, d // 32), np.float32)
    at = 700, 0, 3
    kc[at], ks[at], vs[at] = 0xff, Q.to_bf16(np.float32(17 * np.log(2) / (7 * np.sqrt(d)))), 2.0 ** 110
    pool = sl8.int4_pages(nb, 1, page, d, DEV)
    for i, x in enumerate((kc, ks, vc, vs)):
        pool[i].copy_(torch.from_numpy(x))
    q = torch.ones((1, 1, 2, d), device=DEV)
    out, lse = sl8.attn_int4_paged_decode(q, *pool, i32(tables), i32([L]), num_splits=splits, out_dtype=BF16, return_lse=True)
    _check_attention(out, lse, q, (kc, ks, vc, vs), tables, [L])


@pytest.mark.parametrize("d,T,G", [(32, 1, 3), (64, 1, 16), (128, 2, 4), (128, 1, 24), (256, 1, 8)])
def test_the_lse_has_the_same_bits_for_any_values(d, T, G):
    rng = np.random.default_rng(d + G)
    lens = [700, 33, 1, 260]
    pool, host = _filled(rng, 80, 1, 16, d)
    tables = _tables(rng, lens, 44, 16, 80)
    q = torch.from_numpy(rng.standard_normal((4, T, G, d)).astype(np.float32) * 3).to(DEV)
    for splits in (0, 1, 4, 12):
        call = lambda odt: sl8.attn_int4_paged_decode(q, *pool, i32(tables), i32(lens), num_splits=splits, out_dtype=odt, return_lse=True)  # noqa: E731
        for odt in (F16, BF16):
            pool[3].copy_(torch.from_numpy(host[3]))
            _, want = call(odt)
            for make in (lambda s: s * 0, lambda s: 10.0 ** rng.uniform(-28, 33, s.shape), lambda s: np.where(rng.random(s.shape) < 0.1, np.inf, s)):
                pool[3].copy_(torch.from_numpy(make(host[3]).astype(np.float32)))
                assert torch.equal(call(odt)[1], want), (splits, odt)


@pytest.mark.parametrize("d,splits", [(32, 1), (64, 3), (128, 12), (256, 1)])
def test_large_queries_meet_small_keys(d, splits):
    """Queries just below 2^106 and key scales that make ordinary logits of them."""
    rng = np.random.default_rng(d)
    pool, (kc, ks, vc, vs) = _filled(rng, 10, 1, 16, d)
    ks = ks * np.float32(2.0 ** -104)
    pool[1].copy_(torch.from_numpy(ks))
    x = rng.standard_normal((1, 1, 5, d)).clip(-4, 4).astype(np.float32) * np.float32(2.0 ** 103)
    x[0, 0, 0, 0] = 2.0 ** 106 * (1 - 2.0 ** -24)
    q = torch.from_numpy(x).to(DEV)
    for odt in (F32, F16):
        out, lse = sl8.attn_int4_paged_decode(q, *pool, i32(np.arange(10)[None]), i32([150]), num_splits=splits, out_dtype=odt, return_lse=True)
        _check_attention(out, lse, q, (kc, ks, vc, vs), [np.arange(10)], [150], tag=odt)
