"""Serving from the paged int8 cache on the GPU, against the CPU definitions: the page plan,
the rotary append, page bounds, page selection and sparse decode, alone and as one step.

Tolerances.  Page plans, bounds, scores and selections are fixed bit for bit.  Rotations:
the angle is good to 2^-23 turns (7.5e-7 rad) or better, sincospif to 2 ulp, and each output takes
three fp32 roundings, so a rotated value is within 2e-6 of its pair's length, then half a
step of its type.  Codes: half a scale plus that.  Attention: each probability is rounded
to fp16 (2^-11 of itself, or 2^-25 of the range of P' = p s_v 2^-E at the bottom of fp16,
at most 2^-24 max|v| a token), then the output's type.
"""
import numpy as np
import pytest
import torch

import w8a8_int8_flashattention_gb300 as sl8
from oracle import serving as S

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda"
NP = {torch.float16: np.float16, torch.float32: np.float32}


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


# ------------------------------------------------------------------ page plan

def _plan_case(rng, B, nb, page, releases, spare):
    ctx = rng.integers(0, nb * page + 1, B)
    ctx[rng.random(B) < 0.2] = 0
    held = -(-ctx // page)
    total = int(held.sum()) + spare
    perm = rng.permutation(total)
    table, at = np.full((B, nb), -1), 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = np.full(total + 1, -1)
    free[:spare] = perm[at:]
    return ctx, table, free, spare, (rng.integers(0, 2, B) if releases else None)


def _check_plan(got, want, table, free, tag):
    for name in ("seqlens", "granted", "cu_new", "slot_map", "token_pos"):
        np.testing.assert_array_equal(got[name].cpu().numpy(), want[name], err_msg=f"{tag} {name}")
    assert got["free_count"].item() == want["free_count"], tag
    np.testing.assert_array_equal(table.cpu().numpy(), want["block_table"], err_msg=tag)
    np.testing.assert_array_equal(free.cpu().numpy(), want["free_pages"], err_msg=tag)


@pytest.mark.parametrize("B,nb,page,max_new,max_tokens,releases", [
    (1, 4, 16, 1, 1, False), (3, 3, 1, 2, 5, True), (8, 7, 16, 40, 300, True), (33, 5, 3, 9, 200, True),
    (256, 40, 16, 700, 60000, True), (1025, 4, 8, 20, 9000, True), (2500, 3, 16, 30, 50000, False)])
def test_paged_assign(B, nb, page, max_new, max_tokens, releases):
    rng = np.random.default_rng(B * 7 + page)
    for spare in (0, B // 2, 4 * B):
        ctx, table, free, count, release = _plan_case(rng, B, nb, page, releases, spare)
        new = rng.integers(0, max_new + 1, B)
        want = S.paged_assign(ctx, new, release, table, free, count, page, max_tokens)
        tab, fr = i32(table), i32(free)
        got = sl8.paged_assign(i32(ctx), i32(new), tab, fr, i32([count]), page, max_tokens,
                               release=None if release is None else i32(release))
        _check_plan(got, want, tab, fr, f"spare {spare}")


def test_paged_assign_in_place_and_steps():
    """Lengths and the count kept in place over many steps, slots released and refilled."""
    rng = np.random.default_rng(11)
    B, nb, page, T = 1300, 6, 4, 3000
    seqlens, table, count = np.zeros(B, np.int64), np.full((B, nb), -1), 900
    free = rng.permutation(900)
    d = dict(seq=i32(seqlens), table=i32(table), free=i32(free), count=i32([count]))
    out = None
    for step in range(8):
        new, release = rng.integers(0, 5, B), (rng.random(B) < 0.1).astype(np.int64)
        want = S.paged_assign(seqlens, new, release, table, free, count, page, T)
        if out is None:
            out = sl8.paged_assign(d["seq"], i32(new), d["table"].clone(), d["free"].clone(), d["count"], page, T,
                                   release=i32(release))
            out.update(seqlens=d["seq"], free_count=d["count"])
        out["granted"].copy_(i32(new))  # new lengths in, granted tokens out
        got = sl8.paged_assign(d["seq"], out["granted"], d["table"], d["free"], d["count"], page, T, release=i32(release),
                               out=out)
        _check_plan(got, want, d["table"], d["free"], f"step {step}")
        seqlens, table, free, count = want["seqlens"], want["block_table"], want["free_pages"], want["free_count"]


def test_paged_assign_captured_with_many_tokens():
    """The plan and the kernel that maps the tokens, captured and replayed on new lengths."""
    rng = np.random.default_rng(5)
    B, nb, page, T = 40, 100, 16, 20000
    ctx, table, free, count, _ = _plan_case(rng, B, nb, page, False, 1500)
    d = dict(ctx=i32(ctx), new=i32(np.zeros(B)), table=i32(table), free=i32(free), count=i32([count]))
    call = lambda out: sl8.paged_assign(d["ctx"], d["new"], d["table"], d["free"], d["count"], page, T, out=out)  # noqa: E731
    out = call(None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    for _ in range(3):
        new = rng.integers(0, 900, B)
        d["new"].copy_(i32(new))
        d["table"].copy_(i32(table))
        g.replay()
        _check_plan(out, S.paged_assign(ctx, new, None, table, free, count, page, T), d["table"], d["free"], "replay")


def test_paged_assign_no_requests_and_bad_lengths():
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    out = sl8.paged_assign(z, z, z.view(0, 4), i32([1, 2]), i32([2]), 16, 3)
    assert out["slot_map"].tolist() == [-1] * 3 and out["token_pos"].tolist() == [0] * 3
    assert out["cu_new"].tolist() == [0] and out["free_count"].item() == 2
    # a negative length, a context above the table and a count above the list: recorded,
    # refused, and nothing else is touched
    table = i32([[3, -1], [4, 5], [6, -1]])
    free = i32([7, 8, -1])
    out = sl8.paged_assign(i32([4, 99, 2]), i32([-1, 1, 3]), table, free, i32([2]), 4, 8)
    assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
    assert out["granted"].tolist() == [0, 0, 3] and out["seqlens"].tolist() == [4, 8, 5]
    assert out["cu_new"].tolist() == [0, 0, 0, 3] and out["slot_map"].tolist() == [26, 27, 32] + [-1] * 5
    assert table.tolist() == [[3, -1], [4, 5], [6, 8]] and out["free_count"].item() == 1
    out = sl8.paged_assign(i32([0]), i32([1]), i32([[-1]]), free, i32([9]), 4, 1)
    assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
    # a released slot whose pages would pass the list's end
    out = sl8.paged_assign(i32([8]), i32([0]), i32([[1, 2]]), i32([0]), i32([0]), 4, 1, release=i32([1]))
    assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
    assert out["free_count"].item() == 1 and out["seqlens"].tolist() == [0]


def test_paged_assign_released_slots_with_bad_lengths():
    """An ended request whose length is out of range: its pages are not released and no new
    one starts in its slot; the other slots go on."""
    table, free = i32([[0, 1], [2, 3], [4, -1]]), i32([5, 6, -1, -1, -1])
    out = sl8.paged_assign(i32([-3, 9, 4]), i32([2, 2, 2]), table, free, i32([2]), 4, 8, release=i32([1, 1, 1]))
    assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
    assert out["granted"].tolist() == [0, 0, 2] and out["seqlens"].tolist() == [0, 0, 2]
    assert out["cu_new"].tolist() == [0, 0, 0, 2] and out["slot_map"].tolist() == [16, 17] + [-1] * 6
    assert table.tolist() == [[0, 1], [2, 3], [4, -1]] and out["free_count"].item() == 2 and free[:2].tolist() == [5, 6]
    # a bad count of new tokens leaves the release as it is
    out = sl8.paged_assign(i32([5]), i32([-1]), i32([[7, 8]]), free, i32([2]), 4, 8, release=i32([1]))
    assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
    assert out["free_count"].item() == 4 and free[:4].tolist() == [5, 6, 7, 8] and out["seqlens"].tolist() == [0]


# ------------------------------------------------------------------ rotary append

def _rotation_tol(x, rot, adjacent):
    """2e-6 of each rotated channel's pair length; 0 for the others."""
    t = np.zeros_like(x)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if adjacent else (slice(0, rot // 2), slice(rot // 2, rot))
    t[..., a] = t[..., b] = 2e-6 * np.hypot(x[..., a], x[..., b])
    return t


@pytest.mark.parametrize("d,rot,axes,adjacent,hq,hkv,dtype,T,page", [
    (128, 128, 1, False, 32, 8, torch.bfloat16, 1, 16), (128, 96, 3, False, 5, 1, torch.float16, 37, 16),
    (64, 64, 1, True, 7, 3, torch.bfloat16, 130, 7), (32, 8, 2, False, 3, 3, torch.float32, 65, 32),
    (256, 256, 4, True, 2, 2, torch.float32, 9, 16), (256, 64, 1, False, 16, 8, torch.float16, 700, 64),
    (32, 32, 1, True, 1, 1, torch.float16, 3000, 1000), (64, 0, 0, False, 2, 2, torch.bfloat16, 20, 16),
    (128, 128, 1, False, 0, 2, torch.bfloat16, 20, 16)])
def test_rope_append(d, rot, axes, adjacent, hq, hkv, dtype, T, page):
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
    pages = torch.full((2, num_pages, hkv, page, d), 77, dtype=torch.int8, device=DEV)
    scales = torch.full((2, num_pages, hkv, page), -7.0, dtype=torch.float32, device=DEV)
    out = sl8.rope_append(q, k, v, i32(pos if axes > 1 else pos[0]) if rot else None,
                          torch.from_numpy(inv).to(DEV) if rot else None, i32(slots), pages[0], scales[0], pages[1],
                          scales[1], pair_axis=axis if axes > 1 else None, adjacent=adjacent)
    host = qkv.double().numpy()
    eps = torch.finfo(dtype).eps / 2
    used = axis if axes > 1 else None
    if hq:
        x = host[:, :hq * d].reshape(T, hq, d)
        want = S.rope(x, pos, inv, used, adjacent)
        err = np.abs(np64(out) - want)
        # a value rounds from within the rotation's error; tiny fp16 results round to 2^-25
        assert np.all(err <= _rotation_tol(x, rot, adjacent) * (1 + eps) + eps * np.abs(want) + 2.0 ** -25)
    kx = host[:, hq * d:(hq + hkv) * d].reshape(T, hkv, d)
    want, tol = S.rope(kx, pos, inv, used, adjacent), _rotation_tol(kx, rot, adjacent)
    vc, vs = S._quant(host[:, (hq + hkv) * d:(hq + 2 * hkv) * d].reshape(T, hkv, d).astype(np.float32))
    gk, gs = pages.cpu().numpy(), scales.cpu().numpy()
    touched = np.zeros((num_pages, page), bool)
    for t in range(T):
        if slots[t] < 0:
            continue
        at = slots[t] // page, slice(None), slots[t] % page
        touched[at[0], at[2]] = True
        np.testing.assert_array_equal(gk[1][at], vc[t])
        np.testing.assert_array_equal(gs[1][at], vs[t])
        amax = np.abs(want[t]).max(-1)
        assert np.all(np.abs(gs[0][at] * 127.0 - amax) <= tol[t].max(-1) + 2.0 ** -23 * amax)
        near = gk[0][at].astype(np.float64) * gs[0][at][:, None].astype(np.float64)
        step = gs[0][at][:, None].astype(np.float64)
        assert np.all(np.abs(near - want[t]) <= step * (0.5 + 127 * 2.0 ** -23) + tol[t])
    # rows without a slot stay as they were
    assert np.all(gk.transpose(0, 1, 3, 2, 4)[:, ~touched] == 77) and np.all(gs.transpose(0, 1, 3, 2)[:, ~touched] == -7.0)


def test_rope_append_in_place_and_bad_slot():
    T, hq, hkv, d = 6, 4, 2, 64
    qkv = torch.randn((T, (hq + 2 * hkv) * d), device=DEV).half()
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    pos, inv = torch.arange(T, dtype=torch.int32, device=DEV), torch.rand(d // 2, device=DEV)
    pages, scales = torch.zeros((2, 2, hkv, 4, d), dtype=torch.int8, device=DEV), torch.zeros((2, 2, hkv, 4), device=DEV)
    slots = i32([0, 1, 2, 8, -3, 5])  # slot 8 lies past the two pages
    want = sl8.rope_append(q, k, v, pos, inv, slots, pages[0], scales[0], pages[1], scales[1])
    assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
    kept = k.clone()
    got = sl8.rope_append(q, k, v, pos, inv, i32([0, 1, 2, -1, -3, 5]), pages[0], scales[0], pages[1], scales[1], q_out=q)
    assert got.data_ptr() == qkv.data_ptr() and torch.equal(got, want) and torch.equal(k, kept)
    assert int((scales[0] != 0).sum()) == 4 * hkv


def test_stored_rows_are_the_quantisers():
    """Codes without a division per value: the bits of the quantiser's definition, on values that
    sit on rounding borders and on tiny and huge rows; a row with an infinity gets the scale
    inf and codes 0, a NaN the code 0."""
    g = torch.Generator().manual_seed(9)
    T, hkv, d = 512, 4, 64
    v = torch.randn((T, hkv, d), generator=g)
    v[0:64] = torch.randint(-254, 255, (64, hkv, d), generator=g).float() / 2  # halves of a step of 1
    v[0:64, :, 0] = 127.0
    v[64:128] *= torch.logspace(-44, 37, 64)[:, None, None]
    v[128:192] = torch.randint(-254, 255, (64, hkv, d), generator=g).float() / 2 * (1 + 2.0 ** -23)
    v[128:192, :, 1] = -127.0
    v[192, :, 3], v[193, :, 3], v[194, :, 3] = float("inf"), float("-inf"), float("nan")
    v[195, :, 3], v[195, :, 9] = float("nan"), float("inf")
    v[196] = float("nan")
    v[197] = 0
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        x = v.to(dtype).to(DEV)
        pages, scales = torch.zeros((2, 1, hkv, T, d), dtype=torch.int8, device=DEV), torch.zeros((2, 1, hkv, T), device=DEV)
        sl8.rope_append(None, x, x, None, None, i32(np.arange(T)), pages[0], scales[0], pages[1], scales[1])
        h = x.float().cpu().numpy()
        want, s = S._quant(np.where(np.isnan(h), 0, h))
        want[np.isinf(h).any(-1)] = 0
        for i in range(2):
            np.testing.assert_array_equal(pages[i, 0].transpose(0, 1).cpu().numpy(), want)
            np.testing.assert_array_equal(scales[i, 0].T.cpu().numpy(), s)


def test_rope_append_to_a_contiguous_cache():
    """page_size = Lmax: the contiguous cache of attn_int8_decode."""
    B, hq, hkv, d, L = 3, 8, 2, 128, 50
    lens = [50, 1, 33]
    g = torch.Generator(device=DEV).manual_seed(5)
    kc, vc = (torch.zeros((B, hkv, 64, d), dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((B, hkv, 64), device=DEV) for _ in range(2))
    k, v = (torch.randn((B * L, hkv, d), generator=g, device=DEV).bfloat16() for _ in range(2))
    slots = torch.cat([torch.where(torch.arange(L) < n, torch.arange(L) + 64 * b, -1) for b, n in enumerate(lens)])
    sl8.rope_append(None, k, v, None, None, i32(slots), kc, ks, vc, vs)
    want, wants = sl8.quant_rowwise(k.view(B, L, hkv, d).transpose(1, 2).contiguous())
    for b, n in enumerate(lens):
        assert torch.equal(kc[b, :, :n], want[b, :, :n]) and torch.equal(ks[b, :, :n], wants[b, :, :n])
    q = torch.randn((B, hq, d), generator=g, device=DEV).bfloat16()
    out = sl8.attn_int8_decode(q, kc, ks, vc, vs, i32(lens))
    assert torch.isfinite(out).all()


# ------------------------------------------------------------------ page bounds

def _pool(rng, num_pages, hkv, page, d):
    """A page pool with rows of very different scales (some zero) and its tensors."""
    codes = [rng.integers(-127, 128, (num_pages, hkv, page, d)).astype(np.int8) for _ in range(2)]
    scales = [(rng.random((num_pages, hkv, page)) * 10.0 ** rng.integers(-3, 1, (num_pages, hkv, page)) * 0.03).astype(np.float32)
              for _ in range(2)]
    scales[0][rng.random(scales[0].shape) < 0.05] = 0
    return codes, scales, [torch.from_numpy(x).to(DEV) for x in codes], [torch.from_numpy(x).to(DEV) for x in scales]


def _tables(rng, lens, nb, page, spare=2):
    need = -(-np.asarray(lens) // page)
    perm = rng.permutation(int(need.sum()) + spare)
    table, at = np.full((len(lens), nb), -1), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, int(need.sum()) + spare


@pytest.mark.parametrize("d,hkv,page", [(32, 1, 16), (64, 3, 7), (128, 2, 64), (256, 8, 16), (128, 1, 300)])
def test_page_bounds(d, hkv, page):
    rng = np.random.default_rng(d + page)
    lens = [1, page, page + 1, 3 * page - 1, 4 * page, 0]
    new = [1, 1, 2, 2 * page, 0, 0]
    table, num_pages = _tables(rng, lens, 5, page)
    codes, scales, dk, ds = _pool(rng, num_pages, hkv, page, d)
    for some in (True, False):
        bounds = torch.full((num_pages, hkv, 2, d), 99, dtype=torch.int8, device=DEV)
        bs = torch.full((num_pages, hkv), -3.0, device=DEV)
        sl8.page_bounds(dk[0], ds[0], i32(table), i32(lens), bounds, bs, new_lens=i32(new) if some else None,
                        max_new=2 * page if some else None)
        gb, gs = bounds.cpu().numpy(), bs.cpu().numpy()
        seen = set()
        for b, L in enumerate(lens):
            n = new[b] if some else L
            for j in range((L - n) // page, -(-L // page)) if n else []:
                p, rows = table[b, j], min(page, L - j * page)
                seen.add(p)
                for h in range(hkv):
                    lo, hi, s = S.page_bounds(codes[0][p, h, :rows], scales[0][p, h, :rows])
                    np.testing.assert_array_equal(gb[p, h, 0], lo)
                    np.testing.assert_array_equal(gb[p, h, 1], hi)
                    assert gs[p, h] == s
        rest = [p for p in range(num_pages) if p not in seen]
        assert np.all(gb[rest] == 99) and np.all(gs[rest] == -3.0)


def test_page_bounds_reports_bad_lengths_and_pages():
    k, ks = torch.ones((2, 1, 16, 64), dtype=torch.int8, device=DEV), torch.ones((2, 1, 16), device=DEV)
    b, bs = torch.zeros((2, 1, 2, 64), dtype=torch.int8, device=DEV), torch.zeros((2, 1), device=DEV)
    for table, lens, new in (([[0], [5]], [16, 16], [1, 1]), ([[0], [1]], [16, 17], [1, 1]), ([[0], [1]], [16, 16], [1, 3])):
        sl8.page_bounds(k, ks, i32(table), i32(lens), b, bs, new_lens=i32(new), max_new=2)
        assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
        assert bs[0, 0] == 1.0


def test_rows_with_infinities_stay_out_of_a_selection():
    """A key row with an infinity: its page's bounds are zero, its score -inf, and only a
    forced page is listed in spite of it; the same for a query row."""
    num_pages, page, hkv, d = 40, 16, 2, 64
    rng = np.random.default_rng(3)
    k = torch.randn((num_pages * page, hkv, d), generator=torch.Generator().manual_seed(2))
    k[5 * page + 3, 0, 7] = float("inf")    # one row of a page
    k[9 * page, 1, 0] = -float("inf")       # the only row of a page (the last: page 39 of the table)
    codes, scales = (torch.zeros(s, dtype=t, device=DEV) for s, t in (((num_pages, hkv, page, d), torch.int8),
                                                                      ((num_pages, hkv, page), torch.float32)))
    vc, vs = codes.clone(), scales.clone()
    sl8.rope_append(None, k.to(DEV), k.to(DEV), None, None, torch.arange(num_pages * page, dtype=torch.int32, device=DEV),
                    codes, scales, vc, vs)
    table = [[i for i in range(num_pages) if i != 9] + [9]]
    L = (num_pages - 1) * page + 1
    bounds, bs = torch.full((num_pages, hkv, 2, d), 99, dtype=torch.int8, device=DEV), torch.zeros((num_pages, hkv), device=DEV)
    sl8.page_bounds(codes, scales, i32(table), i32([L]), bounds, bs)
    nc, ns, gb, gs = (x.cpu().numpy() for x in (codes, scales, bounds, bs))
    for j, pg in enumerate(table[0]):
        for h in range(hkv):
            lo, hi, s = S.page_bounds(nc[pg, h, :min(page, L - j * page)], ns[pg, h, :min(page, L - j * page)])
            np.testing.assert_array_equal(gb[pg, h], np.stack([lo, hi]))
            assert gs[pg, h] == s
    assert np.isinf(gs[5, 0]) and np.isinf(gs[9, 1]) and not gb[5, 0].any() and not gb[9, 1].any()
    q = torch.randn((1, 2 * hkv, d), generator=torch.Generator().manual_seed(4))
    q[0, 1, 3] = float("inf")               # one of the first kv head's two query heads
    for last in (0, 1):
        out = sl8.page_select(q.to(DEV), bounds, bs, i32(table), i32([L]), page, 38, 0, last)
        for h in range(hkv):
            ids = np.array(table[0])
            want = S.page_scores(q[0, 2 * h:2 * h + 2].numpy(), gb[ids, h, 0].astype(np.int64), gb[ids, h, 1].astype(np.int64),
                                 gs[ids, h])
            assert np.isneginf(want[5 if h == 0 else 39])
            kept = S.select(want, 38, 0, last)
            assert (5 not in kept) if h == 0 else ((39 in kept) == bool(last))
            np.testing.assert_array_equal(out["blocks"][0, 0, h].cpu().numpy(), kept)


# ------------------------------------------------------------------ page selection

def _bounds_pool(rng, num_pages, hkv, d, coarse=False):
    lo = rng.integers(-127, 100, (num_pages, hkv, d))
    hi = np.minimum(127, lo + rng.integers(0, 60, lo.shape))
    s = rng.random((num_pages, hkv)).astype(np.float32) * 0.02 + 0.01
    if coarse:  # many equal pages: the scores tie
        lo, hi, s = lo[rng.integers(0, 3, num_pages)], hi[rng.integers(0, 3, num_pages)], np.full_like(s, 0.5)
        hi = np.maximum(lo, hi)
    b = np.stack([lo, hi], 2).astype(np.int8)
    return b, s, torch.from_numpy(b).to(DEV), torch.from_numpy(s).to(DEV)


@pytest.mark.parametrize("B,T,hq,hkv,d,page,nb,max_sel,first,last,dtype,coarse", [
    (1, 1, 4, 1, 64, 16, 1, 1, 1, 0, torch.bfloat16, False), (3, 1, 32, 8, 128, 64, 40, 8, 1, 2, torch.bfloat16, False),
    (2, 3, 6, 2, 64, 16, 300, 33, 2, 1, torch.float16, True), (1, 1, 8, 8, 32, 16, 3000, 200, 0, 0, torch.float32, False),
    (1, 1, 16, 1, 256, 16, 2100, 100, 1, 1, torch.bfloat16, False), (2, 2, 40, 1, 128, 32, 600, 64, 4, 4, torch.float16, False),
    (1, 1, 2, 1, 64, 16, 9000, 8990, 1, 2, torch.bfloat16, True), (5, 4, 12, 4, 128, 16, 70, 16, 8, 8, torch.bfloat16, False),
    (2, 1, 64, 1, 32, 16, 520, 1, 0, 1, torch.bfloat16, True), (60, 1, 8, 4, 64, 16, 90, 20, 1, 2, torch.bfloat16, True)])
def test_page_select(B, T, hq, hkv, d, page, nb, max_sel, first, last, dtype, coarse):
    rng = np.random.default_rng(B * 1000 + nb)
    lens = rng.integers(1, nb * page + 1, B)
    lens[0] = nb * page
    if B > 1:
        lens[1] = min(2, nb * page)  # with drafts: fewer tokens than queries
    if B > 2:
        lens[2] = 0
    table, num_pages = _tables(rng, lens, nb, page)
    b, s, db, ds = _bounds_pool(rng, num_pages, hkv, d, coarse)
    q = torch.randn((B, T, hq, d), generator=torch.Generator().manual_seed(nb)).to(dtype)
    q[0, 0, 0] = 0  # a head without a direction scores every page 0
    scores = torch.full((B, T, hkv, nb), -9.0, device=DEV)
    out = sl8.page_select(q.to(DEV) if T > 1 else q[:, 0].to(DEV), db, ds, i32(table), i32(lens), page, max_sel, first, last,
                          scores=scores)
    plain = sl8.page_select(q.to(DEV), db, ds, i32(table), i32(lens), page, max_sel, first, last)
    for name in plain:
        assert torch.equal(out[name], plain[name])
    blocks, pages, got_lens, sc = (x.cpu().numpy() for x in (out["blocks"], out["pages"], out["lens"], scores))
    qf, G = q.float().numpy(), hq // hkv
    for i in range(B):
        for t in range(T):
            L = max(0, int(lens[i]) - T + 1 + t)
            n = -(-L // page)
            ids = table[i, :n]
            for h in range(hkv):
                want = S.page_scores(qf[i, t, h * G:(h + 1) * G], b[ids, h, 0].astype(np.int64), b[ids, h, 1].astype(np.int64),
                                     s[ids, h]) if n else np.zeros(0, np.float32)
                if n > max_sel:
                    np.testing.assert_array_equal(sc[i, t, h, :n], want)
                assert np.all(sc[i, t, h, n if n > max_sel else 0:] == -9.0)
                kept = S.select(want, max_sel, first, last)
                np.testing.assert_array_equal(blocks[i, t, h], kept + [-1] * (max_sel - len(kept)))
                np.testing.assert_array_equal(pages[i, t, h], [*ids[kept]] + [-1] * (max_sel - len(kept)))
                tokens = sum(page if j < n - 1 else L - (n - 1) * page for j in kept)
                assert got_lens[i, t, h] == tokens


def test_page_select_long_table():
    """More pages than a CTA holds in shared memory, and far more than are kept."""
    nb, page, d = 120000, 16, 32
    rng = np.random.default_rng(8)
    b, s, db, ds = _bounds_pool(rng, 1000, 1, d)
    table = rng.integers(0, 1000, (1, nb))
    q = torch.randn((1, 2, d), generator=torch.Generator().manual_seed(1))
    out = sl8.page_select(q.to(DEV), db, ds, i32(table), i32([nb * page - 3]), page, 512, 1, 1)
    ids = table[0]
    want = S.page_scores(q[0].numpy(), b[ids, 0, 0].astype(np.int64), b[ids, 0, 1].astype(np.int64), s[ids, 0])
    kept = S.select(want, 512, 1, 1)
    np.testing.assert_array_equal(out["blocks"].cpu().numpy()[0, 0, 0], kept)
    assert out["lens"].item() == 512 * page - 3


@pytest.mark.parametrize("B,lens,max_sel,first,last", [(40, 9000, 5000, 2, 3), (200, 5000, 64, 1, 2), (3, 40000, 30000, 0, 0)])
def test_page_select_wide_tables(B, lens, max_sel, first, last):
    """Tables wider than a CTA holds keys of: long rows, short rows and rows that are kept whole."""
    nb, page, hkv, d = 40000, 16, 2, 32
    rng = np.random.default_rng(B)
    b, s, db, ds = _bounds_pool(rng, 500, hkv, d, coarse=B == 200)
    table = rng.integers(0, 500, (B, nb)).astype(np.int32)
    n = rng.integers(1, lens + 1, B)
    n[0] = lens
    q = torch.randn((B, 2 * hkv, d), generator=torch.Generator().manual_seed(B))
    out = sl8.page_select(q.to(DEV), db, ds, i32(table), i32(n * page - 5), page, max_sel, first, last)
    blocks, pages, got = (out[x].cpu().numpy()[:, 0] for x in ("blocks", "pages", "lens"))
    for i in list(range(min(B, 6))) + [B - 1]:
        ids = table[i, :n[i]]
        for h in range(hkv):
            score = S.page_scores(q[i, 2 * h:2 * h + 2].numpy(), b[ids, h, 0].astype(np.int64), b[ids, h, 1].astype(np.int64),
                                  s[ids, h])
            kept = S.select(score, max_sel, first, last)
            np.testing.assert_array_equal(blocks[i, h], kept + [-1] * (max_sel - len(kept)))
            np.testing.assert_array_equal(pages[i, h, :len(kept)], ids[kept])
            assert got[i, h] == len(kept) * page - (5 if n[i] - 1 in set(kept) else 0)


@pytest.mark.parametrize("first,last", [(4, 4), (8, 0), (0, 8), (1, 0)])
def test_page_select_only_forced_pages_over_a_cluster(first, last):
    """Nothing is left to choose by score, in rows that several CTAs share."""
    nb, page, hkv, d, keep = 2050, 16, 2, 64, first + last
    rng = np.random.default_rng(keep)
    _, _, db, ds = _bounds_pool(rng, 300, hkv, d)
    table = rng.integers(0, 300, (2, nb)).astype(np.int32)
    lens = [nb * page - 1, 700 * page]
    q = torch.randn((2, 2 * hkv, d), generator=torch.Generator().manual_seed(1)).to(DEV)
    for _ in range(5):
        out = sl8.page_select(q, db, ds, i32(table), i32(lens), page, keep, first, last)
        for i, L in enumerate(lens):
            n = -(-L // page)
            kept = [*range(first), *range(n - last, n)]
            for h in range(hkv):
                assert out["blocks"][i, 0, h].tolist() == kept
                assert out["pages"][i, 0, h].tolist() == table[i, kept].tolist()
                assert out["lens"][i, 0, h].item() == keep * page - (n * page - L if last else 0)


def test_page_select_reports_bad_lengths_and_pages():
    b, s = torch.ones((2, 1, 2, 64), dtype=torch.int8, device=DEV), torch.ones((2, 1), device=DEV)
    q = torch.ones((1, 1, 64), device=DEV)
    b[0] = 3
    out = sl8.page_select(q, b, s, i32([[0, 1, 7]]), i32([48]), 16, 2, 1, 0)
    assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
    # page 7 is scored as page 0, above page 1
    assert out["blocks"].tolist() == [[[[0, 2]]]] and out["lens"].item() == 32
    for L, want in ((49, 48), (-1, 0)):
        out = sl8.page_select(q, b, s, i32([[0, 1, 0]]), i32([L]), 16, 4, 1, 0)
        assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
        assert out["lens"].item() == want


# ------------------------------------------------------------------ sparse decode

def _check_attention(out, lse, want, wlse, vmax, n):
    eps = 0 if out.dtype == torch.float32 else torch.finfo(out.dtype).eps / 2
    err = np.abs(np64(out).reshape(want.shape) - want)
    tol = (2.0 ** -11 + 2.0 ** -24 * n) * vmax * (1 + eps) + eps * np.abs(want) + 2.0 ** -25
    assert np.all(err <= tol), (err.max(), np.max(tol))
    got = np64(lse).reshape(wlse.shape)
    dead = np.isinf(wlse)
    assert np.array_equal(got == -np.inf, dead)
    # logits: an exact integer times three fp32 factors; the sum: ex2.approx (2^-22) of each
    assert np.all(np.abs(got[~dead] - wlse[~dead]) <= 1e-5 + 1e-6 * np.abs(wlse[~dead]))
    assert np.all(np64(out).reshape(want.shape)[dead] == 0)


@pytest.mark.parametrize("R,hq,hkv,d,page,max_sel,splits,dtype,odt", [
    (1, 4, 1, 64, 16, 1, 0, torch.bfloat16, torch.float32), (3, 32, 8, 128, 16, 20, 0, torch.bfloat16, torch.bfloat16),
    (5, 6, 2, 64, 48, 7, 1, torch.float16, torch.float16), (2, 16, 1, 128, 64, 9, 3, torch.float32, torch.float32),
    (4, 12, 1, 256, 16, 33, 0, torch.bfloat16, torch.float32), (2, 3, 3, 32, 32, 5, 2, torch.float16, torch.bfloat16),
    (70, 16, 8, 128, 16, 12, 0, torch.bfloat16, torch.bfloat16), (2, 64, 2, 64, 16, 40, 5, torch.bfloat16, torch.float32),
    (300, 2, 2, 64, 16, 3, 0, torch.float16, torch.float16),
    # more than 8 splits: the split kernel and the combine
    (2, 8, 2, 128, 16, 40, 20, torch.bfloat16, torch.float32), (1, 12, 1, 256, 32, 30, 9, torch.float16, torch.float16),
    (1, 3, 3, 32, 16, 64, 30, torch.float32, torch.bfloat16), (1, 4, 1, 64, 64, 520, 0, torch.bfloat16, torch.float32),
    # one CTA a list and more lists than one wave of them
    (240, 4, 2, 128, 48, 5, 0, torch.bfloat16, torch.float32), (500, 8, 1, 64, 16, 20, 0, torch.float16, torch.float32),
    (120, 4, 4, 32, 16, 11, 0, torch.bfloat16, torch.float32), (180, 9, 3, 256, 16, 6, 0, torch.bfloat16, torch.float32)])
def test_sparse_decode(R, hq, hkv, d, page, max_sel, splits, dtype, odt):
    rng = np.random.default_rng(R * 31 + d)
    num_pages = max_sel * 2 + 3
    codes, scales, dc, ds = _pool(rng, num_pages, hkv, page, d)
    pages = np.stack([np.stack([rng.permutation(num_pages)[:max_sel] for _ in range(hkv)]) for _ in range(R)])
    lens = rng.integers(0, max_sel * page + 1, (R, hkv))
    lens[0] = max_sel * page
    if R > 1:
        lens[1] = 0
        lens[1, 0] = 1
    # entries past a list are never read
    for r in range(R):
        for h in range(hkv):
            pages[r, h, -(-lens[r, h] // page):] = -1
    q = torch.randn((R, hq, d), generator=torch.Generator().manual_seed(R)).to(dtype)
    q[-1, -1] = 0
    out, lse = sl8.attn_int8_sparse_decode(q.to(DEV), dc[0], ds[0], dc[1], ds[1], i32(pages), i32(lens), num_splits=splits,
                                           out_dtype=odt, return_lse=True)
    want, wlse = S.sparse_attention(q.float().numpy(), codes[0], scales[0], codes[1], scales[1], pages, lens)
    vmax = np.abs(codes[1].astype(np.float64) * scales[1][..., None]).max()
    _check_attention(out, lse, want, wlse, vmax, max_sel * page)
    again = sl8.attn_int8_sparse_decode(q.to(DEV), dc[0], ds[0], dc[1], ds[1], i32(pages), i32(lens), num_splits=splits,
                                        out_dtype=odt)
    assert torch.equal(out, again)


@pytest.mark.parametrize("R,hq,hkv,d,page,max_sel,splits", [
    (330, 4, 2, 64, 16, 6, 0), (350, 2, 2, 32, 32, 3, 0), (270, 4, 2, 128, 16, 6, 0), (80, 4, 2, 64, 32, 31, 0),
    (20, 8, 2, 32, 16, 70, 0), (110, 2, 1, 64, 64, 9, 8), (330, 2, 2, 64, 16, 9, 2)])
def test_sparse_decode_where_ctas_crowd_an_sm(R, hq, hkv, d, page, max_sel, splits):
    """Every number of CTAs an SM runs, with whole lists and with split ones."""
    test_sparse_decode(R, hq, hkv, d, page, max_sel, splits, torch.bfloat16, torch.float32)


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("splits", [0, 3, 9])
def test_what_lies_past_a_list_does_not_matter(d, splits):
    """NaN and infinite scales and codes of -128 in the rows of the last page past the list, and
    page ids past it that are none."""
    rng = np.random.default_rng(d + splits)
    R, hq, hkv, page, max_sel = 3, 4, 2, 32, 24
    num_pages = R * hkv * max_sel
    _, _, dc, ds = _pool(rng, num_pages, hkv, page, d)
    pages = rng.permutation(num_pages).reshape(R, hkv, max_sel)  # no page in two lists
    lens = np.array([[1, 33], [page * max_sel - 1, 17], [page * 9 + 16, page * 20 + 5]])
    q = torch.randn((R, hq, d), generator=torch.Generator().manual_seed(d)).half().to(DEV)
    call = lambda p: sl8.attn_int8_sparse_decode(q, dc[0], ds[0], dc[1], ds[1], i32(p), i32(lens), num_splits=splits,  # noqa: E731
                                                 return_lse=True)
    want, wl = call(pages)
    for r in range(R):
        for h in range(hkv):
            last, used = pages[r, h, (lens[r, h] - 1) // page], (lens[r, h] - 1) % page + 1
            for i in range(2):
                dc[i][last, h, used:] = -128
                ds[i][last, h, used:] = float("nan")
                ds[i][last, h, used + 1::2] = float("inf")
            pages[r, h, (lens[r, h] - 1) // page + 1:] = 1 << 30
    got, gl = call(pages)
    assert torch.equal(got, want) and torch.equal(gl, wl)


def test_offsets_past_32_bits():
    """A pool of more than 4 GB for each of K and V: the last pages through every operator."""
    hq, hkv, d, page, num_pages = 8, 4, 256, 64, 70000
    k, v = (torch.empty((num_pages, hkv, page, d), dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.empty((num_pages, hkv, page), device=DEV) for _ in range(2))
    b, bs = torch.empty((num_pages, hkv, 2, d), dtype=torch.int8, device=DEV), torch.empty((num_pages, hkv), device=DEV)
    assert k.numel() > 1 << 32
    ids, n = np.array([num_pages - 1, 3, num_pages - 2, num_pages - 7]), 3 * page + 21
    slots = (ids[:, None] * page + np.arange(page)).reshape(-1)[:n]
    g = torch.Generator().manual_seed(3)
    x = torch.randn((n, hkv, 2 * d), generator=g).bfloat16()
    xd = x.to(DEV)
    sl8.rope_append(None, xd[..., :d].contiguous(), xd[..., d:].contiguous(), None, None, i32(slots), k, ks, v, vs)
    sl8.page_bounds(k, ks, i32(ids[None]), i32([n]), b, bs)
    q = torch.randn((1, hq, d), generator=g).bfloat16()
    sel = sl8.page_select(q.to(DEV), b, bs, i32(ids[None]), i32([n]), page, 3, 1, 1)
    out = sl8.attn_int8_sparse_decode(q.to(DEV), k, ks, v, vs, sel["pages"], sel["lens"], out_dtype=torch.float32)
    kc, kscale = S._quant(x[..., :d].float().numpy())
    vc, vscale = S._quant(x[..., d:].float().numpy())
    pad = lambda a: np.concatenate([a, np.zeros((4 * page - n, *a.shape[1:]), a.dtype)]).reshape(4, page, *a.shape[1:]).swapaxes(1, 2)  # noqa: E731,E501
    kc, kscale, vc, vscale = (pad(a) for a in (kc, kscale, vc, vscale))
    for h in range(hkv):
        box = [S.page_bounds(kc[j, h, :n - j * page], kscale[j, h, :n - j * page]) for j in range(4)]
        score = S.page_scores(q[0, 2 * h:2 * h + 2].float().numpy(), np.stack([x[0] for x in box]), np.stack([x[1] for x in box]),
                              np.array([x[2] for x in box]))
        kept = S.select(score, 3, 1, 1)
        assert sel["blocks"][0, 0, h].tolist() == kept and sel["pages"][0, 0, h].tolist() == ids[kept].tolist()
    blocks, lens = sel["blocks"].cpu().numpy()[0], sel["lens"].cpu().numpy()[0]
    want, _ = S.sparse_attention(q.float().numpy(), kc, kscale, vc, vscale, blocks, lens)
    vmax = np.abs(vc.astype(np.float64) * vscale[..., None]).max()
    assert np.all(np.abs(np64(out) - want) <= (2.0 ** -11 + 2.0 ** -24 * n) * vmax)


def test_sparse_decode_of_every_page_is_the_paged_decode():
    rng = np.random.default_rng(6)
    B, hq, hkv, d, page, nb = 4, 16, 4, 128, 16, 30
    lens = [nb * page, 5, 0, 333]
    table, num_pages = _tables(rng, lens, nb, page)
    codes, scales, dc, ds = _pool(rng, num_pages, hkv, page, d)
    q = torch.randn((B, hq, d), generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    out, lse = sl8.attn_int8_sparse_decode(q, dc[0], ds[0], dc[1], ds[1], i32(np.repeat(table[:, None], hkv, 1)),
                                           i32(np.repeat(np.array(lens)[:, None], hkv, 1)), return_lse=True)
    want, wl = sl8.attn_int8_paged_decode(q, dc[0], ds[0], dc[1], ds[1], i32(table), i32(lens), return_lse=True)
    vmax = np.abs(codes[1].astype(np.float64) * scales[1][..., None]).max()
    # two roundings of the probabilities and of the output apart
    assert (out.float() - want.float()).abs().max() <= vmax * (2.0 ** -10 + 2.0 ** -8)
    assert torch.equal(torch.isinf(lse), torch.isinf(wl))
    live = ~torch.isinf(lse)
    assert (lse - wl)[live].abs().max() <= 1e-5


def test_sparse_decode_reports_bad_pages_and_lengths():
    k, s = torch.ones((2, 1, 16, 64), dtype=torch.int8, device=DEV), torch.ones((2, 1, 16), device=DEV)
    q = torch.ones((1, 1, 64), device=DEV)
    for pages, n in (([[[0, 9]]], 32), ([[[0, 1]]], 33), ([[[0, 1]]], -4)):
        out = sl8.attn_int8_sparse_decode(q, k, s, k, s, i32(pages), i32([[n]]))
        assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
        assert torch.isfinite(out).all()


# ------------------------------------------------------------------ one step

def _serving_state(B, hq, hkv, d, page, nb, num_pages, T):
    z = lambda *n, t=torch.int32: torch.zeros(n, dtype=t, device=DEV)  # noqa: E731
    return dict(seq=z(B), new=z(B), release=z(B), table=z(B, nb) - 1, free=torch.arange(num_pages, dtype=torch.int32, device=DEV),
                count=i32([num_pages]), k=z(num_pages, hkv, page, d, t=torch.int8), v=z(num_pages, hkv, page, d, t=torch.int8),
                ks=z(num_pages, hkv, page, t=torch.float32), vs=z(num_pages, hkv, page, t=torch.float32),
                bounds=z(num_pages, hkv, 2, d, t=torch.int8), bs=z(num_pages, hkv, t=torch.float32),
                qkv=z(T, (hq + 2 * hkv) * d, t=torch.bfloat16), dims=(B, hq, hkv, d, page, T))


def _serving_step(s, inv, max_sel, plan=None, sel=None, out=None):
    """One step of one layer: plan, rotary append, bounds, selection and attention of the
    step's last token of every sequence."""
    B, hq, hkv, d, page, T = s["dims"]
    plan = sl8.paged_assign(s["seq"], s["new"], s["table"], s["free"], s["count"], page, T, release=s["release"], out=plan)
    s["seq"].copy_(plan["seqlens"])
    s["count"].copy_(plan["free_count"])
    q, k, v = (x.unflatten(1, (-1, d)) for x in s["qkv"].split([hq * d, hkv * d, hkv * d], 1))
    q = sl8.rope_append(q, k, v, plan["token_pos"], inv, plan["slot_map"], s["k"], s["ks"], s["v"], s["vs"])
    sl8.page_bounds(s["k"], s["ks"], s["table"], s["seq"], s["bounds"], s["bs"], new_lens=plan["granted"], max_new=T)
    last = (plan["cu_new"][1:] - 1).clamp(min=0).long()
    sel = sl8.page_select(q[last], s["bounds"], s["bs"], s["table"], s["seq"], page, max_sel, out=sel)
    out = sl8.attn_int8_sparse_decode(q[last], s["k"], s["ks"], s["v"], s["vs"], sel["pages"], sel["lens"], out=out)
    return plan, sel, out, q


def test_a_serving_loop():
    """Prompts, decode steps, a release and a new request in its slot, against attention in
    64 bits over the cache's own keys and values; the budget holds every page, then not."""
    B, hq, hkv, d, page, nb, T = 5, 8, 2, 64, 16, 12, 256
    for max_sel in (nb, 4):
        s = _serving_state(B, hq, hkv, d, page, nb, 40, T)
        inv = (10000.0 ** (-torch.arange(0, d, 2, device=DEV) / d)).float()
        g = torch.Generator(device=DEV).manual_seed(max_sel)
        steps = [([60, 33, 1, 100, 0], [0] * 5)] + [([1, 1, 1, 1, 0], [0] * 5)] * 18 + [([1, 20, 1, 1, 16], [0, 1, 0, 0, 0])] + \
                [([1] * 5, [0] * 5)] * 3
        for new, release in steps:
            s["new"].copy_(i32(new))
            s["release"].copy_(i32(release))
            s["qkv"].copy_(torch.randn(s["qkv"].shape, generator=g, device=DEV))
            plan, sel, out, q = _serving_step(s, inv, max_sel)
        lens = s["seq"].cpu().numpy()
        assert list(lens) == [82, 23, 23, 122, 19]
        kn, vn, ksn, vsn = (s[x].cpu().numpy() for x in ("k", "v", "ks", "vs"))
        last = (plan["cu_new"][1:] - 1).long()
        pages, n = sel["pages"].cpu().numpy()[:, 0], sel["lens"].cpu().numpy()[:, 0]
        want, _ = S.sparse_attention(q[last].float().cpu().numpy(), kn, ksn, vn, vsn, pages, n)
        tol = (2.0 ** -11 + 2.0 ** -24 * nb * page) * 5.0 + 2.0 ** -8 * np.abs(want)
        assert np.all(np.abs(np64(out) - want) <= tol)
        # the selection is the definition's over the cache as it stands
        table = s["table"].cpu().numpy()
        for b in range(B):
            nblk = -(-lens[b] // page)
            for h in range(hkv):
                box = [S.page_bounds(kn[table[b, j], h, :lens[b] - j * page], ksn[table[b, j], h, :lens[b] - j * page])
                       for j in range(nblk)]
                score = S.page_scores(q[last][b].float().cpu().numpy()[h * 4:h * 4 + 4], np.stack([x[0] for x in box]),
                                      np.stack([x[1] for x in box]), np.array([x[2] for x in box]))
                kept = S.select(score, max_sel, 1, 2)
                assert sel["blocks"][b, 0, h].tolist() == kept + [-1] * (max_sel - len(kept))


def test_two_captured_steps_and_an_eager_one():
    """Two graphs of a step over the same buffers, replayed in turn on a side stream, do what
    eager calls do; graphs of different steps replayed at the same time share nothing."""
    B, hq, hkv, d, page, nb, T = 3, 8, 2, 64, 16, 20, 8
    inv = (10000.0 ** (-torch.arange(0, d, 2, device=DEV) / d)).float()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    runs = []
    for seed in (1, 2, 3):
        s = _serving_state(B, hq, hkv, d, page, nb, 60, T)
        s["new"].fill_(2)
        _serving_step(s, inv, 3)  # warms up what a capture may not do
        torch.cuda.synchronize()
        s["seq"].zero_(), s["table"].fill_(-1), s["count"].fill_(60)
        s["free"].copy_(torch.arange(60)), s["k"].zero_(), s["v"].zero_(), s["ks"].zero_(), s["vs"].zero_()
        s["bounds"].zero_(), s["bs"].zero_()
        g = torch.cuda.CUDAGraph()
        if seed < 3:
            with torch.cuda.graph(g):
                res = _serving_step(s, inv, 3)
        else:
            res = None
        runs.append([s, g, res])
    for step in range(40):
        x = torch.randn(runs[0][0]["qkv"].shape, generator=torch.Generator(device=DEV).manual_seed(step), device=DEV)
        for s, _, _ in runs:
            s["qkv"].copy_(x)
        for st in (side, other):
            st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            runs[0][1].replay()
        with torch.cuda.stream(other):
            runs[1][1].replay()
        runs[2][2] = _serving_step(runs[2][0], inv, 3)
        for st in (side, other):
            torch.cuda.current_stream().wait_stream(st)
        for s, _, res in runs[:2]:
            for a, b in zip(res[1].values(), runs[2][2][1].values()):
                assert torch.equal(a, b), step
            assert torch.equal(res[2], runs[2][2][2]) and torch.equal(s["k"], runs[2][0]["k"]), step
    assert runs[0][0]["seq"].tolist() == [80] * 3


def test_side_stream_and_refusals():
    q = torch.randn((2, 4, 64), device=DEV).half()
    pages, scales = torch.ones((2, 3, 2, 16, 64), dtype=torch.int8, device=DEV), torch.ones((2, 3, 2, 16), device=DEV)
    lists, lens = i32(np.zeros((2, 2, 2))), i32(np.full((2, 2), 20))
    args = (pages[0], scales[0], pages[1], scales[1], lists, lens)
    want = sl8.attn_int8_sparse_decode(q, *args)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = sl8.attn_int8_sparse_decode(q, *args)
    st.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(ValueError):
        sl8.attn_int8_sparse_decode(q.transpose(0, 1), *args)
    with pytest.raises(TypeError):
        sl8.attn_int8_sparse_decode(q, *args[:4], lists.long(), lens)
    with pytest.raises(ValueError):
        sl8.attn_int8_sparse_decode(q, *args[:4], lists, lens[:1])
    with pytest.raises(sl8.SL8Error):
        sl8.attn_int8_sparse_decode(q, *args[:4], i32(np.zeros((2, 2, 64))), lens, num_splits=40,
                                    workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    k = torch.randn((4, 2, 64), device=DEV).half()
    slots = i32([0, 1, 2, 3])
    with pytest.raises(ValueError):
        sl8.rope_append(None, k[..., ::2], k[..., ::2], None, None, slots, *args[:4])
    with pytest.raises(TypeError):
        sl8.rope_append(None, k, k.float(), None, None, slots, *args[:4])
    with pytest.raises(ValueError):
        sl8.rope_append(None, k, k, slots, None, slots, *args[:4])
    with pytest.raises(ValueError):
        sl8.rope_append(k, k, k, i32([0, 1, 2]), torch.ones(32, device=DEV), slots, *args[:4])


# ------------------------------------------------------------------ sparse decode: NaN, ranges and long lists

@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("splits", [0, 1, 3, 8, 9, 20])
def test_nan_logits_reach_the_output(splits, d):
    """An infinite scale with codes of 0, as the append stores a row that holds an infinity, and
    an infinite query row have NaN logits: out and lse of their queries are NaN, as the
    definition has it, and no others' are."""
    rng = np.random.default_rng(d + splits)
    R, hq, hkv, page, max_sel = 8, 4, 2, 32, 40
    num_pages = R * hkv * max_sel
    codes, scales, _, _ = _pool(rng, num_pages, hkv, page, d)
    pages = rng.permutation(num_pages).reshape(R, hkv, max_sel)  # no page in two lists
    lens = rng.integers(page * 30, max_sel * page + 1, (R, hkv))
    lens[4], lens[5, 0], lens[6] = 0, 1, 1
    q = torch.randn((R, hq, d), generator=torch.Generator().manual_seed(d)).half()

    def infinite(i, r, h, t):
        at = pages[r, h, t // page], h, t % page
        codes[i][at], scales[i][at] = 0, np.inf

    infinite(0, 1, 0, lens[1, 0] - 1)             # one key, in the list's last stage
    for t in range(0, 48):
        infinite(0, 2, 1, t)                      # all keys of some warps, before and behind finite ones
    for t in range(lens[3, 0]):
        infinite(0, 3, 0, t)                      # every key
    q[3, 3, 5], q[4, 0, 0] = np.inf, -np.inf      # a query row; one whose list is empty
    infinite(0, 5, 0, 0)                          # the only key
    infinite(1, 6, 1, 0), infinite(1, 7, 0, 77)   # value rows
    dc, ds = ([torch.from_numpy(x).to(DEV) for x in y] for y in (codes, scales))
    out, lse = sl8.attn_int8_sparse_decode(q.to(DEV), dc[0], ds[0], dc[1], ds[1], i32(pages), i32(lens), num_splits=splits,
                                           out_dtype=torch.float32, return_lse=True)
    with np.errstate(invalid="ignore"):
        want, wlse = S.sparse_attention(q.float().numpy(), codes[0], scales[0], codes[1], scales[1], pages, lens)
    nan = np.zeros((R, hq), bool)
    nan[1, :2] = nan[2, 2:] = nan[3, :2] = nan[3, 3] = nan[5, :2] = True
    assert np.array_equal(np.isnan(wlse), nan) and np.array_equal(np.isnan(np64(lse)), nan)
    assert np.array_equal(np64(lse) == -np.inf, np.arange(R)[:, None].repeat(hq, 1) == 4)
    nan[6, 2:] = nan[7, :2] = True
    assert np.array_equal(np.isnan(want), np.broadcast_to(nan[..., None], want.shape))
    assert np.array_equal(np.isnan(np64(out)), np.isnan(want))
    assert np.all(np64(out)[4] == 0)
    vmax = np.abs(codes[1].astype(np.float64) * np.where(np.isinf(scales[1]), 0, scales[1])[..., None]).max()
    tol = (2.0 ** -11 + 2.0 ** -24 * max_sel * page) * vmax
    assert np.all(np.abs(np64(out)[~nan] - want[~nan]) <= tol)


def test_a_length_out_of_range_counts_as_the_whole_list():
    """Also where several splits are joined, and where the length is the largest number."""
    rng = np.random.default_rng(8)
    hq, hkv, d, page, max_sel = 4, 2, 64, 32, 60
    _, _, dc, ds = _pool(rng, 64, hkv, page, d)
    pages = i32(rng.permutation(64)[:max_sel][None, None].repeat(hkv, 1))
    q = torch.randn((1, hq, d), generator=torch.Generator().manual_seed(4)).to(DEV)
    for splits in (1, 4, 12, 40):
        call = lambda n: sl8.attn_int8_sparse_decode(q, dc[0], ds[0], dc[1], ds[1], pages, i32([[n, n]]), num_splits=splits,  # noqa: E731
                                                     return_lse=True)
        want, wl = call(max_sel * page)
        assert sl8.last_device_status()[0] == sl8.SL8_OK and torch.isfinite(wl).all()
        for n in ((1 << 31) - 1, (1 << 31) - 40, max_sel * page + 1):
            got, gl = call(n)
            assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
            assert torch.equal(got, want) and torch.equal(gl, wl), (splits, n)


def test_a_list_of_almost_2_31_tokens():
    """2,047 times the same page of 2^20 tokens: the attention over one, its LSE above by
    log(2047)."""
    hq, d, page, times = 2, 32, 1 << 20, 2047
    g = torch.Generator(device=DEV).manual_seed(7)
    k, v = (torch.randint(-127, 128, (1, 1, page, d), generator=g, device=DEV, dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand((1, 1, page), generator=g, device=DEV) * 0.01 + 0.005 for _ in range(2))
    q = torch.randn((1, hq, d), generator=g, device=DEV)
    lists = torch.zeros((1, 1, times), dtype=torch.int32, device=DEV)
    out, lse = sl8.attn_int8_sparse_decode(q, k, ks, v, vs, lists, i32([[times * page]]), return_lse=True)
    one, lse1 = sl8.attn_int8_sparse_decode(q, k, ks, v, vs, lists[..., :1].contiguous(), i32([[page]]), return_lse=True)
    # 64 splits, ten warps each: a lane adds to its sums once for every 160 tokens, each time off by
    # at most 2^-24 of the sum so far; the values' sum runs over codes offset by 128
    off = times * page / 64 / 160 * 2.0 ** -24
    assert off < 0.02 and (lse - lse1 - np.log(times)).abs().max() <= 2 * off
    vmax = float((v.float() * vs[..., None]).abs().max())
    assert (out - one).abs().max() <= (2.0 ** -10 + 6 * off) * vmax


def _attention_tol(q, codes, scales, pages, lens, want, wlse, dtype):
    """Per channel, from the weights w_t = p_t s_v,t of the normalised probabilities:
    each P' is rounded to fp16, off by 2^-11 of itself or by 2^-24 of the list's largest weight;
    a logit is three fp32 products of an exact integer (3 * 2^-24 of itself), which moves its p
    and the sum alike; ex2.approx and the sum add 2^-20; and the fp32 sums run over V codes offset
    by 128, in which each of a warp's additions of 16 tokens and each of the merge's 20 is off by
    2^-22 of the 255 sum w so far."""
    R, hq, d = q.shape
    hkv, P = codes[0].shape[1], codes[0].shape[2]
    eps = torch.finfo(dtype).eps / 2
    c, sq = S._quant(q)
    tol = np.zeros((R, hq, d))
    for r in range(R):
        for h in range(hkv):
            n = int(lens[r, h])
            if n == 0:
                continue
            ids = pages[r, h, :-(-n // P)]
            rows = lambda x: x[ids, h].astype(np.float64).reshape(-1, *x.shape[3:])[:n]  # noqa: E731
            k, v = rows(codes[0]) * rows(scales[0])[:, None], rows(codes[1])
            for j in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = k @ c[r, j].astype(np.float64) * float(sq[r, j]) / np.sqrt(d)
                w = np.exp(x - wlse[r, j]) * rows(scales[1])
                logit = 2 * 3 * 2.0 ** -24 * np.abs(x).max()
                tol[r, j] = ((2.0 ** -11 + 2.0 ** -20 + logit) * (w @ np.abs(v)) + n * 2.0 ** -24 * 127 * w.max()
                             + (n / 64 + 20) * 2.0 ** -22 * 255 * w.sum())
    return tol * (1 + eps) + eps * np.abs(want) + 2.0 ** -25


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("splits", [1, 3, 8, 12])
def test_a_huge_value_row_of_no_weight(splits, d):
    """Value rows whose scales are 2^18 and 2^60 times the others' and whose probabilities are
    nothing: they take no bits from the other rows, wherever they stand."""
    rng = np.random.default_rng(d * splits)
    R, hq, hkv, page, max_sel = 5, 4, 2, 32, 40
    num_pages = max_sel + 5
    codes, scales, _, _ = _pool(rng, num_pages, hkv, page, d)
    scales[0][:], scales[1][:] = 0.004, rng.random(scales[1].shape) * 0.02 + 0.01
    pages = np.stack([np.stack([rng.permutation(num_pages - 2)[:max_sel] for _ in range(hkv)]) for _ in range(R)])
    pages[3, :, :2] = num_pages - 2, num_pages - 1  # a list that begins with nothing else
    lens = rng.integers(page * 30, max_sel * page + 1, (R, hkv))
    q = rng.integers(50, 128, (R, hq, d)).astype(np.float32) / 16  # all positive
    q[..., 0] = 127.0 / 16
    # the first row of some pages, one in the middle, the last; keys against every query, some 60
    # below the others' logits
    for at, far, row in ((slice(0, -2, 9), 2.0 ** 18, 0), (slice(1, -2, 9), 2.0 ** 18, 17), (slice(2, -2, 9), 2.0 ** 60, 31),
                         (slice(-2, None), 2.0 ** 18, slice(None))):
        codes[0][at, :, row], scales[0][at, :, row] = -127, 0.086 / np.sqrt(d)
        scales[1][at, :, row] *= far
    dc, ds = ([torch.from_numpy(x).to(DEV) for x in y] for y in (codes, scales))
    out, lse = sl8.attn_int8_sparse_decode(torch.from_numpy(q).to(DEV), dc[0], ds[0], dc[1], ds[1], i32(pages), i32(lens),
                                           num_splits=splits, return_lse=True)
    want, wlse = S.sparse_attention(q, codes[0], scales[0], codes[1], scales[1], pages, lens)
    tol = _attention_tol(q, codes, scales, pages, lens, want, wlse, torch.float32)
    err = np.abs(np64(out) - want)
    assert np.all(err <= tol), (err / tol).max()
    assert np.all(np.abs(np64(lse) - wlse) <= 1e-5 + 1e-6 * np.abs(wlse))


@pytest.mark.parametrize("adjacent", [False, True])
def test_slow_and_fast_frequencies_at_far_positions(adjacent):
    """Frequencies down to where no int32 position turns by 1e-6 rad, and up to 1,000 rad a
    position."""
    inv = np.array([2.0 ** -39, 2.0 ** -40, 0.999 * 2.0 ** -40, 2.0 ** -41, 1.7 * 2.0 ** -42, 2.0 ** -45, 1.3 * 2.0 ** -50,
                    2.0 ** -60, 2.0 ** -100, 0.0, -2.0 ** -41, 1.0, -1.0, 3.7, 255.9, 1000.0], np.float32)
    pos = np.array([(1 << 31) - 1, -(1 << 31), 1 << 30, -12345678, 0, 1, 77777777])
    T, h, d = len(pos), 2, 32
    x = torch.randn((T, h, d), generator=torch.Generator().manual_seed(5))
    pages, scales = torch.zeros((2, 1, h, T, d), dtype=torch.int8, device=DEV), torch.zeros((2, 1, h, T), device=DEV)
    out = sl8.rope_append(x.to(DEV), x.to(DEV), x.to(DEV), i32(pos), torch.from_numpy(inv).to(DEV), i32(np.arange(T)),
                          pages[0], scales[0], pages[1], scales[1], adjacent=adjacent)
    # the definition's angle in 64 bits is off by 2^-53 of itself: 1000 * 2^31 * 2^-53 = 2.4e-4 rad is
    # too much, so whole turns are taken out of exact integers first
    turns = np.array([[float(_turns(int(p), float(f))) for f in inv] for p in pos]) * 2 * np.pi
    host = x.double().numpy()
    a, b = (slice(0, d, 2), slice(1, d, 2)) if adjacent else (slice(0, d // 2), slice(d // 2, d))
    c, s = np.cos(turns)[:, None], np.sin(turns)[:, None]
    want = np.empty_like(host)
    want[..., a], want[..., b] = host[..., a] * c - host[..., b] * s, host[..., b] * c + host[..., a] * s
    assert np.all(np.abs(np64(out) - want) <= _rotation_tol(host, d, adjacent) + 2.0 ** -24 * np.abs(want))


def _turns(pos, f):
    """pos * f / (2 pi) mod 1, from integers: 1 / (2 pi) to 200 bits."""
    from fractions import Fraction
    inv_2pi = Fraction(0x28BE60DB9391054A7F09D5F47D4D377036D8A5664F10E4107F9458, 1 << 216)
    x = Fraction(f) * pos * inv_2pi
    return x - round(x)


@pytest.mark.parametrize("max_tokens", [8, 20000])
def test_paged_assign_of_pages_past_2_31_slots(max_tokens):
    """A page id whose slots do not fit 31 bits (a pool too large, an entry that is none) is
    recorded and its tokens get no slot, instead of another page's."""
    last = (1 << 27) - 1  # pages of 16 tokens: the slots of this one end at 2^31 - 1
    ids = [last, last + 1, (1 << 28) + 3, -1, (1 << 31) - 1]
    table = i32(np.array(ids + [5])[:, None].repeat(2, 1))
    ctx, new = [14, 3, 2, 1, 0, 15], [1, 1, 1, 1, 1, 2]
    out = sl8.paged_assign(i32(ctx), i32(new), table, i32([(1 << 28) - 2, (1 << 31) - 7]), i32([2]), 16, max_tokens)
    assert sl8.last_device_status()[0] == sl8.SL8_ERR_DEVICE_ARG
    assert out["granted"].tolist() == new and out["free_count"].item() == 0
    assert out["slot_map"][:8].tolist() == [(1 << 31) - 2, -1, -1, -1, -1, 5 * 16 + 15, -1, -1]
    assert out["token_pos"][:8].tolist() == [14, 3, 2, 1, 0, 15, 16, 0]
    out = sl8.paged_assign(i32([14]), i32([2]), i32([[last]]), i32([1]), i32([0]), 16, max_tokens)
    assert sl8.last_device_status()[0] == sl8.SL8_OK
    assert out["slot_map"][:3].tolist() == [(1 << 31) - 2, (1 << 31) - 1, -1]


@pytest.mark.parametrize("d,hq,hkv,splits", [(32, 2, 1, 1), (64, 4, 2, 0), (64, 8, 1, 5), (128, 4, 2, 1), (128, 8, 2, 8), (128, 2, 1, 12),
                                            (256, 3, 1, 3), (256, 2, 1, 9)])
def test_every_value_row_counts(d, hq, hkv, splits):
    """Lists of some 4,096 tokens whose value rows each hold one channel, so that a row that is
    lost, doubled or exchanged moves its channel by more than the roundings of all others."""
    rng = np.random.default_rng(d + splits)
    R, page, max_sel = 2, 32, 128
    num_pages = max_sel + 6
    codes, scales, _, _ = _pool(rng, num_pages, hkv, page, d)
    codes[1][:] = 0
    at = rng.integers(0, d, (num_pages, hkv, page))
    np.put_along_axis(codes[1], at[..., None], rng.choice([-1, 1], at.shape)[..., None] * rng.integers(100, 128, at.shape)[..., None], -1)
    scales[0][:], scales[1][:] = 0.01, rng.random(scales[1].shape) * 0.02 + 0.01
    pages = np.stack([np.stack([rng.permutation(num_pages)[:max_sel] for _ in range(hkv)]) for _ in range(R)])
    lens = rng.integers(page * 120, max_sel * page + 1, (R, hkv))
    q = rng.standard_normal((R, hq, d)).astype(np.float32)
    dc, ds = ([torch.from_numpy(x).to(DEV) for x in y] for y in (codes, scales))
    out, lse = sl8.attn_int8_sparse_decode(torch.from_numpy(q).to(DEV), dc[0], ds[0], dc[1], ds[1], i32(pages), i32(lens),
                                           num_splits=splits, return_lse=True)
    want, wlse = S.sparse_attention(q, codes[0], scales[0], codes[1], scales[1], pages, lens)
    tol = _attention_tol(q, codes, scales, pages, lens, want, wlse, torch.float32)
    # what half of the rows add to their channels is above twice what the channels may be off
    k = (codes[0][pages[0, 0], 0].astype(np.float64) * 0.01).reshape(-1, d)[:lens[0, 0]]
    c, sq = S._quant(q[0, 0])
    w = np.exp(k @ c.astype(np.float64) * float(sq) / np.sqrt(d) - wlse[0, 0]) * scales[1][pages[0, 0], 0].reshape(-1)[:lens[0, 0]]
    assert np.median(w) * 100 > 2 * tol[0, 0].max()
    assert np.all(np.abs(np64(out) - want) <= tol)
    assert np.all(np.abs(np64(lse) - wlse) <= 1e-5 + 1e-6 * np.abs(wlse))


@pytest.mark.parametrize("G,hkv,d,splits", [(11, 2, 128, 0), (13, 1, 64, 1), (22, 1, 32, 3), (11, 1, 256, 10), (26, 2, 128, 12)])
def test_sparse_decode_of_heads_that_do_not_divide_by_eight(G, hkv, d, splits):
    test_sparse_decode(3, G * hkv, hkv, d, 16, 40, splits, torch.bfloat16, torch.float32)


def test_sparse_decode_of_many_split_lists():
    """More lists than the split kernel sorts by length."""
    test_sparse_decode(90, 16, 8, 64, 16, 30, 9, torch.bfloat16, torch.float32)


@pytest.mark.parametrize("T,G,d,page,dtype,splits", [(1, 4, 64, 16, torch.float32, 0), (3, 4, 128, 32, torch.bfloat16, 0),
                                                     (5, 2, 64, 16, torch.float16, 4), (4, 16, 32, 48, torch.float32, 0),
                                                     (2, 1, 256, 64, torch.bfloat16, 11)])
def test_drafts_from_selection_to_attention(T, G, d, page, dtype, splits):
    """q [B, T, Hq, d]: the drafts' own lists as the selection returns them, into the attention,
    with out and lse of the caller's."""
    rng = np.random.default_rng(T * d)
    B, hkv, nb, max_sel = 3, 2, 24, 9
    lens = [nb * page - 3, 7 * page + T, T - 1]
    table, num_pages = _tables(rng, lens, nb, page)
    codes, scales, dc, ds = _pool(rng, num_pages, hkv, page, d)
    bounds = torch.zeros((num_pages, hkv, 2, d), dtype=torch.int8, device=DEV)
    bs = torch.zeros((num_pages, hkv), device=DEV)
    sl8.page_bounds(dc[0], ds[0], i32(table), i32(lens), bounds, bs)
    q = torch.randn((B, T, G * hkv, d), generator=torch.Generator().manual_seed(T)).to(dtype)
    sel = sl8.page_select(q.to(DEV), bounds, bs, i32(table), i32(lens), page, max_sel, 1, 1)
    out = torch.empty((B, T, G * hkv, d), dtype=torch.float32, device=DEV)
    lse = torch.empty((B, T, G * hkv), device=DEV)
    got = sl8.attn_int8_sparse_decode(q.to(DEV), dc[0], ds[0], dc[1], ds[1], sel["pages"], sel["lens"], num_splits=splits,
                                      out=out, lse=lse, return_lse=True)
    assert got[0] is out and got[1] is lse
    # the definition, from lists of its own
    pages, n = np.full((B * T, hkv, max_sel), -1), np.zeros((B * T, hkv), int)
    x = q.float().numpy()
    for b in range(B):
        for t in range(T):
            L = max(0, lens[b] - (T - 1 - t))
            ids = table[b, :-(-L // page)]
            for h in range(hkv):
                box = [S.page_bounds(codes[0][p, h, :lens[b] - j * page], scales[0][p, h, :lens[b] - j * page]) for j, p in enumerate(ids)]
                score = S.page_scores(x[b, t, h * G:(h + 1) * G], np.stack([y[0] for y in box]), np.stack([y[1] for y in box]),
                                      np.array([y[2] for y in box])) if L else []
                kept = S.select(score, max_sel, 1, 1)
                pages[b * T + t, h, :len(kept)] = ids[kept]
                n[b * T + t, h] = len(kept) * page - (len(ids) * page - L)  # the last page is always kept
    assert np.array_equal(sel["pages"].cpu().numpy().reshape(pages.shape), pages)
    assert np.array_equal(sel["lens"].cpu().numpy().reshape(n.shape), n)
    flat = x.reshape(B * T, G * hkv, d)
    want, wlse = S.sparse_attention(flat, codes[0], scales[0], codes[1], scales[1], pages, n)
    tol = _attention_tol(flat, codes, scales, pages, n, want, wlse, torch.float32)
    assert np.all(np.abs(np64(out).reshape(want.shape) - want) <= tol)
    got, dead = np64(lse).reshape(wlse.shape), np.isinf(wlse)
    assert np.array_equal(got == -np.inf, dead) and np.all(np64(out).reshape(want.shape)[dead] == 0)
    assert np.all(np.abs(got[~dead] - wlse[~dead]) <= 1e-5 + 1e-6 * np.abs(wlse[~dead]))


def test_a_contiguous_cache_from_append_to_decode():
    """page_size = Lmax: what the append stores is what attn_int8_decode reads, against attention in
    64 bits over the quantised rows."""
    B, hq, hkv, d, L, cap = 3, 8, 2, 128, 50, 64
    lens = [50, 1, 33]
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn((B * L, hkv, d), generator=g).bfloat16() for _ in range(2))
    q = torch.randn((B, hq, d), generator=g).bfloat16()
    kc, vc = (torch.zeros((B, hkv, cap, d), dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((B, hkv, cap), device=DEV) for _ in range(2))
    slots = torch.cat([torch.where(torch.arange(L) < n, torch.arange(L) + cap * b, -1) for b, n in enumerate(lens)])
    sl8.rope_append(None, k.to(DEV), v.to(DEV), None, None, i32(slots), kc, ks, vc, vs)
    out, lse = sl8.attn_int8_decode(q.to(DEV), kc, ks, vc, vs, i32(lens), out_dtype=torch.float32, return_lse=True)
    rows = [S._quant(x.view(B, L, hkv, d).transpose(1, 2).float().numpy()) for x in (k, v)]
    codes, scales = [r[0] for r in rows], [r[1] for r in rows]
    pages, n = np.arange(B)[:, None, None].repeat(hkv, 1), np.array(lens)[:, None].repeat(hkv, 1)
    want, wlse = S.sparse_attention(q.float().numpy(), codes[0], scales[0], codes[1], scales[1], pages, n)
    tol = _attention_tol(q.float().numpy(), codes, scales, pages, n, want, wlse, torch.float32)
    assert np.all(np.abs(np64(out) - want) <= tol)
    assert np.all(np.abs(np64(lse) - wlse) <= 1e-5 + 1e-6 * np.abs(wlse))


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("R,splits", [(1, 0), (4, 1), (300, 0), (2, 2), (3, 10)])
def test_fp32_outputs_keep_more_than_fp16_of_the_weights(R, splits, d):
    """Short lists, flat and peaked, with fp32 queries and outputs: what rounding the weights to
    fp16 alone would leave is above the bound."""
    rng = np.random.default_rng(d + R)
    hq, hkv, page, max_sel = 4, 2, 16, 10
    num_pages = 40
    codes, scales, _, _ = _pool(rng, num_pages, hkv, page, d)
    scales[0][:], scales[1][:] = 0.02, rng.random(scales[1].shape) * 0.02 + 0.01
    pages = np.stack([np.stack([rng.permutation(num_pages)[:max_sel] for _ in range(hkv)]) for _ in range(R)])
    lens = rng.integers(1, max_sel * page + 1, (R, hkv))
    q = (rng.standard_normal((R, hq, d)) * np.array([0.05, 0.3, 1, 2])[None, :, None]).astype(np.float32)
    dc, ds = ([torch.from_numpy(x).to(DEV) for x in y] for y in (codes, scales))
    out, lse = sl8.attn_int8_sparse_decode(torch.from_numpy(q).to(DEV), dc[0], ds[0], dc[1], ds[1], i32(pages), i32(lens),
                                           num_splits=splits, return_lse=True)
    want, wlse = S.sparse_attention(q, codes[0], scales[0], codes[1], scales[1], pages, lens)
    # as _attention_tol, but 2^-22 for the weights, and for the offset codes' sums two additions
    # a unit of 16 tokens a warp and four for the warps
    tol, coarse = np.zeros(want.shape), 0.0
    c, sq = S._quant(q)
    for r in range(R):
        for j in range(hq):
            h, n = j // (hq // hkv), int(lens[r, j // (hq // hkv)])
            ids = pages[r, h, :-(-n // page)]
            k, v = (x[ids, h].astype(np.float64).reshape(-1, d)[:n] for x in codes)
            ks, vs = (x[ids, h].astype(np.float64).reshape(-1)[:n] for x in scales)
            x = k @ c[r, j].astype(np.float64) * ks * float(sq[r, j]) / np.sqrt(d)
            w = np.exp(x - wlse[r, j]) * vs
            tol[r, j] = ((2.0 ** -22 + 2.0 ** -20 + 6 * 2.0 ** -24 * np.abs(x).max()) * (w @ np.abs(v)) + n * 2.0 ** -24 * 127 * w.max()
                         + (2 * -(-n // 64) + 4) * 2.0 ** -22 * 255 * w.sum())
            half = w.astype(np.float16).astype(np.float64)  # weights of some 2^-7: normal numbers of fp16
            coarse = max(coarse, (np.abs((half - w) @ v) / tol[r, j]).max())
    assert R == 1 or coarse > 1.5
    err = np.abs(np64(out) - want)
    assert np.all(err <= tol), (err / tol).max()
    assert np.all(np.abs(np64(lse) - wlse) <= 1e-5 + 1e-6 * np.abs(wlse))
