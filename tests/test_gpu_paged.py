"""Rotary positions and the paged cache (append, read-back, attention) through the C ABI, against the
float64 model in paged_model.py."""
import math

import numpy as np
import pytest
import torch

import paged_model as M
from head_partitioned_sparse_b200 import binding as B

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "f32": torch.float32}
KDT = {"bf16": B.SPA_BF16, "f32": B.SPA_F32}
FMT = {"int4": B.SPA_PAGE_INT4, "bf16": B.SPA_PAGE_BF16}
LAYOUT = {"half": B.SPA_ROPE_HALF, "interleaved": B.SPA_ROPE_INTERLEAVED}
SCALING = {"plain": B.SPA_ROPE_PLAIN, "linear": B.SPA_ROPE_LINEAR, "base": B.SPA_ROPE_BASE,
           "bands": B.SPA_ROPE_BANDS, "ramp": B.SPA_ROPE_RAMP}
EXTRA = {"plain": {}, "linear": dict(factor=4.0), "base": dict(factor=8.0),
         "bands": dict(factor=8.0, low=1.0, high=4.0, orig_ctx=8192),
         "ramp": dict(factor=16.0, low=1.0, high=32.0, orig_ctx=4096, magnitude=1.27)}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


class Rope:
    def __init__(self, rot=128, layout="half", scaling="plain", theta=500000.0):
        self.model = dict(rot=rot, layout=layout, scaling=scaling, theta=theta, **EXTRA[scaling])
        self.h = B.spa_rope_create(B.make_rope_config(rot_dim=rot, layout=LAYOUT[layout], scaling=SCALING[scaling],
                                                      theta=theta, **EXTRA[scaling]))

    def __enter__(self):
        return self

    def __exit__(self, *a):
        B.spa_rope_destroy(self.h)


class Paged:
    """A paged handle, its pool and a block table over pages in random order."""

    def __init__(self, *, Bsz, Hq, Hkv, fmt, page, max_pages, dtype="bf16", rope=None, spare=2, seed=0, fill=None):
        self.n_pages = Bsz * max_pages + spare
        self.cfg = B.make_paged_config(max_batch=Bsz, n_q_heads=Hq, n_kv_heads=Hkv, kv_dtype=KDT[dtype],
                                       page_format=FMT[fmt], page_size=page, n_pages=self.n_pages, max_pages=max_pages)
        self.h = B.spa_paged_create(self.cfg, rope.h if rope else None)
        self.B, self.Hq, self.Hkv, self.fmt, self.page, self.dtype = Bsz, Hq, Hkv, fmt, page, dtype
        self.rope = rope.model if rope else None
        rng = np.random.default_rng(seed)
        self.table = rng.permutation(self.n_pages)[:Bsz * max_pages].reshape(Bsz, max_pages).astype(np.int32)
        shape = (self.n_pages, Hkv, page // 16, M.block_bytes(fmt))
        data = rng.integers(0, 256, shape, dtype=np.uint8) if fill is None else np.full(shape, fill, np.uint8)
        self.pool = M.Pool(data, fmt, page)
        self.dtable = torch.from_numpy(self.table).cuda()
        self.pages = torch.from_numpy(data.copy()).cuda()
        assert B.spa_paged_page_bytes(self.cfg) * self.n_pages == self.pages.numel()

    def close(self):
        B.spa_paged_destroy(self.h)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    def q_model(self, q, L):
        q = np.asarray(q, np.float64)
        return M.rotate(q, float(max(L - 1, 0)), **self.rope) if self.rope else q

    def append_model(self, k, v, starts, counts):
        """k, v float64 [B][Hkv][T][128]."""
        for b in range(len(counts)):
            for i in range(int(counts[b])):
                pos = int(starts[b]) + i
                kk = M.rotate(k[b, :, i], float(pos), **self.rope) if self.rope else k[b, :, i]
                for g in range(self.Hkv):
                    self.pool.put(self.table, b, g, pos, kk[g], v[b, g, i])


def i64(x):
    return torch.tensor(list(x), dtype=torch.int64, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------------------------------------ rotary
ROPE_CASES = [
    # dtype, B, T, H, d, rot, layout, order, scaling, transpose
    ("bf16", 1, 1, 1, 128, 128, "half", "heads", "plain", False),
    ("bf16", 2, 7, 5, 128, 128, "half", "tokens", "bands", False),
    ("bf16", 2, 7, 5, 128, 128, "interleaved", "tokens", "ramp", True),
    ("bf16", 1, 33, 3, 96, 64, "half", "heads", "linear", True),
    ("bf16", 1, 33, 9, 80, 36, "half", "tokens", "base", False),        # 2-element chunks
    ("bf16", 1, 5, 2, 130, 66, "interleaved", "heads", "plain", False),  # 2-element chunks
    ("bf16", 1, 5, 2, 67, 14, "half", "tokens", "plain", False),        # single elements
    ("bf16", 1, 5, 2, 67, 14, "interleaved", "tokens", "plain", True),
    ("bf16", 3, 700, 40, 64, 64, "half", "tokens", "plain", False),     # heads grouped in a thread
    ("bf16", 2, 1200, 33, 128, 32, "interleaved", "heads", "bands", False),
    ("f32", 1, 1, 1, 2, 2, "half", "heads", "plain", False),
    ("f32", 2, 9, 3, 128, 128, "half", "heads", "ramp", False),
    ("f32", 2, 9, 3, 80, 36, "half", "tokens", "bands", True),
    ("f32", 1, 17, 3, 75, 10, "interleaved", "tokens", "linear", False),
    ("f32", 1, 17, 3, 75, 10, "half", "tokens", "linear", True),
    ("f32", 1, 3, 2, 512, 512, "interleaved", "heads", "plain", False),
]


def rope_bound(x, y, dtype, m):
    """Half a step of the output, and 4e-7 of both elements of the pair: cos and sin are off by at most 1.6e-7 (the
    angle in units of pi rounded to float32, the function, the magnitude) and the products and their sum by 2^-24 each."""
    big = np.abs(x).max(-1, keepdims=True)
    return HALF_STEP[dtype] * np.abs(y) + 2 * 4e-7 * m * big


@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope_matches_the_definition(case):
    dtype, Bs, T, H, d, rot, layout, order, scaling, tr = case
    g = torch.Generator(device="cuda").manual_seed(7)
    shape = (Bs, H, T, d) if order == "heads" else (Bs, T, H, d)
    x = torch.randn(shape, generator=g, device="cuda", dtype=TDT[dtype])
    y = torch.full_like(x, float("nan"))
    starts = [5, 1 << 20, (1 << 24) - T][:Bs]
    strides = (T * H * d, H * d, d) if order == "tokens" else None
    with Rope(rot, layout, scaling) as r:
        B.spa_rope_apply(r.h, x, y, Bs, T, H, d, KDT[dtype], start_pos=i64(starts), x_strides=strides,
                         y_strides=strides, transpose=tr)
        xs = f64(x) if order == "heads" else f64(x).transpose(0, 2, 1, 3)
        got = f64(y) if order == "heads" else f64(y).transpose(0, 2, 1, 3)
        pos = np.array(starts, np.float64)[:, None, None] + np.arange(T)
        want = M.rotate(xs, pos, transpose=tr, **r.model)
        m = max(1.0, r.model.get("magnitude", 1.0))
    assert (np.abs(got - want) <= rope_bound(xs, want, dtype, m)).all()
    assert np.array_equal(got[..., rot:], xs[..., rot:])


def test_rope_positions_of_each_token_in_place_unaligned_and_broadcast():
    H, T, d, rot = 3, 6, 128, 128
    pos = torch.tensor([[0, 3, 3, -17, 1 << 30, 12345]], device="cuda")
    with Rope() as r:
        # one element past a 16-byte boundary, written in place; what lies around stays
        buf = torch.randn(H * T * d + 2, device="cuda", dtype=torch.bfloat16)
        before = buf.clone()
        x = buf[1:-1]
        B.spa_rope_apply(r.h, x, x, 1, T, H, d, B.SPA_BF16, positions=pos)
        xs = f64(before[1:-1]).reshape(H, T, d)
        want = M.rotate(xs, pos.cpu().numpy()[0], **r.model)
        assert (np.abs(f64(x).reshape(H, T, d) - want) <= rope_bound(xs, want, "bf16", 1.0)).all()
        assert torch.equal(buf[:1], before[:1]) and torch.equal(buf[-1:], before[-1:])
        # one key head read by every output head (stride 0)
        k = torch.randn(T, d, device="cuda")
        y = torch.empty(H, T, d, device="cuda")
        B.spa_rope_apply(r.h, k, y, 1, T, H, d, B.SPA_F32, positions=pos, x_strides=(0, d, 0))
        want = M.rotate(f64(k), pos.cpu().numpy()[0], **r.model)
        for h in range(H):
            assert (np.abs(f64(y[h]) - want) <= rope_bound(f64(k), want, "f32", 1.0)).all()


def test_rope_transpose_is_the_gradient():
    """<gy, R x> = <R^T gy, x>, and central differences of sum(gy * R x) give R^T gy."""
    Bs, T, H, d, rot = 1, 4, 2, 40, 24
    with Rope(rot, "interleaved", "ramp") as r:
        x, gy = torch.randn(2, Bs, H, T, d, device="cuda")
        gx, y = torch.empty_like(x), torch.empty_like(x)
        go = lambda a, o, tr: B.spa_rope_apply(r.h, a, o, Bs, T, H, d, B.SPA_F32, start_pos=i64([777]), transpose=tr)
        go(x, y, False)
        go(gy, gx, True)
        n = x.numel()
        scale = float((gy.double().abs() * y.double().abs()).sum())
        assert abs(float((gy.double() * y.double()).sum() - (gx.double() * x.double()).sum())) <= 4e-6 * scale
        # the map is linear, so a difference has no error but rounding: 2^-24 of values of size ~4, over 2 eps
        flat, eps = x.view(-1), 0.5
        for i in range(0, n, 37):
            out = []
            for sgn in (1, -1):
                z = flat.clone()
                z[i] += sgn * eps
                go(z.view_as(x), y, False)
                out.append(float((gy.double() * y.double()).sum()))
            assert abs((out[0] - out[1]) / (2 * eps) - float(gx.view(-1)[i])) <= 1e-4


def test_rope_frequencies():
    for scaling in SCALING:
        for rot in (128, 36):
            with Rope(rot, "half", scaling, theta=10000.0) as r:
                f = np.array(B.spa_rope_inv_freq(r.h, rot // 2))
                want = M.frequencies(**{k: v for k, v in r.model.items() if k not in ("layout", "magnitude")})
                assert np.allclose(f, want, rtol=1e-13, atol=0)


# ------------------------------------------------------------------------------------------------ append and read
def rows_of(seed, shape, dtype, order="heads"):
    """Gaussian rows with rounding ties, outliers and a zero row; [B][Hkv][T][128] views in either memory order."""
    Bs, Hkv, T, _ = shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    mem = torch.randn((Bs, T, Hkv, 128) if order == "tokens" else shape, generator=g, device="cuda")
    x = mem.transpose(1, 2) if order == "tokens" else mem
    x[..., 5] *= 20
    x[:, :, ::3, 64:] = (x[:, :, ::3, 64:] * 8).round() / 8 * 0.875     # many values on a quarter of their scale
    x[0, 0, 0, 32:] = 0
    x[0, -1, T - 1, :] = 0
    return (mem.to(TDT[dtype]).transpose(1, 2) if order == "tokens" else mem.to(TDT[dtype]))


def strides_of(x):
    return (x.stride(0), x.stride(2), x.stride(1))


APPEND_CASES = [
    # fmt, dtype, B, Hkv, T, page, start, counts, rope (rot, layout, scaling) or None, order
    ("int4", "bf16", 1, 1, 1, 16, [0], None, (128, "half", "plain"), "heads"),
    ("int4", "bf16", 3, 2, 37, 16, [5, 0, 31], [37, 0, 12], (128, "half", "bands"), "tokens"),
    ("int4", "bf16", 2, 9, 20, 48, [47, 100], None, (128, "interleaved", "ramp"), "tokens"),
    ("int4", "bf16", 2, 3, 18, 32, [1, 15], [1, 18], (64, "half", "linear"), "heads"),
    ("int4", "bf16", 1, 2, 18, 64, [60], None, (36, "half", "base"), "tokens"),
    ("int4", "bf16", 1, 2, 18, 64, [60], None, (18, "interleaved", "plain"), "heads"),
    ("int4", "bf16", 1, 4, 33, 64, [3], None, None, "tokens"),
    ("int4", "f32", 2, 2, 33, 16, [9, 16], None, (128, "half", "plain"), "heads"),
    ("int4", "f32", 1, 3, 21, 16, [1 << 15], None, (100, "half", "ramp"), "tokens"),
    ("int4", "f32", 1, 3, 21, 80, [3], None, None, "heads"),
    ("bf16", "bf16", 2, 3, 35, 16, [7, 0], [35, 16], (128, "half", "bands"), "tokens"),
    ("bf16", "bf16", 1, 1, 9, 48, [40], None, None, "heads"),
    ("bf16", "f32", 2, 2, 17, 32, [0, 100], None, (128, "interleaved", "plain"), "tokens"),
    ("bf16", "f32", 1, 2, 17, 32, [0], None, (20, "half", "plain"), "heads"),
]


@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_append_and_read(case):
    """Every byte of the pool against the model (4 bits: equal; bf16: within the rotation's float32 error of a
    half step), the bytes around untouched, and the rows read back."""
    fmt, dtype, Bs, Hkv, T, page, start, counts, rope, order = case
    mp = (max(start) + T + page - 1) // page + 1
    k, v = rows_of(1, (Bs, Hkv, T, 128), dtype, order), rows_of(2, (Bs, Hkv, T, 128), dtype, order)
    r = Rope(*rope) if rope else None
    with Paged(Bsz=Bs, Hq=Hkv, Hkv=Hkv, fmt=fmt, page=page, max_pages=mp, dtype=dtype, rope=r) as P:
        n = None if counts is None else i64(counts)
        cnt = [T] * Bs if counts is None else counts
        B.spa_kv_append_paged(P.h, k, v, i64(start), Bs, T, P.dtable, P.pages, n_new=n, k_strides=strides_of(k),
                              v_strides=strides_of(v))
        before = P.pool.data.copy()
        P.append_model(f64(k), f64(v), start, cnt)
        got = P.pages.cpu().numpy()
        if fmt == "int4":
            assert np.array_equal(got, P.pool.data)
        else:
            gp = M.Pool(got, fmt, page)
            m = max(1.0, P.rope.get("magnitude", 1.0)) if P.rope else 1.0
            for b in range(Bs):
                for g in range(Hkv):
                    pos = range(start[b], start[b] + cnt[b])
                    gk, gv = gp.rows(P.table, b, g, pos)
                    x = f64(k)[b, g, :cnt[b]]
                    want = M.rotate(x, np.array(pos, np.float64), **P.rope) if P.rope else x
                    if len(x):
                        assert (np.abs(gk - want) <= HALF_STEP["bf16"] * np.abs(want) + 8e-7 * m * np.abs(x).max(-1, keepdims=True)).all()
                    assert np.array_equal(gv, M.rne_bf16(f64(v)[b, g, :cnt[b]]))
            assert not ((got != before) & ~written_mask(P, start, cnt)).any()
        # read back a range that begins before the rows and ends behind them, into the middle of larger tensors
        kr = torch.full((Bs, Hkv, T + 3, 128), 7.0, device="cuda", dtype=TDT[dtype])
        vr = torch.full((Bs, T + 3, Hkv, 128), 7.0, device="cuda", dtype=TDT[dtype])
        B.spa_kv_read_paged(P.h, P.pages, P.dtable, i64(start), Bs, T, kr, vr, n_rows=n, k_strides=strides_of(kr),
                            v_strides=(vr.stride(0), vr.stride(1), vr.stride(2)))
        B.spa_paged_status(P.h)
        gp = M.Pool(got, fmt, page)
        for b in range(Bs):
            for g in range(Hkv):
                kk, vv = gp.rows(P.table, b, g, range(start[b], start[b] + cnt[b]))
                to = (lambda a: M.rne_bf16(a)) if dtype == "bf16" else (lambda a: a)
                assert np.array_equal(f64(kr[b, g, :cnt[b]]), to(kk))
                assert np.array_equal(f64(vr[b, :cnt[b], g]), to(vv))
                assert (kr[b, g, cnt[b]:] == 7).all() and (vr[b, cnt[b]:, g] == 7).all()
    if r:
        B.spa_rope_destroy(r.h)


def written_mask(P, start, cnt):
    w = np.zeros(P.pool.data.shape, bool)
    for b in range(len(cnt)):
        for pos in range(start[b], start[b] + cnt[b]):
            r = pos % 16
            blk = w[P.table[b, pos // P.page], :, pos % P.page // 16]
            for part in (0, 1):
                blk[:, 4096 * part + 256 * r:4096 * part + 256 * r + 256] = True
    return w


def test_append_int4_special_values():
    """Zero, tiny, huge, infinite and NaN groups; a NaN or infinity spoils its own group (and its pair's) only."""
    T = 8
    k = torch.randn(1, 1, T, 128, device="cuda")
    v = torch.randn(1, 1, T, 128, device="cuda")
    for x in (k, v):
        x[0, 0, 0] = 0
        x[0, 0, 1] = 1e-36
        x[0, 0, 2, 3] = 3e38
        x[0, 0, 3, 8] = float("inf")
        x[0, 0, 4, 127] = float("nan")
        x[0, 0, 5] = 2.0 ** -100
        x[0, 0, 6, 40] = -float("inf")
        x[0, 0, 7] = torch.arange(128, device="cuda") % 15 - 7.0       # scale 1 exactly
    with Paged(Bsz=1, Hq=1, Hkv=1, fmt="int4", page=16, max_pages=1, dtype="f32") as P:
        B.spa_kv_append_paged(P.h, k, v, i64([4]), 1, T, P.dtable, P.pages)
        with np.errstate(all="ignore"):
            P.append_model(f64(k), f64(v), [4], [T])
        assert np.array_equal(P.pages.cpu().numpy(), P.pool.data)
    with Rope() as r, Paged(Bsz=1, Hq=1, Hkv=1, fmt="int4", page=16, max_pages=1, dtype="f32", rope=r) as P:
        B.spa_kv_append_paged(P.h, k, v, i64([4]), 1, T, P.dtable, P.pages)
        kr, vr = torch.empty_like(k), torch.empty_like(v)
        B.spa_kv_read_paged(P.h, P.pages, P.dtable, i64([4]), 1, T, kr, vr)
        bad = np.zeros((T, 128), bool)
        for row, d in ((3, 8), (4, 127), (6, 40)):
            for dd in (d, d ^ 64):
                bad[row] |= M.GROUP_K == M.GROUP_K[dd]
        assert np.array_equal(np.isnan(f64(kr)[0, 0]), bad)
        assert (f64(kr)[0, 0, :2] == 0).all()


def test_append_rows_out_of_range_are_skipped_and_reported():
    T, page = 20, 16
    k = torch.randn(2, 2, T, 128, device="cuda", dtype=torch.bfloat16)
    with Paged(Bsz=2, Hq=2, Hkv=2, fmt="int4", page=page, max_pages=2) as P:
        before = P.pages.clone()
        # sequence 0 runs past its two pages, sequence 1 starts before 0
        B.spa_kv_append_paged(P.h, k, k, i64([20, -3]), 2, T, P.dtable, P.pages)
        with pytest.raises(B.SpaError) as e:
            B.spa_paged_status(P.h)
        assert e.value.status == B.SPA_ERR_DEVICE_RANGE and "position" in str(e.value)
        B.spa_paged_status(P.h)   # cleared
        P.append_model(f64(k)[:, :, :12], f64(k)[:, :, :12], [20, 40], [12, 0])
        P.append_model(f64(k)[:, :, 3:], f64(k)[:, :, 3:], [40, 0], [0, T - 3])
        assert np.array_equal(P.pages.cpu().numpy(), P.pool.data)
        # a block table entry outside the pool, and a count above T
        P.pages.copy_(before)
        t = P.dtable.clone()
        t[0, 1], t[1, 0] = P.n_pages, -1
        B.spa_kv_append_paged(P.h, k, k, i64([0, 0]), 2, T, t, P.pages, n_new=i64([T + 1, -1]))
        with pytest.raises(B.SpaError) as e:
            B.spa_paged_status(P.h)
        assert "block_table" in str(e.value) and "length" in str(e.value)
        kr = torch.full((2, 2, T, 128), 3.0, device="cuda", dtype=torch.bfloat16)
        vr = kr.clone()
        B.spa_kv_read_paged(P.h, P.pages, t, i64([0, 0]), 2, T, kr, vr)
        with pytest.raises(B.SpaError):
            B.spa_paged_status(P.h)
        assert (kr[0, :, 16:] == 3).all() and (kr[1, :, :16] == 3).all() and not (kr[0, :, :16] == 3).all()


# ------------------------------------------------------------------------------------------------ attention
def fill_rows(P, lens, seed=3, scale=1.0):
    """Appends Gaussian rows [0, lens[b]) to the model's pool and copies it to the device."""
    rng = np.random.default_rng(seed)
    for b, L in enumerate(lens):
        for g in range(P.Hkv):
            for t in range(L):
                k, v = scale * rng.standard_normal((2, M.D))
                P.pool.put(P.table, b, g, t, k, v)
    P.pages.copy_(torch.from_numpy(P.pool.data))


def check_attend(P, q, lens, out, lse=None, mask=None, n_sink=0, window=0, lists=None):
    G = P.Hq // P.Hkv
    got, q64 = f64(out), f64(q)
    for b, L in enumerate(lens):
        qr = P.q_model(q64[b], L)
        for g in range(P.Hkv):
            ret = mask is None or bool(mask[g])
            rows = M.attended(L, ret, None if lists is None else lists.get((b, g), []), n_sink, window, mask is not None)
            k, v = P.pool.rows(P.table, b, g, rows)
            want, wl, bound = M.attend(qr[g * G:(g + 1) * G], k, v)
            err = np.abs(got[b, g * G:(g + 1) * G] - want)
            assert (err <= bound + 1e-30).all(), (b, g, L, float((err / (bound + 1e-30)).max()))
            if lse is not None:
                gl = f64(lse)[b, g * G:(g + 1) * G]
                if L == 0 or not rows:
                    assert np.isneginf(gl).all()
                else:
                    off = (np.abs(qr[g * G:(g + 1) * G]) @ np.abs(k).T).max() / math.sqrt(M.D) * 2.0 ** -16 + 2e-5
                    assert (np.abs(gl - wl) <= off * 1.45).all()


ATTEND_CASES = [
    # fmt, dtype, G, Hkv, page, lens, rope
    ("int4", "bf16", 1, 1, 16, [1], ("half", "plain")),
    ("int4", "bf16", 4, 2, 16, [0, 15, 16, 17, 300], ("half", "plain")),
    ("int4", "bf16", 8, 1, 48, [431, 0, 1], ("half", "bands")),
    ("int4", "f32", 3, 2, 64, [200, 77], ("interleaved", "ramp")),
    ("int4", "f32", 5, 1, 128, [129], None),
    ("int4", "bf16", 7, 1, 32, [260], ("interleaved", "plain")),
    ("int4", "bf16", 2, 64, 16, [33, 2], ("half", "plain")),
    ("bf16", "bf16", 1, 3, 16, [1, 0, 100], ("half", "plain")),
    ("bf16", "bf16", 4, 2, 32, [0, 15, 16, 17, 300], ("half", "bands")),
    ("bf16", "bf16", 8, 1, 48, [431, 90], ("interleaved", "plain")),
    ("bf16", "f32", 6, 2, 64, [200, 77], None),
]


@pytest.mark.parametrize("case", ATTEND_CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
@pytest.mark.parametrize("kind", ["all", "stream", "mixed", "lists"])
def test_attend_matches_the_definition(case, kind):
    fmt, dtype, G, Hkv, page, lens, rope = case
    Bs = len(lens)
    r = Rope(128, *rope) if rope else None
    with Paged(Bsz=Bs, Hq=G * Hkv, Hkv=Hkv, fmt=fmt, page=page, max_pages=max(1, -(-max(lens) // page)), dtype=dtype,
               rope=r, fill=0xff) as P:     # unwritten rows hold NaN scales or values
        fill_rows(P, lens)
        q = torch.randn(Bs, G * Hkv, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).mul_(2).to(TDT[dtype])
        out = torch.full((Bs, G * Hkv, 128), float("nan"), device="cuda")
        lse = torch.full((Bs, G * Hkv), float("nan"), device="cuda")
        kw = {}
        lists = None
        if kind != "all":
            mask = [0] * Hkv if kind == "stream" else [int(g % 2 == 0) for g in range(Hkv)]
            kw = dict(mask=mask, n_sink=3, window=37)
        if kind == "lists":
            rng = np.random.default_rng(1)
            stride = max(lens) + 5
            sel = torch.full((Bs, Hkv, stride), 1 << 30, dtype=torch.int32, device="cuda")
            cnt = torch.zeros(Bs * Hkv, dtype=torch.int32, device="cuda")
            lists = {}
            for b, L in enumerate(lens):
                for g in range(Hkv):
                    cand = np.arange(min(3, L), max(min(3, L), L - 37))
                    rows = np.sort(rng.choice(cand, size=rng.integers(0, len(cand) + 1), replace=False)) if len(cand) else cand
                    if kw["mask"][g]:
                        lists[(b, g)] = rows
                    sel[b, g, :len(rows)] = torch.from_numpy(rows.astype(np.int32)).cuda()
                    cnt[b * Hkv + g] = len(rows)
            kw["lists"] = lists
            B.spa_attend_paged(P.h, q, P.pages, P.dtable, i64(lens), Bs, 0, out, head_mask=kw["mask"], n_sink=3,
                               window=37, sel_idx=sel, sel_count=cnt, sel_stride=stride, lse=lse)
        else:
            B.spa_attend_paged(P.h, q, P.pages, P.dtable, i64(lens), Bs, max(1, max(lens)), out,
                               head_mask=kw.get("mask"), n_sink=kw.get("n_sink", 0), window=kw.get("window", 0), lse=lse)
        B.spa_paged_status(P.h)
        check_attend(P, q, lens, out, lse, **kw)
    if r:
        B.spa_rope_destroy(r.h)


@pytest.mark.parametrize("n_sink,window", [(0, 1), (1, 0), (16, 16), (5, 1000), (0, 17), (40, 3)])
@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_attend_sinks_and_window_edges(fmt, n_sink, window):
    lens = [1, 16, 18, 50, 64, 0]
    with Paged(Bsz=6, Hq=8, Hkv=2, fmt=fmt, page=32, max_pages=2, fill=0xff) as P:
        fill_rows(P, lens)
        q = torch.randn(6, 8, 128, device="cuda", dtype=torch.bfloat16)
        out = torch.empty(6, 8, 128, device="cuda")
        B.spa_attend_paged(P.h, q, P.pages, P.dtable, i64(lens), 6, 0, out, head_mask=[0, 1], n_sink=n_sink, window=window)
        B.spa_paged_status(P.h)
        check_attend(P, q, lens, out, mask=[0, 1], n_sink=n_sink, window=window)


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_attend_bad_pages_lengths_and_lists_are_skipped_and_reported(fmt):
    L = 100
    with Paged(Bsz=1, Hq=4, Hkv=1, fmt=fmt, page=16, max_pages=7) as P:
        fill_rows(P, [L])
        q = torch.randn(1, 4, 128, device="cuda", dtype=torch.bfloat16)
        out = torch.empty(1, 4, 128, device="cuda")

        def reported(word, **kw):
            B.spa_attend_paged(P.h, q, P.pages, kw.pop("table", P.dtable), i64([kw.pop("L", L)]), 1, kw.pop("cap", 0), out, **kw)
            with pytest.raises(B.SpaError) as e:
                B.spa_paged_status(P.h)
            assert e.value.status == B.SPA_ERR_DEVICE_RANGE and word in str(e.value)

        def want(rows):
            k, v = P.pool.rows(P.table, 0, 0, rows)
            w, _, bound = M.attend(f64(q)[0], k, v)
            assert (np.abs(f64(out)[0] - w) <= bound).all()

        t = P.dtable.clone()
        t[0, 2], t[0, 5] = -1, P.n_pages + 7
        reported("block_table", table=t)
        want([p for p in range(L) if p // 16 not in (2, 5)])
        reported("length", L=200, cap=90)
        want(range(90))
        reported("length", L=-4)
        assert (out == 0).all()
        sel = torch.tensor([[[7, -1, 50, 100, 50]]], dtype=torch.int32, device="cuda")
        cnt = torch.tensor([5], dtype=torch.int32, device="cuda")
        reported("selected", head_mask=[1], n_sink=1, window=2, sel_idx=sel, sel_count=cnt, sel_stride=5)
        want([0, 98, 99, 7, 50, 50])
        cnt.fill_(6)
        reported("selected", head_mask=[1], n_sink=1, window=2, sel_idx=sel, sel_count=cnt, sel_stride=5)
        want([0, 98, 99])


def test_attend_shared_pages_and_repeats_give_the_same_bits():
    """Two sequences over one prefix's pages; the same call twice, and split differently in a larger batch, agree."""
    with Rope() as r, Paged(Bsz=2, Hq=8, Hkv=2, fmt="int4", page=16, max_pages=64, rope=r) as P:
        P.table[1] = P.table[0]
        P.dtable.copy_(torch.from_numpy(P.table))
        fill_rows(P, [1000])
        q = torch.randn(1, 8, 128, device="cuda", dtype=torch.bfloat16).expand(2, 8, 128).contiguous()
        outs = [torch.empty(2, 8, 128, device="cuda") for _ in range(3)]
        for o in outs:
            B.spa_attend_paged(P.h, q, P.pages, P.dtable, i64([1000, 1000]), 2, 0, o)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        check_attend(P, q, [1000, 1000], outs[0])


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_offsets_past_32_bits(fmt):
    """A pool over 4 GB: rows at its far end are written, read and attended there."""
    Hkv, page = 8, 256
    per_page = Hkv * page // 16 * M.block_bytes(fmt)
    n_pages = (1 << 32) // per_page + 8
    cfg = B.make_paged_config(max_batch=1, n_q_heads=Hkv, n_kv_heads=Hkv, kv_dtype=B.SPA_BF16, page_format=FMT[fmt],
                              page_size=page, n_pages=n_pages, max_pages=4)
    h = B.spa_paged_create(cfg)
    try:
        pages = torch.zeros(n_pages * per_page, dtype=torch.uint8, device="cuda")
        table = torch.tensor([[n_pages - 1, 0, n_pages - 3, n_pages - 2]], dtype=torch.int32, device="cuda")
        T = 600
        k, v = (torch.randn(1, Hkv, T, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        B.spa_kv_append_paged(h, k, v, i64([0]), 1, T, table, pages)
        kr, vr = torch.empty_like(k), torch.empty_like(v)
        B.spa_kv_read_paged(h, pages, table, i64([0]), 1, T, kr, vr)
        q = torch.randn(1, Hkv, 128, device="cuda", dtype=torch.bfloat16)
        out = torch.empty(1, Hkv, 128, device="cuda")
        B.spa_attend_paged(h, q, pages, table, i64([T]), 1, 0, out)
        B.spa_paged_status(h)
        assert pages[(1 << 32):].any()
        for g in range(Hkv):
            kk, vv = f64(kr)[0, g], f64(vr)[0, g]
            if fmt == "int4":
                kk, vv = (c_s(x, grp) for x, grp in ((f64(k)[0, g], M.GROUP_K), (f64(v)[0, g], M.GROUP_V)))
                assert np.array_equal(f64(kr)[0, g], M.rne_bf16(kk)) and np.array_equal(f64(vr)[0, g], M.rne_bf16(vv))
            else:
                assert torch.equal(kr, k) and torch.equal(vr, v)
            w, _, bound = M.attend(f64(q)[0, g:g + 1], kk, vv)
            assert (np.abs(f64(out)[0, g] - w[0]) <= bound[0]).all()
    finally:
        B.spa_paged_destroy(h)


def c_s(x, group):
    codes, s = M.quantise(x, group)
    return (codes.astype(np.float64) - 8) * s[..., group]
