"""Attention over pages where its number formats could give out: scores far from 1, values and queries whose
magnitudes differ from row to row, group to group and head to head, and the precision it documents.

The bound.  A score is sum_g s_g sum_{d in g} q_d (n_d + 8) - 8 sum_d q_d over the scale groups g.  Queries are kept to 22
bits (2^-22 relative), the tensor cores' sums of a group's 32 products are off by at most 2^-21 of the largest term for
each of two products, float32 adds 2^-22 for the four groups: together at most 2^-20 of sum_d |q_d| 8 s_g(d), in units
of the score.  Over bf16 pages 8 s is |k| (24 bits, eight products of 2^-21 in two chains: 2^-19 of sum |q k|).  A weight is then off by
twice the largest score's error, relative, its own 2^-22 and the exponential's; an item's sums by 2^-21, the sums over
the items by 2^-24 each: 2^-19 + items 2^-24 of sum p |v|."""
import math

import numpy as np
import pytest
import torch

import paged_model as M
from head_partitioned_sparse_b200 import binding as B
from test_gpu_paged import f64, i64
from test_gpu_paged_flow import Cache

pytestmark = pytest.mark.gpu

GK = torch.from_numpy(M.GROUP_K).long()


def attend(c, q, lse=None):
    out = torch.full((c.B, c.Hq, 128), float("nan"), device="cuda")
    B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, c.B, 0, out, lse=lse)
    B.spa_paged_status(c.h)
    return out


def scales_k(c, b, g, n):
    """Bounds 8 s of the stored keys' scales, by dim: of the codes' largest magnitude, 7 at most (and 4 at least, since the
    group's largest value is 7 steps long but for the scale's rounding)."""
    k = c.kr[b, g, :n].double().abs()
    top = torch.stack([k[:, GK.cuda() == i].amax(-1) for i in range(4)], -1)
    return (8 / 6 * top)[:, GK.cuda()]


def reference(c, q, fmt):
    """(want, bound, log2 denominators, their bound) of every head, float64 on the GPU; c without a rotation."""
    G = c.Hq // c.Hkv
    q64 = q.double()
    want, bound = torch.zeros(2, c.B, c.Hq, 128, device="cuda", dtype=torch.float64).unbind(0)
    lse, lb = torch.zeros(2, c.B, c.Hq, device="cuda", dtype=torch.float64).unbind(0)
    for b in range(c.B):
        L = c.lens[b]
        for g in range(c.Hkv):
            k, v = c.kr[b, g, :L].double(), c.vr[b, g, :L].double()
            qq = q64[b, g * G:(g + 1) * G]
            s = qq @ k.T / math.sqrt(128)
            if fmt == "int4":
                off = (qq.abs() @ scales_k(c, b, g, L).T / math.sqrt(128)).amax(-1) * 2.0 ** -20
            else:
                off = (qq.abs() @ k.abs().T / math.sqrt(128)).amax(-1) * 2.0 ** -19
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m)
            z = p.sum(-1, keepdim=True)
            h = slice(g * G, (g + 1) * G)
            want[b, h] = p @ v / z
            bound[b, h] = (2 * off[:, None] + 2.0 ** -19 + -(-L // 16) * 2.0 ** -24) * (p @ v.abs() / z)
            lse[b, h] = ((m + z.log()) / math.log(2.0))[:, 0]
            # the maximum and the sum in float32, and the score's own error
            lb[b, h] = 1.45 * 2 * off + 2.0 ** -22 * lse[b, h].abs() + 2.0 ** -18
    return want, bound, lse, lb


def check(c, q, fmt, dims=slice(None)):
    lse = torch.full((c.B, c.Hq), float("nan"), device="cuda")
    out = attend(c, q, lse)
    want, bound, wl, lb = reference(c, q, fmt)
    err = (out.double() - want).abs()
    ok = err <= bound
    assert ok[..., dims].all(), float((err / bound)[..., dims].nan_to_num(1e9).max())
    assert ((lse.double() - wl).abs() <= lb).all()
    return out, want


# ------------------------------------------------------------------------------------------------ scores
def signs(seed):
    return torch.randint(0, 2, (128,), generator=torch.Generator().manual_seed(seed)).float().mul(2).sub(1).cuda()


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(fmt, sign):
    """Equal keys, so equal weights, whatever the score: its log2 is sign * 2^e for e from 10 to 100 in steps of 1 / 3.  Values whose
    largest scale is a power of two (7 2^n) and others."""
    mags = 2.0 ** (np.arange(10, 100, 1 / 3) / 2) / math.sqrt(128 / math.sqrt(128) * math.log2(math.e))
    n, L, G = len(mags), 40, 4
    k = torch.zeros(n, 1, L, 128, device="cuda")
    q = torch.zeros(n, G, 128, device="cuda")
    for i, a in enumerate(mags):
        k[i, 0] = sign * float(a) * signs(i)
        q[i] = float(a) * signs(i)
    g = torch.Generator(device="cuda").manual_seed(1)
    v = torch.randint(-7, 8, (n, 1, L, 128), generator=g, device="cuda").float()
    v[..., :8] = 7
    v[1::2] *= 1.37
    with Cache([L] * n, G, 1, fmt, 16, "f32", k=k, v=v) as c:
        out = attend(c, q)
        want = c.vr.double().mean(2)
        bound = (2.0 ** -19 + 2.0 ** -20) * c.vr.double().abs().mean(2)
        assert torch.isfinite(out).all()
        assert ((out.double() - want).abs() <= bound).all()
        check(c, q, fmt)


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_rows_far_below_each_other(fmt):
    """One row takes all the weight: at the front, at the end, alone in its sequence; scores down to -1e37."""
    L, G = 70, 2
    e = torch.tensor([1e4, 1e9, 1e14, 3e16, 1e18], device="cuda")
    n = len(e)
    for at in (0, 35, L - 1, None):
        k = -(e * torch.ones(1, device="cuda"))[:, None, None, None] * signs(3).expand(n, 1, L, 128)
        v = torch.randn(n, 1, L, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
        q = (e[:, None, None] * signs(3).expand(n, G, 128)).contiguous()
        lens = [1] * n
        if at is not None:
            lens = [L] * n
            k[:, :, at] *= 0.5
        with Cache(lens, G, 1, fmt, 16, "f32", k=k.contiguous(), v=v) as c:
            out = attend(c, q)
            row = c.vr[:, :, at or 0]
            assert ((out - row).abs() <= 2.0 ** -19 * row.abs()).all()


# ------------------------------------------------------------------------------------------------ values
def unit_cache(seed, n, Hkv, L, fmt, lens=None, change=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(n, Hkv, L, 128, generator=g, device="cuda")
    v = torch.randn(n, Hkv, L, 128, generator=g, device="cuda")
    q = 1.5 * torch.randn(n, Hkv * 4, 128, generator=g, device="cuda")
    if change:
        change(q, k, v)
    return q, Cache(lens or [L] * n, 4 * Hkv, Hkv, fmt, 16, "f32", k=k, v=v)


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
@pytest.mark.parametrize("gap", [0, 12, 30, 90])
@pytest.mark.parametrize("at", [0, 57, 899])
def test_one_row_of_larger_values(fmt, gap, at):
    """A row whose values are 2^k times the others', its score about `gap` below them: it has no weight, all of it, or some."""
    ks = [0, 8, 12, 14, 18, 20, 22, 26, 30, 45, 60, 90]

    def change(q, k, v):
        q[:] = q[:, :1]     # one direction, so that the row is low for every head
        for i, e in enumerate(ks):
            v[i, :, at] *= 2.0 ** e
            u = q[i, 0] / q[i, 0].norm()
            k[i, 0, at] = -u * gap * math.sqrt(128) / float(q[i, 0].norm())
    q, c = unit_cache(5, len(ks), 1, 900, fmt, change=change)
    with c:
        check(c, q, fmt)


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
@pytest.mark.parametrize("e", [12, 20, 30, 70, -30, -70])
def test_one_group_of_larger_values(fmt, e):
    """One channel 2^e times the rest: the groups of dims have their own scales, and keep their own precision."""
    def change(q, k, v):
        v[0, :, :, 37] *= 2.0 ** e
        v[1] *= 2.0 ** e
        v[1, :, ::2] = v[1, :, ::2] * 2.0 ** -e
        v[2, :, :500] *= 2.0 ** e
    q, c = unit_cache(6, 3, 2, 1000, fmt, change=change)
    with c:
        check(c, q, fmt)


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_values_that_grow_as_their_weights_fall(fmt):
    """Weights and values that make up for each other: every row counts alike."""
    def change(q, k, v):
        q[:] = q[:, :1]
        for i in range(2):
            u = q[i, 0] / q[i, 0].norm()
            x = torch.linspace(0, 60, 800, device="cuda")
            k[i, 0] = -u * x[:, None] * math.sqrt(128) * math.log(2) / q[i, 0].norm()
            v[i, 0] *= torch.exp2(x)[:, None]
        k[1], v[1] = k[1].flip(1), v[1].flip(1)
    q, c = unit_cache(7, 2, 1, 800, fmt, change=change)
    with c:
        check(c, q, fmt)


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_values_near_the_end_of_float32(fmt):
    """Values up to 2^123 with groups and rows of zeros beside them; the sum of a row's weights times its values stays
    within float32."""
    def change(q, k, v):
        v[0, :, :, 32:] = 0
        v[0, :, 3:] = 0
        v *= 2.0 ** 121 / v.abs().amax()
    q, c = unit_cache(8, 2, 1, 20, fmt, change=change)
    with c:
        out, _ = check(c, q, fmt)
        assert torch.isfinite(out).all()


# ------------------------------------------------------------------------------------------------ queries
@pytest.mark.parametrize("fmt", ["int4", "bf16"])
@pytest.mark.parametrize("e", [10, 16, 24, 40, 60])
def test_queries_and_keys_of_unequal_groups(fmt, e):
    """Queries 2^e times larger in one scale group, keys as much smaller there: every group counts alike.  Heads with the large group in
    different places."""
    def change(q, k, v):
        k *= 0.5
        grp = GK.cuda()
        for h in range(4):
            q[0, h, grp == 2] *= 2.0 ** e
            q[1, h, grp == h] *= 2.0 ** e
        k[0, :, :, grp == 2] *= 2.0 ** -e
        k[1, :, :, grp == 0] *= 2.0 ** -e
        q[1, 1:] *= 2.0 ** -e     # one head sees its large group small, the others theirs at full size
    q, c = unit_cache(9, 2, 1, 600, fmt, change=change)
    with c:
        check(c, q, fmt)


# ------------------------------------------------------------------------------------------------ precision
@pytest.mark.parametrize("fmt", ["int4", "bf16"])
@pytest.mark.parametrize("L,Hkv,G", [(257, 8, 4), (5000, 2, 8), (400000, 1, 4)])
def test_precision_in_the_norm(fmt, L, Hkv, G):
    """Gaussian rows: the 2-norm of the error over that of the result.  A score's error is a sum of 128 independent roundings
    of 2^-22 / sqrt(3) of terms of size 1.5 / sqrt(128), 2e-7 to 3e-7 with the tensor cores' own, and so is a weight's, relative; a
    probability's own rounding and an item's sums add 2^-22 each.  Rows' errors are independent as the values are, so
    the result's relative error is a row's: 5e-7, and 1e-6 with room.  (Operands of 16 bits and residuals of 8 would give 4e-6, sums left in
    the tensor cores' accumulators 4e-6 at the longest.)"""
    g = torch.Generator(device="cuda").manual_seed(L)
    k, v = torch.randn(2, 1, Hkv, L, 128, generator=g, device="cuda").unbind(0)
    with Cache([L], Hkv * G, Hkv, fmt, 64, "f32", k=k, v=v) as c:
        q = 1.5 * torch.randn(1, Hkv * G, 128, generator=g, device="cuda")
        out, want = check(c, q, fmt)
        assert float((out.double() - want).norm() / want.norm()) <= 1e-6


def test_the_way_a_sequence_is_shared_out_changes_roundings_only():
    """One sequence alone, and among others of a batch (its rows then split over other CTAs, its pages shared): equal to the
    sums' roundings."""
    L, Hkv = 6000, 2
    g = torch.Generator(device="cuda").manual_seed(12)
    k, v = torch.randn(2, 1, Hkv, L, 128, generator=g, device="cuda").unbind(0)
    with Cache([L], 8, Hkv, "int4", 16, "f32", k=k, v=v) as c:
        q = 1.5 * torch.randn(1, 8, 128, generator=g, device="cuda")
        want, bound, _, _ = reference(c, q, "int4")
        one = attend(c, q)
        n = 100
        cfg = B.make_paged_config(max_batch=n, n_q_heads=8, n_kv_heads=Hkv, kv_dtype=B.SPA_F32, page_format=B.SPA_PAGE_INT4,
                                  page_size=16, n_pages=c.pages.numel() // (Hkv * 2304), max_pages=c.table.shape[1])
        h = B.spa_paged_create(cfg)
        table = c.table.expand(n, -1).contiguous()
        lens = i64([L if b % 3 == 0 else b for b in range(n)])
        many = torch.empty(n, 8, 128, device="cuda")
        B.spa_attend_paged(h, q.expand(n, -1, -1).contiguous(), c.pages, table, lens, n, 0, many)
        B.spa_paged_status(h)
        B.spa_paged_destroy(h)
        same = many[0::3]
        assert ((same.double() - want).abs() <= bound).all()
        rel = float((same - one).double().norm() / (one.double().norm() * math.sqrt(len(same))))
        assert rel <= 2e-6      # twice the precision of one


# ------------------------------------------------------------------------------------------------ the way through float32
FAR = [
    # lens, Hq, Hkv, page, heads that see every row (None: all), with lists
    ([700, 650], 8, 2, 16, None, False),                   # a CTA a slice
    ([9000], 4, 1, 64, None, False),                       # one slice over many CTAs
    ([5000, 12000, 1], 24, 8, 48, None, False),            # aligned to slices
    ([2000] * 20, 16, 8, 128, None, False),                # 160 slices: equal shares, straddling
    ([40, 1500, 0, 17] * 10, 21, 7, 32, None, False),      # 280 slices of very unequal lengths
    ([6000, 2500, 0], 16, 4, 16, [1, 0, 0, 1], False),     # sinks and window beside them
    ([6000, 2500, 90], 16, 4, 32, [1, 0, 1, 1], True),     # lists
]


@pytest.mark.parametrize("case", FAR, ids=lambda c: "%dx%d-%d%s" % (len(c[0]), c[2], max(c[0]), "-lists" if c[5] else "-mask" if c[4] else ""))
@pytest.mark.parametrize("which", ["rows", "head", "query"])
def test_far_apart_in_every_share(case, which):
    """Values or queries that 4 bits take in float32, in every slice or in one, for each way of sharing the work out."""
    lens, Hq, Hkv, page, mask, listed = case
    Bs, T, n_sink, window = len(lens), max(lens), 3, 500
    g = torch.Generator(device="cuda").manual_seed(31)
    k, v = torch.randn(2, Bs, Hkv, T, 128, generator=g, device="cuda").unbind(0)
    if which == "rows":
        v[:, :, 5::37] *= 2.0 ** 20
        k[:, :, 5::37] *= 0.1
    if which == "head":
        v[0, Hkv - 1, :, 40:44] *= 2.0 ** -30
    with Cache(lens, Hq, Hkv, "int4", page, "f32", k=k, v=v) as c:
        q = 1.5 * torch.randn(Bs, Hq, 128, generator=g, device="cuda")
        if which == "query":
            q[0, 0, GK.cuda() == 1] *= 2.0 ** -20
        kw, lists = {}, None
        if mask:
            kw = dict(head_mask=mask, n_sink=n_sink, window=window)
        if listed:
            lists, sel, cnt = {}, torch.full((Bs, Hkv, T), -1, dtype=torch.int32, device="cuda"), torch.zeros(Bs * Hkv, dtype=torch.int32, device="cuda")
            for b, L in enumerate(lens):
                for h in range(Hkv):
                    lo, hi = min(n_sink, L), max(min(n_sink, L), L - window)
                    lists[b, h] = lo + torch.randperm(hi - lo, generator=g, device="cuda")[:(hi - lo) // 3].sort().values
                    sel[b, h, :len(lists[b, h])] = lists[b, h].to(torch.int32)
                    cnt[b * Hkv + h] = len(lists[b, h])
            kw.update(sel_idx=sel, sel_count=cnt, sel_stride=T)
        outs = [torch.full((Bs, Hq, 128), float("nan"), device="cuda") for _ in range(2)]
        lse = torch.full((Bs, Hq), float("nan"), device="cuda")
        for out in outs:
            B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, Bs, 0, out, lse=lse, **kw)
        B.spa_paged_status(c.h)
        assert torch.equal(*outs)
        c.check(q, outs[0], lse, mask=mask, n_sink=n_sink if mask else 0, window=window if mask else 0, lists=lists)


def test_far_apart_rows_and_bad_pages():
    """Block table entries and listed positions out of range are skipped there, too, and NaN stays in its scale group."""
    L = 300
    g = torch.Generator(device="cuda").manual_seed(32)
    k, v = torch.randn(2, 1, 1, L, 128, generator=g, device="cuda").unbind(0)
    v[0, 0, ::7] *= 2.0 ** 25
    with Cache([L], 4, 1, "int4", 16, "f32", k=k, v=v) as c:
        q = 1.5 * torch.randn(1, 4, 128, generator=g, device="cuda")
        t = c.table.clone()
        t[0, 2], t[0, 9] = -1, 1 << 30
        out = torch.empty(1, 4, 128, device="cuda")
        B.spa_attend_paged(c.h, q, c.pages, t, c.n, 1, 0, out)
        with pytest.raises(B.SpaError):
            B.spa_paged_status(c.h)
        rows = torch.tensor([p for p in range(L) if p // 16 not in (2, 9)], device="cuda")
        c.check(q, out, mask=[1], lists={(0, 0): rows})
        sel = torch.tensor([[[7, -1, 50, 300, 50, 7 * 16]]], dtype=torch.int32, device="cuda")
        cnt = torch.tensor([6], dtype=torch.int32, device="cuda")
        B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, 1, 0, out, head_mask=[1], n_sink=1, window=2, sel_idx=sel, sel_count=cnt, sel_stride=6)
        with pytest.raises(B.SpaError):
            B.spa_paged_status(c.h)
        c.check(q, out, mask=[1], n_sink=1, window=2, lists={(0, 0): torch.tensor([7, 50, 50, 112], device="cuda")})
    v[0, 0, 77, 4] = float("nan")
    with Cache([L], 4, 1, "int4", 16, "f32", k=k, v=v) as c:
        out = attend(c, q)
        bad = torch.from_numpy(M.GROUP_V == M.GROUP_V[4]).cuda()
        assert torch.isnan(out[..., bad]).all() and torch.isfinite(out[..., ~bad]).all()
