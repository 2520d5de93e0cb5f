"""Calls of the rotary and paged-cache operators at the ends of what they accept."""
import numpy as np
import pytest
import torch

import paged_model as M
from head_partitioned_sparse_b200 import binding as B
from test_gpu_paged import Paged, Rope, f64, i64
from test_gpu_paged_flow import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
@pytest.mark.parametrize("Bs,Hkv", [(1, 1), (7, 4), (60, 5)])
def test_attend_without_a_row(fmt, Bs, Hkv):
    """Every sequence empty: zeros, and no weight; with lists and a mask, too."""
    with Paged(Bsz=Bs, Hq=2 * Hkv, Hkv=Hkv, fmt=fmt, page=16, max_pages=1, fill=0xff) as P:
        q = torch.full((Bs, 2 * Hkv, 128), float("nan"), device="cuda", dtype=torch.bfloat16)
        sel = torch.zeros(Bs, Hkv, 4, dtype=torch.int32, device="cuda")
        cnt = torch.zeros(Bs * Hkv, dtype=torch.int32, device="cuda")
        for kw in ({}, dict(head_mask=[1] * Hkv, n_sink=1, window=2), dict(head_mask=[1] * Hkv, n_sink=1, window=2, sel_idx=sel, sel_count=cnt, sel_stride=4)):
            out = torch.full((Bs, 2 * Hkv, 128), 7.0, device="cuda")
            lse = torch.full((Bs, 2 * Hkv), 7.0, device="cuda")
            B.spa_attend_paged(P.h, q, P.pages, P.dtable, i64([0] * Bs), Bs, 0, out, lse=lse, **kw)
            B.spa_paged_status(P.h)
            assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("start", [(1 << 63) - 1, (1 << 63) - 3, -(1 << 63), (1 << 32) - 1, -1])
def test_start_positions_of_any_size(start):
    """Positions past either end of 64 bits, or of 32, write and read nothing."""
    T = 6
    k = torch.randn(1, 2, T, 128, device="cuda", dtype=torch.bfloat16)
    with Rope() as r, Paged(Bsz=1, Hq=2, Hkv=2, fmt="int4", page=16, max_pages=1, rope=r) as P:
        before = P.pages.clone()
        first = max(0, -start) if start > -T else T      # rows from 0 on
        B.spa_kv_append_paged(P.h, k, k, i64([start]), 1, T, P.dtable, P.pages)
        with pytest.raises(B.SpaError):
            B.spa_paged_status(P.h)
        if start == -1:
            P.append_model(f64(k)[:, :, first:], f64(k)[:, :, first:], [0], [T - first])
        assert np.array_equal(P.pages.cpu().numpy(), P.pool.data)
        kr, vr = torch.full((2, 1, 2, T, 128), 3.0, device="cuda", dtype=torch.bfloat16).unbind(0)
        B.spa_kv_read_paged(P.h, before, P.dtable, i64([start]), 1, T, kr, vr)
        with pytest.raises(B.SpaError):
            B.spa_paged_status(P.h)
        assert (kr[:, :, :first if start == -1 else T] == 3).all()


def test_the_largest_sequence_and_page():
    """2^24 tokens in pages of 65536: the last rows appended, read back and attended through the window."""
    n, page = 1 << 24, 65536
    mp = n // page
    with Rope() as r, Paged(Bsz=1, Hq=4, Hkv=1, fmt="int4", page=page, max_pages=1, spare=1, rope=r) as P:
        cfg = B.make_paged_config(max_batch=1, n_q_heads=4, n_kv_heads=1, kv_dtype=B.SPA_BF16, page_format=B.SPA_PAGE_INT4,
                                  page_size=page, n_pages=2, max_pages=mp)
        h = B.spa_paged_create(cfg, r.h)
        table = torch.full((1, mp), -1, dtype=torch.int32, device="cuda")
        table[0, -1] = 1
        T = 40
        k, v = torch.randn(2, 1, 1, T, 128, device="cuda").bfloat16().unbind(0)
        B.spa_kv_append_paged(h, k, v, i64([n - T]), 1, T, table, P.pages)
        q = torch.randn(1, 4, 128, device="cuda").bfloat16()
        out = torch.empty(1, 4, 128, device="cuda")
        B.spa_attend_paged(h, q, P.pages, table, i64([n]), 1, 0, out, head_mask=[0], n_sink=0, window=T)
        B.spa_paged_status(h)
        P.table = np.array([[0] * (mp - 1) + [1]], np.int32)
        P.pool.data[:] = P.pages.cpu().numpy()
        kk, vv = P.pool.rows(P.table, 0, 0, range(n - T, n))
        codes, s = M.quantise(M.rotate(f64(k)[0, 0], np.arange(n - T, n, dtype=np.float64), **r.model), M.GROUP_K)
        assert np.array_equal(kk, (codes.astype(np.float64) - 8) * s[..., M.GROUP_K])
        want, _, bound = M.attend(M.rotate(f64(q)[0], float(n - 1), **r.model), kk, vv)
        assert (np.abs(f64(out)[0] - want) <= bound).all()
        B.spa_paged_destroy(h)


def test_rope_far_positions_and_gradient_of_a_shared_head():
    """Positions to 2^50, and the gradient of a key head that several heads read: the transposed map of each, summed."""
    H, T, d = 4, 3, 64
    pos = torch.tensor([[1 << 50, -(1 << 50), (1 << 40) + 12345]], device="cuda")
    with Rope(64, "half", "plain", theta=10000.0) as r:
        x = torch.randn(1, H, T, d, device="cuda")
        y, z = torch.empty_like(x), torch.empty_like(x)
        B.spa_rope_apply(r.h, x, y, 1, T, H, d, B.SPA_F32, positions=pos)
        B.spa_rope_apply(r.h, y, z, 1, T, H, d, B.SPA_F32, positions=pos, transpose=True)
        # angles of 2^50 to 2^-52 of them are known to 0.25 only, but both calls take the same: R^T R = 1
        assert (z - x).abs().max() <= 4 * 4e-7 * float(x.abs().max())
        near = torch.tensor([[5, 70000, 1 << 24]], device="cuda")
        k, gy = torch.randn(T, d, device="cuda"), torch.randn(1, H, T, d, device="cuda")
        g = torch.empty_like(gy)
        B.spa_rope_apply(r.h, gy, g, 1, T, H, d, B.SPA_F32, positions=near, transpose=True)
        out = torch.empty_like(gy)
        B.spa_rope_apply(r.h, k, out, 1, T, H, d, B.SPA_F32, positions=near, x_strides=(0, d, 0))
        lhs, rhs = float((out.double() * gy.double()).sum()), float((g.double().sum(1)[0] * k.double()).sum())
        assert abs(lhs - rhs) <= 8e-7 * float((gy.double().abs().sum(1)[0] * k.double().abs().amax(-1, keepdim=True)).sum())


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_calls_of_one_handle_on_two_streams(fmt):
    """Appends and reads of one handle may run beside its attention."""
    with Cache([5000, 3000], 8, 2, fmt, 32, "bf16", handles=1) as c:
        g = torch.Generator(device="cuda").manual_seed(5)
        q = torch.randn(2, 8, 128, generator=g, device="cuda").bfloat16()
        want = torch.empty(2, 8, 128, device="cuda")
        B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, 2, 0, want)
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        k, v = torch.empty(2, 2, 2, 5000, 128, device="cuda", dtype=torch.bfloat16).unbind(0)
        outs = torch.empty(20, 2, 8, 128, device="cuda")
        bad = c.table.clone()
        bad[1, 0] = -1
        torch.cuda.synchronize()
        for i in range(20):
            B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, 2, 0, outs[i], stream=a)
            B.spa_kv_read_paged(c.h, c.pages, bad if i == 13 else c.table, c.zero, 2, 5000, k, v, n_rows=c.n, stream=b)
        torch.cuda.synchronize()
        assert (outs == want).all()
        with pytest.raises(B.SpaError) as e:
            B.spa_paged_status(c.h, stream=a)
        assert "block_table" in str(e.value)
        B.spa_paged_status(c.h, stream=b)
        assert torch.equal(k[0].float(), c.kr[0].bfloat16().float())
