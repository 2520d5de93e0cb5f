"""The rotary and paged-cache operators together and at size: a decode step through selection and pages, a
prefix read back for prefill, captured graphs, two streams, every way of sharing slices out, and extreme values.

References are float64 on the GPU over rows read back in float32 (exact for both formats; the append and the read are
checked byte by byte in test_gpu_paged.py)."""
import math

import numpy as np
import pytest
import torch

import paged_model as M
from head_partitioned_sparse_b200 import binding as B
from test_gpu_paged import FMT, KDT, TDT, Rope, f64, i64, rope_bound

pytestmark = pytest.mark.gpu


class Cache:
    """A paged cache filled by the append, with its rows in float64."""

    def __init__(self, lens, Hq, Hkv, fmt, page, dtype="f32", rope=None, k=None, v=None, seed=0, handles=1):
        self.B, self.Hq, self.Hkv, self.lens = len(lens), Hq, Hkv, list(lens)
        mp = max(1, -(-max(lens) // page))
        n_pages = self.B * mp + 1
        cfg = B.make_paged_config(max_batch=self.B, n_q_heads=Hq, n_kv_heads=Hkv, kv_dtype=KDT[dtype],
                                  page_format=FMT[fmt], page_size=page, n_pages=n_pages, max_pages=mp)
        self.rope, self.dtype = rope, dtype
        self.handles = [B.spa_paged_create(cfg, rope.h if rope else None) for _ in range(handles)]
        self.h = self.handles[0]
        g = torch.Generator(device="cuda").manual_seed(seed)
        perm = torch.randperm(n_pages, generator=g, device="cuda")[:self.B * mp]
        self.table = perm.view(self.B, mp).to(torch.int32)
        self.pages = torch.full((n_pages * B.spa_paged_page_bytes(cfg),), 0xff, dtype=torch.uint8, device="cuda")
        T = max(1, max(lens))
        shape = (self.B, Hkv, T, 128)
        self.k = (torch.randn(shape, generator=g, device="cuda") if k is None else k).to(TDT[dtype])
        self.v = (torch.randn(shape, generator=g, device="cuda") if v is None else v).to(TDT[dtype])
        self.n = i64(lens)
        self.zero = i64([0] * self.B)
        B.spa_kv_append_paged(self.h, self.k, self.v, self.zero, self.B, T, self.table, self.pages, n_new=self.n)
        # rows as stored, in float32
        cfg.kv_dtype = B.SPA_F32
        h32 = B.spa_paged_create(cfg, None)
        self.kr, self.vr = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
        B.spa_kv_read_paged(h32, self.pages, self.table, self.zero, self.B, T, self.kr, self.vr, n_rows=self.n)
        B.spa_paged_status(h32)
        B.spa_paged_destroy(h32)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        for h in self.handles:
            B.spa_paged_destroy(h)

    def rotated(self, q):
        x = f64(q)
        if self.rope:
            pos = np.maximum(np.array(self.lens, np.float64) - 1, 0)
            x = M.rotate(x, pos[:, None], **self.rope.model)
        return torch.from_numpy(x).cuda()

    def check(self, q, out, lse=None, mask=None, n_sink=0, window=0, lists=None, slices=None):
        """Every head (or those of `slices`) against float64, within the bound of paged_model.attend."""
        G = self.Hq // self.Hkv
        qr = self.rotated(q)
        for b, g in (slices or [(b, g) for b in range(self.B) for g in range(self.Hkv)]):
            L = self.lens[b]
            ret = mask is None or bool(mask[g])
            if mask is None or (ret and lists is None):
                rows = torch.arange(L, device="cuda")
            else:
                n_s = min(n_sink, L)
                rows = torch.cat((torch.arange(n_s, device="cuda"), torch.arange(max(n_s, L - window), L, device="cuda")))
                if ret:
                    rows = torch.cat((rows, lists[b, g]))
            got = out[b, g * G:(g + 1) * G].double()
            if len(rows) == 0:
                assert (got == 0).all()
                continue
            k, v = self.kr[b, g, rows].double(), self.vr[b, g, rows].double()
            qq = qr[b, g * G:(g + 1) * G]
            s = qq @ k.T / math.sqrt(128)
            off = (qq.abs() @ k.abs().T / math.sqrt(128)).amax(-1) * 2.0 ** -17
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m)
            z = p.sum(-1, keepdim=True)
            want, bound = p @ v / z, (2 * off[:, None] + 2.0 ** -15) * (p @ v.abs() / z)
            err = (got - want).abs()
            assert (err <= bound).all(), (b, g, float((err / bound).max()))
            if lse is not None:
                wl = ((m + z.log()) / math.log(2.0))[:, 0]
                assert ((lse[b, g * G:(g + 1) * G].double() - wl).abs() <= 3 * off + 2e-5).all()


def queries(c, seed=1, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(c.B, c.Hq, 128, generator=g, device="cuda")).to(TDT[c.dtype])


SHARES = [
    # lens, Hq, Hkv, page: how the work is shared out
    ([700, 650], 8, 2, 16),                       # a CTA a slice
    ([9000], 4, 1, 64),                           # one slice over many CTAs
    ([5000, 20000, 1], 32, 8, 48),                # aligned to slices
    ([3000] * 20, 16, 8, 128),                    # 160 slices: equal shares, straddling
    ([40, 3000, 0, 17] * 10, 21, 7, 32),          # 280 slices of very unequal lengths
]


@pytest.mark.parametrize("case", SHARES, ids=lambda c: "%dx%d-%d" % (len(c[0]), c[2], max(c[0])))
@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_attend_shares(case, fmt):
    lens, Hq, Hkv, page = case
    with Rope(128, "half", "bands") as r, Cache(lens, Hq, Hkv, fmt, page, "bf16", r) as c:
        q = queries(c)
        out = torch.full((c.B, Hq, 128), float("nan"), device="cuda")
        lse = torch.full((c.B, Hq), float("nan"), device="cuda")
        B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, c.B, 0, out, lse=lse)
        B.spa_paged_status(c.h)
        c.check(q, out, lse)
        again = torch.empty_like(out)
        B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, c.B, 0, again)
        assert torch.equal(out, again)


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
@pytest.mark.parametrize("density", [0.02, 0.4, 1.0])
def test_attend_long_lists(fmt, density):
    lens, Hq, Hkv, n_sink, window = [30000, 12345, 4000], 16, 4, 4, 1000
    mask = [1, 0, 1, 1]
    with Cache(lens, Hq, Hkv, fmt, 64, "bf16") as c:
        g = torch.Generator(device="cuda").manual_seed(3)
        stride = max(lens)
        sel = torch.full((c.B, Hkv, stride), -7, dtype=torch.int32, device="cuda")
        cnt = torch.zeros(c.B * Hkv, dtype=torch.int32, device="cuda")
        lists = {}
        for b, L in enumerate(lens):
            for h in range(Hkv):
                n = int(density * (L - n_sink - window)) if mask[h] else 0
                rows = n_sink + torch.randperm(L - n_sink - window, generator=g, device="cuda")[:n].sort().values
                sel[b, h, :n] = rows.to(torch.int32)
                cnt[b * Hkv + h] = n
                lists[b, h] = rows
        q = queries(c)
        outs = [torch.empty(c.B, Hq, 128, device="cuda") for _ in range(2)]
        for o in outs:
            B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, c.B, 0, o, head_mask=mask, n_sink=n_sink, window=window,
                               sel_idx=sel, sel_count=cnt, sel_stride=stride)
        B.spa_paged_status(c.h)
        assert torch.equal(*outs)
        c.check(q, outs[0], mask=mask, n_sink=n_sink, window=window, lists=lists)


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_attend_as_many_slices_as_a_handle_takes(fmt):
    """4096 slices: the shallow ring."""
    rng = np.random.default_rng(0)
    lens = rng.choice([0, 1, 2, 15, 40], 64).tolist()
    with Cache(lens, 128, 64, fmt, 16, "bf16") as c:
        q = queries(c)
        out = torch.full((c.B, 128, 128), float("nan"), device="cuda")
        B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, c.B, 0, out)
        B.spa_paged_status(c.h)
        assert torch.isfinite(out).all()
        c.check(q, out, slices=[(int(b), int(g)) for b, g in zip(rng.integers(0, 64, 200), rng.integers(0, 64, 200))])


@pytest.mark.parametrize("G", [4, 8])
@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_attend_extreme_magnitudes(fmt, G):
    """Rows whose values grow and shrink by powers of two on the way (the running scale of the 4-bit values moves),
    queries and keys far from 1, zero rows, and a maximum that keeps rising."""
    L, Hkv = 3000, 1
    g = torch.Generator(device="cuda").manual_seed(8)
    k = torch.randn(3, Hkv, L, 128, generator=g, device="cuda")
    v = torch.randn(3, Hkv, L, 128, generator=g, device="cuda")
    j = torch.arange(L, device="cuda")
    v[0] *= torch.exp2((j % 61 - 30).float())[None, :, None]
    v[1] *= torch.exp2(-60 + j.float() / 25)[None, :, None]
    v[2, :, ::3] = 0
    k[2, :, ::5] = 0
    k[1] *= 1e3
    with Cache([L] * 3, G, Hkv, fmt, 32, "f32", k=k, v=v) as c:
        q = queries(c)
        q[1] *= 1e-3
        q[2, 0] = 0
        out = torch.empty(3, G, 128, device="cuda")
        B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, 3, 0, out)
        B.spa_paged_status(c.h)
        c.check(q, out)


def test_attend_int4_nan_stays_where_it_is():
    """A NaN among the values spoils its scale group's dims (of that KV head) only, one among the keys its KV head only."""
    L = 500
    k, v = torch.randn(2, 1, 2, L, 128, device="cuda").unbind(0)
    v[0, 0, 77, 4] = float("nan")
    k[0, 1, 33, 100] = float("nan")
    with Cache([L], 4, 2, "int4", 16, "f32", k=k, v=v) as c:
        q = queries(c)
        out = torch.empty(1, 4, 128, device="cuda")
        B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, 1, 0, out)
        bad = torch.from_numpy(M.GROUP_V == M.GROUP_V[4]).cuda()
        assert torch.isnan(out[0, :2][:, bad]).all() and torch.isfinite(out[0, :2][:, ~bad]).all()
        assert torch.isnan(out[0, 2:]).all()
        # the finite groups are right: the same without the NaN
        v2 = v.clone()
        v2[0, 0, 77, 4] = 0
        with Cache([L], 4, 2, "int4", 16, "f32", k=k, v=v2) as c2:
            o2 = torch.empty(1, 4, 128, device="cuda")
            B.spa_attend_paged(c2.h, q, c2.pages, c2.table, c2.n, 1, 0, o2)
            c2.check(q, o2, slices=[(0, 0)])
            assert (out[0, :2][:, ~bad] - o2[0, :2][:, ~bad]).abs().max() <= 1e-5


def test_decode_step_over_pages_matches_the_contiguous_one():
    """rotary -> k_cache and spa_decode, beside the paged append -> spa_select -> spa_attend_paged, on the same inputs."""
    Bs, Hq, Hkv, L, n_sink, window, p = 2, 16, 4, 6000, 4, 512, 0.9
    mask = [1, 0, 1, 0]
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    k, v, q = rnd(Bs, Hkv, L, 128), rnd(Bs, Hkv, L, 128), (2 * rnd(Bs, Hq, 128).float()).bfloat16()
    P_q, P_k = (0.2 * torch.randn(n, 16, 128, generator=g, device="cuda") for n in (Hq, Hkv))
    lens, zero = i64([L, L - 777]), i64([0, 0])
    h = B.spa_create(B.make_config(max_batch=Bs, n_q_heads=Hq, n_kv_heads=Hkv, max_ctx=L, kv_dtype=B.SPA_BF16, P_q=P_q, P_k=P_k))
    idx = torch.zeros(Bs, Hkv, L, 16, dtype=torch.int16, device="cuda")
    with Rope() as r:
        k_cache = torch.empty_like(k)
        B.spa_rope_apply(r.h, k, k_cache, Bs, L, Hkv, 128, B.SPA_BF16, start_pos=zero)
        B.spa_index_append(h, k, zero, Bs, L, idx)
        want = torch.empty(Bs, Hq, 128, device="cuda")
        B.spa_decode(h, q, k_cache, v, idx, mask, lens, Bs, 0, p, n_sink, window, want)
        sel = torch.empty(Bs, Hkv, L, dtype=torch.int32, device="cuda")
        cnt = torch.empty(Bs * Hkv, dtype=torch.int32, device="cuda")
        B.spa_select(h, q, idx, mask, lens, Bs, 0, p, n_sink, window, sel, cnt)
        B.spa_device_status(h)
        lists = {(b, x): sel[b, x, :int(cnt[b * Hkv + x])].long() for b in range(Bs) for x in range(Hkv)}
        for fmt in ("bf16", "int4"):
            with Cache([L, L - 777], Hq, Hkv, fmt, 64, "bf16", r, k=k, v=v) as c:
                out = torch.empty(Bs, Hq, 128, device="cuda")
                B.spa_attend_paged(c.h, q, c.pages, c.table, lens, Bs, 0, out, head_mask=mask, n_sink=n_sink, window=window,
                                   sel_idx=sel, sel_count=cnt, sel_stride=L)
                B.spa_paged_status(c.h)
                c.check(q, out, mask=mask, n_sink=n_sink, window=window, lists=lists)
                if fmt == "bf16":
                    # the same rows; scores of both are known to 2^-16 of sum |q k| / sqrt(128) (about 20 here)
                    assert torch.equal(c.kr[0].bfloat16(), k_cache[0])
                    assert (out - want).abs().max() <= 1e-3
    B.spa_destroy(h)


def test_prefix_read_back_for_prefill():
    """A prefix in 4-bit pages read back as bf16 rows is a cache that spa_prefill takes: its last row is the pages'
    attention, but for the roundings that prefill's tensor cores and the read add (2^-8 on queries, keys, values, weights)."""
    Hq, Hkv, L, T = 8, 2, 1000, 64
    with Rope() as r, Cache([L], Hq, Hkv, "int4", 16, "bf16", r) as c:
        k, v = torch.empty(2, 1, Hkv, L, 128, device="cuda", dtype=torch.bfloat16).unbind(0)
        B.spa_kv_read_paged(c.h, c.pages, c.table, c.zero, 1, L, k, v)
        P = torch.zeros(Hq, 16, 128, device="cuda")
        h = B.spa_create(B.make_config(max_batch=1, n_q_heads=Hq, n_kv_heads=Hkv, max_ctx=L, kv_dtype=B.SPA_BF16, P_q=P, P_k=P[:Hkv]))
        g = torch.Generator(device="cuda").manual_seed(4)
        q = torch.randn(1, Hq, T, 128, generator=g, device="cuda").bfloat16()
        pre = torch.empty(1, Hq, T, 128, device="cuda")
        B.spa_prefill(h, q, k, v, [1] * Hkv, i64([L - T]), 1, T, 4, 64, pre)
        B.spa_device_status(h)
        B.spa_destroy(h)
        last = q[:, :, -1].contiguous()
        out = torch.empty(1, Hq, 128, device="cuda")
        B.spa_attend_paged(c.h, last, c.pages, c.table, c.n, 1, 0, out)
        qq = c.rotated(last)
        for h_ in range(Hq):
            kk, vv = c.kr[0, h_ // 4].double(), c.vr[0, h_ // 4].double()
            p = torch.softmax(kk @ qq[0, h_] / math.sqrt(128), 0)
            off = 2 * 2.0 ** -8 * (kk.abs() @ qq[0, h_].abs() / math.sqrt(128)).max()
            bound = (2 * off + 4 * 2.0 ** -8) * (p @ vv.abs())
            assert ((pre[0, h_, -1] - out[0, h_]).abs() <= bound).all()


def test_graphs_streams_and_handles():
    """An append and an attention captured once and replayed as the sequence grows; two handles' graphs replayed at the same
    time on two streams; a call on a stream of its own."""
    lens, Hq, Hkv = [3000, 100], 8, 2
    with Rope() as r, Cache(lens, Hq, Hkv, "int4", 16, "bf16", r, handles=2) as c:
        q = queries(c)
        new_k, new_v = torch.randn(2, 2, Hkv, 1, 128, device="cuda").bfloat16().unbind(0)
        # room for three more tokens: sequence 1 has it, sequence 0's pages end at 3008
        n = c.n.clone()
        out = torch.empty(2, Hq, 128, device="cuda")
        B.spa_attend_paged(c.h, q, c.pages, c.table, n, 2, 0, out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.spa_kv_append_paged(c.h, new_k, new_v, n, 2, 1, c.table, c.pages)
            n.add_(1)
            B.spa_attend_paged(c.h, q, c.pages, c.table, n, 2, 0, out)
        for step in range(3):
            new_k.normal_()
            new_v.normal_()
            g.replay()
            torch.cuda.synchronize()
            assert n.tolist() == [3001 + step, 101 + step]
            eager = torch.empty_like(out)
            B.spa_attend_paged(c.h, q, c.pages, c.table, n, 2, 0, eager)
            assert torch.equal(eager, out)
        B.spa_paged_status(c.h)
        # two graphs at once, a handle each
        outs = [torch.empty_like(out) for _ in range(2)]
        graphs = []
        for h, o in zip(c.handles, outs):
            gg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gg):
                for _ in range(8):
                    B.spa_attend_paged(h, q, c.pages, c.table, n, 2, 0, o)
            graphs.append(gg)
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(20):
            for gg, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    gg.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager)
        o = torch.zeros_like(out)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        B.spa_attend_paged(c.h, q, c.pages, c.table, n, 2, 0, o, stream=st)
        st.synchronize()
        assert torch.equal(o, eager)
        for h in c.handles:
            B.spa_paged_status(h)


def test_a_mask_of_the_wrong_length_and_host_tensors_are_refused():
    with Cache([20], 4, 2, "int4", 16, "bf16") as c:
        q, out = queries(c), torch.empty(1, 4, 128, device="cuda")
        for mask in ([1], b"\1\1\1", torch.ones(5)):
            with pytest.raises(ValueError):
                B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, 1, 0, out, head_mask=mask, n_sink=1, window=1)
        with pytest.raises(ValueError):
            B.spa_attend_paged(c.h, q.cpu(), c.pages, c.table, c.n, 1, 0, out)
        for kw in (dict(max_seq_len=-1), dict(max_seq_len=33), dict(B=2), dict(B=0), dict(sel_idx=c.table),
                   dict(sel_idx=c.table, sel_count=c.table), dict(head_mask=b"\0\1"), dict(head_mask=b"\0\1", n_sink=-1, window=5),
                   dict(head_mask=b"\0\1", window=1, sel_idx=c.table, sel_count=c.table, sel_stride=0),
                   dict(head_mask=b"\0\1", window=1, sel_idx=c.table, sel_count=c.table, sel_stride=(1 << 24) + 1)):
            a = {**dict(B=1, max_seq_len=0), **kw}
            with pytest.raises(B.SpaError) as e:
                B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, a.pop("B"), a.pop("max_seq_len"), out, **a)
            assert e.value.status == B.SPA_ERR_INVALID_ARG
        with pytest.raises(B.SpaError):
            B.spa_kv_append_paged(c.h, c.k, c.v, c.zero, 1, 33, c.table, c.pages)             # T beyond the capacity
        with pytest.raises(B.SpaError):
            B.spa_kv_append_paged(c.h, c.k, c.v, c.zero, 1, 1, c.table, c.pages, k_strides=(128, 128, 4))
        B.spa_paged_status(c.h)


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_attend_shares_of_unequal_length(fmt):
    """40 slices over the GPU's CTAs, 3 each: the largest share is a quarter above the equal one, yet whole slices."""
    lens, Hq, Hkv = [14000, 14001, 13990, 14000, 13985], 32, 8
    with Rope() as r, Cache(lens, Hq, Hkv, fmt, 16, "bf16", r) as c:
        q = queries(c, seed=3)
        out = torch.full((c.B, Hq, 128), float("nan"), device="cuda")
        lse = torch.full((c.B, Hq), float("nan"), device="cuda")
        B.spa_attend_paged(c.h, q, c.pages, c.table, c.n, c.B, 0, out, lse=lse)
        B.spa_paged_status(c.h)
        c.check(q, out, lse)


@pytest.mark.parametrize("H,T,dtype,rot,layout", [
    (40, 64, "bf16", 128, "interleaved"),   # 2 heads a thread
    (9, 61, "bf16", 128, "half"),           # groups clipped to the heads
    (33, 100, "bf16", 64, "half"),          # some threads with a head more than others
    (12, 700, "f32", 36, "half"),
    (8, 1, "f32", 128, "interleaved"),
])
def test_rope_heads_shared_among_threads(H, T, dtype, rot, layout):
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn((1, T, H, 128), generator=g, device="cuda").to(TDT[dtype])
    y = torch.full_like(x, float("nan"))
    st = (T * H * 128, H * 128, 128)
    with Rope(rot, layout, "plain") as r:
        B.spa_rope_apply(r.h, x, y, 1, T, H, 128, KDT[dtype], start_pos=i64([70001]), x_strides=st, y_strides=st)
        xs = f64(x).transpose(0, 2, 1, 3)
        want = M.rotate(xs, 70001.0 + np.arange(T)[None, None, :], **r.model)
    got = f64(y).transpose(0, 2, 1, 3)
    assert (np.abs(got - want) <= rope_bound(xs, want, dtype, 1.0)).all()
    assert np.array_equal(got[..., rot:], xs[..., rot:])
