"""The paged-cache operators as a user's program calls them, and in plain torch.

Four operators of one path: rotary positions, appending keys and values to a paged cache (rotated on the way),
reading pages back into contiguous rows, and single-token attention over the pages.  A page holds page_size tokens
of every KV head as blocks of 16 tokens:
  int4 block (2304 bytes): K codes [16][64], V codes [16][64], bf16 scales [16][8] (4 K groups, then 4 V groups);
      dim d of a row is nibble d (low nibble first), its value scale * (nibble - 8); the scale group of dim d is
      (d / 8) % 4 for K and (d / 4) % 4 for V, so a group is 32 dims;
  bf16 block (8192 bytes): K [16][128], V [16][128]; the 16-byte piece c of row r sits at piece c ^ (r % 8).
"""
import math

import torch

own = False

D = 128
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the query rotation of one decode step, 16 sequences (the launch is what it costs)
        dict(name="rope_decode", op="rope", B=16, T=1, H=32, d=128, rot=128, layout="half", scaling="plain", dtype="bf16",
             order="heads", transpose=False, theta=500000.0, start=65535),
        # the keys and queries of a long prompt chunk, token-major as the projection leaves them, frequencies in bands
        dict(name="rope_prompt", op="rope", B=1, T=32768, H=40, d=128, rot=128, layout="interleaved", scaling="bands",
             dtype="bf16", order="tokens", transpose=False, theta=500000.0, start=98304),
        # the gradient of a partial rotation in float32, odd sizes
        dict(name="rope_gradient", op="rope", B=2, T=4097, H=9, d=80, rot=36, layout="half", scaling="ramp", dtype="f32",
             order="tokens", transpose=True, theta=10000.0, start=0),
        # one decode step's new rows of 16 sequences into 4-bit pages, and those rows read back
        dict(name="append_decode_int4", op="append", B=16, T=1, Hq=32, Hkv=8, page=16, fmt="int4", dtype="bf16",
             order="tokens", start=4095, ragged=0, layout="half", scaling="plain"),
        # a 32K prompt into 4-bit pages out of the fused projection's rows, read back for the chunk's own attention
        dict(name="append_prompt_int4", op="append", B=1, T=32768, Hq=32, Hkv=8, page=64, fmt="int4", dtype="bf16",
             order="tokens", start=0, ragged=0, layout="half", scaling="bands"),
        # a padded batch of chunks that end inside pages, into bf16 pages
        dict(name="append_ragged_bf16", op="append", B=5, T=1531, Hq=8, Hkv=2, page=48, fmt="bf16", dtype="bf16",
             order="heads", start=777, ragged=311, layout="interleaved", scaling="linear"),
        # a 32K prefix of one sequence out of 4-bit pages
        dict(name="read_int4", op="read", B=1, L=32768, Hkv=8, page=64, fmt="int4", dtype="bf16", ragged=0),
        # ragged prefixes out of bf16 pages
        dict(name="read_ragged_bf16", op="read", B=6, L=20011, Hkv=4, page=16, fmt="bf16", dtype="bf16", ragged=3001),
        # the smallest attention: one short sequence
        dict(name="attend_short_int4", op="attend", B=1, L=257, Hq=32, Hkv=8, page=16, fmt="int4", dtype="bf16", ragged=0,
             heads="all", n_sink=0, window=0, listed=0.0, scaling="plain"),
        # one 1M-token sequence, 8 query heads to a KV head, every row
        dict(name="attend_1m_int4", op="attend", B=1, L=1048576, Hq=64, Hkv=8, page=64, fmt="int4", dtype="bf16", ragged=0,
             heads="all", n_sink=0, window=0, listed=0.0, scaling="plain"),
        # the head-partitioned step at 128K: half the heads stream, the others have a selected list
        dict(name="attend_lists_int4", op="attend", B=4, L=131072, Hq=32, Hkv=8, page=128, fmt="int4", dtype="bf16",
             ragged=9973, heads="even", n_sink=4, window=4096, listed=0.25, scaling="plain"),
        # 16 sequences up to 64K on bf16 pages, two of eight heads see every row, the others stream
        dict(name="attend_batch_bf16", op="attend", B=16, L=65536, Hq=32, Hkv=8, page=32, fmt="bf16", dtype="bf16",
             ragged=3331, heads="quarter", n_sink=4, window=2048, listed=0.0, scaling="bands"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    order, layout = rng.choice(["heads", "tokens"]), rng.choice(["half", "interleaved"])
    scaling = rng.choice(["plain", "linear", "base", "bands", "ramp"])
    if op == "rope":
        d = rng.choice([128, 128, 64, 80, 96, 256, 2 * rng.randint(2, 128)])
        rot = rng.choice([d, d, 2 * rng.randint(2, d // 2)])
        return dict(op=op, B=rng.randint(1, 6), T=_log(rng, 1, 8192), H=rng.randint(1, 48), d=d, rot=rot, layout=layout,
                    scaling=scaling, dtype=dtype, order=order, transpose=rng.random() < 0.4,
                    theta=rng.choice([10000.0, 500000.0]), start=_log(rng, 1, 1 << 20) - 1)
    fmt = rng.choice(["int4", "int4", "bf16"])
    page, Hkv, G = 16 * rng.choice([1, 2, 3, 4, 8, 16]), rng.randint(1, 10), rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if op == "append":
        T = _log(rng, 1, 16384)
        # float32 rows read back out of bf16 pages would be held to float32's bound, which their storage rules out
        dtype = dtype if fmt == "int4" else "bf16"
        return dict(op=op, B=rng.randint(1, 4), T=T, Hq=G * Hkv, Hkv=Hkv, page=page, fmt=fmt, dtype=dtype, order=order,
                    start=_log(rng, 1, 50000) - 1, ragged=rng.choice([0, rng.randint(0, T)]), layout=layout, scaling=scaling)
    L = _log(rng, 1, 100000)
    ragged = rng.choice([0, rng.randint(0, L // 2 + 1)])
    if op == "read":
        return dict(op=op, B=rng.randint(1, 4), L=L, Hkv=Hkv, page=page, fmt=fmt, dtype=dtype, ragged=ragged)
    heads = rng.choice(["all", "even", "quarter", "none"])
    n_sink = rng.randint(0, 9)
    window = rng.randint(1, 5000) if heads != "all" else 0
    return dict(op=op, B=rng.randint(1, 8), L=L, Hq=G * Hkv, Hkv=Hkv, page=page, fmt=fmt, dtype=dtype, ragged=ragged,
                heads=heads, n_sink=n_sink if heads != "all" else 0, window=window,
                listed=rng.choice([0.0, 0.3 * rng.random()]) if heads != "all" else 0.0, scaling=scaling)


# ------------------------------------------------------------------------------------------------ shared sizes
def _rows(case):
    """Rows (append, read) or lengths (attend) of each sequence: a batch whose sequence b is b * ragged shorter."""
    n = case["T"] if case["op"] == "append" else case["L"]
    return [max(0, n - b * case["ragged"]) for b in range(case["B"])]


def _retrieval(case):
    Hkv, kind = case["Hkv"], case["heads"]
    return [kind == "all" or (kind == "even" and g % 2 == 0) or (kind == "quarter" and g % 4 == 0) for g in range(Hkv)]


def _attended(case, L, ret):
    """Rows that one KV head of a sequence of L tokens attends, and how many of them come from its list."""
    if ret and case["listed"] == 0.0:
        return L, 0
    n_s = min(case["n_sink"], L)
    fixed = n_s + L - max(n_s, L - case["window"])
    n = int(case["listed"] * (L - fixed)) if ret else 0
    return fixed + n, n


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        n = case["B"] * case["T"] * case["H"] * case["d"]
        return {"bytes": 2 * n * es + 8 * case["B"] * case["T"], "flops": 3 * n * case["rot"] / case["d"]}
    row = 144 if case["fmt"] == "int4" else 512
    n = sum(_rows(case)) * case["Hkv"]
    if case["op"] == "read":
        return {"bytes": n * (row + 2 * D * es), "flops": n * 2 * D}
    if case["op"] == "append":   # the rows, the pages written, then those pages read and the rows written
        return {"bytes": n * (2 * D * es + row) + n * (row + 2 * D * es), "flops": n * 10 * D}
    rows = [_attended(case, L, r) for L in _rows(case) for r in _retrieval(case)]
    heads = case["B"] * case["Hq"]
    return {"bytes": sum(r * row + 4 * l for r, l in rows) + heads * D * (es + 4), "flops": sum(r for r, _ in rows) * 4 * D * case["Hq"] // case["Hkv"]}


# ------------------------------------------------------------------------------------------------ inputs
class _Handle:
    """A library handle that lives as long as the state that holds it."""

    def __init__(self, value, destroy):
        self.value, self.destroy = value, destroy

    def __del__(self):
        self.destroy(self.value)


def _scaling(case):
    """The arguments of the frequency scaling: what a model's configuration says."""
    return {"plain": dict(), "linear": dict(factor=4.0), "base": dict(factor=8.0),
            "bands": dict(factor=8.0, low=1.0, high=4.0, orig_ctx=8192),
            "ramp": dict(factor=16.0, low=1.0, high=32.0, orig_ctx=4096, magnitude=0.1 * math.log(16.0) + 1.0)}[case["scaling"]]


def _rope_of(case):
    return dict(rot=case.get("rot", D), layout=case.get("layout", "half"), theta=case.get("theta", 500000.0),
                scaling=case["scaling"], **_scaling(case))


def _rope_handle(r):
    from head_partitioned_sparse_b200 import binding as spa
    kinds = {"plain": spa.SPA_ROPE_PLAIN, "linear": spa.SPA_ROPE_LINEAR, "base": spa.SPA_ROPE_BASE,
             "bands": spa.SPA_ROPE_BANDS, "ramp": spa.SPA_ROPE_RAMP}
    cfg = spa.make_rope_config(rot_dim=r["rot"], layout=spa.SPA_ROPE_HALF if r["layout"] == "half" else spa.SPA_ROPE_INTERLEAVED,
                               theta=r["theta"], scaling=kinds[r["scaling"]], factor=r.get("factor", 1.0), low=r.get("low", 1.0),
                               high=r.get("high", 4.0), orig_ctx=r.get("orig_ctx", 0), magnitude=r.get("magnitude", 1.0))
    return _Handle(spa.spa_rope_create(cfg), spa.spa_rope_destroy)


def _paged_handle(case, n_pages, max_pages, rope):
    from head_partitioned_sparse_b200 import binding as spa
    cfg = spa.make_paged_config(max_batch=case["B"], n_q_heads=case.get("Hq", case["Hkv"]), n_kv_heads=case["Hkv"],
                                kv_dtype=spa.SPA_BF16 if case["dtype"] == "bf16" else spa.SPA_F32,
                                page_format=spa.SPA_PAGE_INT4 if case["fmt"] == "int4" else spa.SPA_PAGE_BF16,
                                page_size=case["page"], n_pages=n_pages, max_pages=max_pages)
    return _Handle(spa.spa_paged_create(cfg, rope.value), spa.spa_paged_destroy)


def _filled_pages(case, n_pages, gen):
    """Pages that hold rows of an earlier time: codes as rounded Gaussians have them, scales of unit-variance groups."""
    n = n_pages * case["Hkv"] * (case["page"] // 16)
    dev = gen.device
    if case["fmt"] == "bf16":
        return torch.randn(n * 4096, generator=gen, device=dev, dtype=torch.bfloat16).view(torch.uint8).view(n_pages, case["Hkv"], -1, 8192)
    codes = torch.randn(n * 4096, generator=gen, device=dev, dtype=torch.bfloat16).mul_(3.2).round_().clamp_(-7, 7).add_(8).to(torch.uint8).view(-1, 2)
    blocks = torch.empty(n, 2304, dtype=torch.uint8, device=dev)
    blocks[:, :2048] = (codes[:, 0] | (codes[:, 1] << 4)).view(n, 2048)
    blocks[:, 2048:] = (0.2 + 0.2 * torch.rand(n, 128, generator=gen, device=dev)).bfloat16().view(torch.uint8)
    return blocks.view(n_pages, case["Hkv"], -1, 2304)


def _table(case, need, gen):
    """A block table over pages in random order, and the number of pages in the pool."""
    mp = max(1, -(-need // case["page"]))
    n_pages = case["B"] * mp + 3
    perm = torch.randperm(n_pages, generator=gen, device=gen.device)[: case["B"] * mp]
    return perm.view(case["B"], mp).to(torch.int32), n_pages, mp


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt, B = DT[case["dtype"]], case["B"]
    s = {"case": case}
    if case["op"] == "rope":
        T, H, d = case["T"], case["H"], case["d"]
        shape = (B, H, T, d) if case["order"] == "heads" else (B, T, H, d)
        s["x"] = torch.randn(shape, generator=gen, device=dev, dtype=dt)
        s["y"] = torch.empty_like(s["x"])
        s["start"] = case["start"] + torch.randint(0, 64, (B,), generator=gen, device=dev)
        s["rope"] = _rope_of(case)
        if own:
            s["h"] = _rope_handle(s["rope"])
        return s
    rows = _rows(case)
    s["rows"] = torch.tensor(rows, dtype=torch.int64, device=dev)
    s["rope"] = _rope_of(dict(case, scaling=case.get("scaling", "plain")))
    if case["op"] == "append":
        T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
        s["start"] = case["start"] + torch.randint(0, 8, (B,), generator=gen, device=dev)
        s["table"], n_pages, mp = _table(case, case["start"] + 8 + T, gen)
        nb = case["page"] // 16
        s["pages"] = torch.zeros(n_pages, Hkv, nb, 2304 if case["fmt"] == "int4" else 8192, dtype=torch.uint8, device=dev)
        if case["order"] == "tokens":   # the rows of a fused projection: q heads, then k heads, then v heads
            s["qkv"] = torch.randn(B, T, Hq + 2 * Hkv, D, generator=gen, device=dev, dtype=dt)
            s["k"], s["v"] = s["qkv"][:, :, Hq:Hq + Hkv].transpose(1, 2), s["qkv"][:, :, Hq + Hkv:].transpose(1, 2)
        else:
            s["k"] = torch.randn(B, Hkv, T, D, generator=gen, device=dev, dtype=dt)
            s["v"] = torch.randn(B, Hkv, T, D, generator=gen, device=dev, dtype=dt)
    else:
        s["table"], n_pages, mp = _table(case, case["L"], gen)
        s["pages"] = _filled_pages(case, n_pages, gen)
        T = case["L"]
    if case["op"] != "attend":
        s["zero"] = torch.zeros(B, dtype=torch.int64, device=dev)
        s["k_rows"] = torch.zeros(B, case["Hkv"], T, D, dtype=dt, device=dev)
        s["v_rows"] = torch.zeros(B, case["Hkv"], T, D, dtype=dt, device=dev)
    else:
        Hq, Hkv = case["Hq"], case["Hkv"]
        s["q"] = 1.5 * torch.randn(B, Hq, D, generator=gen, device=dev, dtype=dt)
        s["out"] = torch.empty(B, Hq, D, dtype=torch.float32, device=dev)
        ret = _retrieval(case)
        s["mask"] = None if case["heads"] == "all" else bytes(int(r) for r in ret)
        s["list"] = s["count"] = None
        if case["listed"]:
            s["list"], s["count"] = _lists(case, rows, ret, gen)
    if own:
        s["rope_handle"] = _rope_handle(s["rope"])
        s["h"] = _paged_handle(case, n_pages, mp, s["rope_handle"])
    return s


def _lists(case, rows, ret, gen):
    """Ascending positions outside sinks and window, as a selection returns them: [B][Hkv][L] and their counts."""
    dev, L = gen.device, case["L"]
    lists = torch.zeros(case["B"], case["Hkv"], L, dtype=torch.int32, device=dev)
    counts = [[_attended(case, n, r)[1] for r in ret] for n in rows]
    for b, n in enumerate(rows):
        lo = min(case["n_sink"], n)
        hi = max(lo, n - case["window"])
        for g in range(case["Hkv"]):
            c = counts[b][g]
            if c:
                lists[b, g, :c] = (lo + torch.randperm(hi - lo, generator=gen, device=dev)[:c].sort().values).to(torch.int32)
    return lists, torch.tensor(counts, dtype=torch.int32, device=dev).view(-1)


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "rope":
        x = state["x"] if case["order"] == "tokens" else state["x"].transpose(1, 2)      # [B][T][H][d]
        pos = state["start"][:, None] + torch.arange(case["T"], device=x.device)
        y = _rotate(x.float(), pos[:, :, None], state["rope"], case["transpose"], torch.float32).to(x.dtype)
        return y if case["order"] == "tokens" else y.transpose(1, 2).contiguous()
    if case["op"] == "read":
        return _plain_read(state, case, state["zero"], case["L"])
    if case["op"] == "append":
        _plain_append(state, case)
        return _plain_read(state, case, state["start"], case["T"])
    return _plain_attend(state, case)


def _run_own(state, case):
    from head_partitioned_sparse_b200 import binding as spa
    h, B = state["h"].value, case["B"]
    if case["op"] == "rope":
        T, H, d = case["T"], case["H"], case["d"]
        strides = (T * H * d, H * d, d) if case["order"] == "tokens" else None
        spa.spa_rope_apply(h, state["x"], state["y"], B, T, H, d, spa.SPA_BF16 if case["dtype"] == "bf16" else spa.SPA_F32,
                           start_pos=state["start"], x_strides=strides, y_strides=strides, transpose=case["transpose"])
        return state["y"]
    pages, table, rows = state["pages"], state["table"], state["rows"]
    if case["op"] == "append":
        k, v = state["k"], state["v"]
        strides = None
        if case["order"] == "tokens":
            strides = (k.stride(0), k.stride(2), k.stride(1))
        spa.spa_kv_append_paged(h, k, v, state["start"], B, case["T"], table, pages, n_new=rows, k_strides=strides, v_strides=strides)
        spa.spa_kv_read_paged(h, pages, table, state["start"], B, case["T"], state["k_rows"], state["v_rows"], n_rows=rows)
        return state["k_rows"], state["v_rows"]
    if case["op"] == "read":
        spa.spa_kv_read_paged(h, pages, table, state["zero"], B, case["L"], state["k_rows"], state["v_rows"], n_rows=rows)
        return state["k_rows"], state["v_rows"]
    spa.spa_attend_paged(h, state["q"], pages, table, rows, B, case["L"], state["out"], head_mask=state["mask"],
                         n_sink=case["n_sink"], window=case["window"], sel_idx=state["list"], sel_count=state["count"],
                         sel_stride=case["L"])
    return state["out"]


# ------------------------------------------------------------------------------------------------ the plain form
def _frequencies(r, device):
    """Inverse frequencies of the rot / 2 pairs, in 64 bits."""
    rot, theta = r["rot"], r["theta"]
    if r["scaling"] == "base":
        theta = theta * r["factor"] ** (rot / (rot - 2))
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    f = theta ** (-2 * i / rot)
    if r["scaling"] == "linear":
        f = f / r["factor"]
    if r["scaling"] == "bands":
        keep = ((r["orig_ctx"] * f / (2 * math.pi) - r["low"]) / (r["high"] - r["low"])).clamp(0, 1)
        f = f * (keep + (1 - keep) / r["factor"])
    if r["scaling"] == "ramp":
        at = [rot * math.log(r["orig_ctx"] / (2 * math.pi * turns)) / (2 * math.log(theta)) for turns in (r["high"], r["low"])]
        lo, hi = min(max(math.floor(at[0]), 0), rot - 1), min(max(math.ceil(at[1]), 0), rot - 1)
        keep = 1 - ((i - lo) / (hi - lo if hi > lo else 0.001)).clamp(0, 1)
        f = f * (keep + (1 - keep) / r["factor"])
    return f


def _rotate(x, pos, r, transpose, dtype):
    """x [..., d] at positions pos (broadcast over the leading dims); angles in 64 bits, the products in `dtype`."""
    rot = r["rot"]
    a = pos[..., None].double() * _frequencies(r, x.device)
    m = r.get("magnitude", 1.0)
    c, s = (a.cos() * m).to(dtype), (a.sin() * (-m if transpose else m)).to(dtype)
    if r["layout"] == "half":
        u, v = x[..., : rot // 2], x[..., rot // 2: rot]
        return torch.cat((u * c - v * s, u * s + v * c, x[..., rot:]), -1)
    u, v = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat((torch.stack((u * c - v * s, u * s + v * c), -1).flatten(-2), x[..., rot:]), -1)


def _quantise(x, groups):
    """Codes 1..15 (uint8) and bf16 scales [..., 4] of x [..., 128] in 64 bits; groups: the scale group of each dim."""
    amax = torch.stack([x[..., groups == g].abs().amax(-1) for g in range(4)], -1)
    # rounded to bf16 once: 64-bit values have no tie that float32 would make or break here beyond its own grid
    e = torch.floor(torch.log2(torch.where(amax > 0, amax / 7, 1.0)))
    step = torch.exp2(e - 7)
    scale = torch.where(amax > 0, torch.round(amax / 7 / step) * step, 0.0)
    q = x / torch.where(scale > 0, scale, 1.0)[..., groups]
    return (torch.round(q).clamp(-7, 7) + 8).to(torch.uint8), scale.bfloat16()


def _groups(device):
    d = torch.arange(D, device=device)
    return (d // 8) % 4, (d // 4) % 4


def _plain_append(state, case):
    """Rotates, rounds and writes the new rows into their pages."""
    k, v, dev = state["k"], state["v"], state["k"].device
    B, Hkv, T, _ = k.shape
    i = torch.arange(T, device=dev)
    pos = state["start"][:, None] + i                                                    # [B][T]
    b, t = torch.nonzero(i < state["rows"][:, None], as_tuple=True)
    pos = pos[b, t]
    page, block, r = state["table"].long()[b, pos // case["page"]], pos % case["page"] // 16, pos % 16
    k, v = k[b, :, t], v[b, :, t]                                                        # [n][Hkv][128]
    pages = state["pages"]
    heads = torch.arange(Hkv, device=dev)[None, :, None]
    page, block, r = page[:, None, None], block[:, None, None], r[:, None, None]
    if case["fmt"] == "int4":
        kq, ks = _quantise(_rotate(k.double(), pos[:, None], state["rope"], False, torch.float64), _groups(dev)[0])
        vq, vs = _quantise(v.double(), _groups(dev)[1])
        byte = torch.arange(64, device=dev)
        pages[page, heads, block, r * 64 + byte] = kq[..., 0::2] | (kq[..., 1::2] << 4)
        pages[page, heads, block, 1024 + r * 64 + byte] = vq[..., 0::2] | (vq[..., 1::2] << 4)
        pages[page, heads, block, 2048 + r * 16 + torch.arange(16, device=dev)] = torch.cat((ks, vs), -1).view(torch.uint8)
        return
    k = _rotate(k.float(), pos[:, None], state["rope"], False, torch.float32)
    byte = torch.arange(256, device=dev)
    at = r * 256 + (((byte // 16) ^ (r % 8)) * 16 + byte % 16)
    pages[page, heads, block, at] = k.bfloat16().view(torch.uint8)
    pages[page, heads, block, 4096 + at] = v.bfloat16().view(torch.uint8)


def _unpack(blocks, fmt):
    """K and V [..., 16, 128] in 32 bits out of blocks [..., bytes]."""
    lead = blocks.shape[:-1]
    if fmt == "bf16":
        r, d = torch.arange(16, device=blocks.device)[:, None], torch.arange(D, device=blocks.device)
        at = ((d // 8) ^ (r % 8)) * 8 + d % 8
        kv = blocks.contiguous().view(torch.bfloat16).view(*lead, 2, 16, D)
        kv = torch.gather(kv, -1, at.expand(*lead, 2, 16, D)).float()
        return kv[..., 0, :, :], kv[..., 1, :, :]
    scale = blocks[..., 2048:].contiguous().view(torch.bfloat16).view(*lead, 16, 8).float()
    gk, gv = _groups(blocks.device)
    n = blocks[..., :2048].unflatten(-1, (2, 16, 64))
    n = torch.stack((n & 15, n >> 4), -1).flatten(-2).float() - 8
    return n[..., 0, :, :] * scale[..., :4][..., gk], n[..., 1, :, :] * scale[..., 4:][..., gv]


def _gathered(state, case):
    """K and V of every sequence's table, [B][Hkv][positions][128]."""
    blocks = state["pages"][state["table"].long()].transpose(1, 2)                       # [B][Hkv][max_pages][blocks][bytes]
    k, v = _unpack(blocks.flatten(2, 3), case["fmt"])
    return k.flatten(2, 3), v.flatten(2, 3)


def _plain_read(state, case, start, T):
    k, v = _gathered(state, case)
    i = torch.arange(T, device=k.device)
    at = (start[:, None] + i).clamp(max=k.shape[2] - 1)[:, None, :, None].expand(-1, case["Hkv"], -1, D)
    live = (i < state["rows"][:, None])[:, None, :, None]
    dt = DT[case["dtype"]]
    return (torch.where(live, k.gather(2, at), 0.0).to(dt), torch.where(live, v.gather(2, at), 0.0).to(dt))


def _plain_attend(state, case):
    k, v = _gathered(state, case)                                                        # [B][Hkv][N][128]
    B, Hkv, N, _ = k.shape
    L, G = state["rows"][:, None, None], case["Hq"] // Hkv
    j = torch.arange(N, device=k.device)
    seen = (j < L).expand(B, Hkv, N)
    if state["mask"] is not None:
        near = seen & ((j < case["n_sink"]) | (j >= L - case["window"]))
        ret = torch.tensor(list(state["mask"]), device=k.device, dtype=torch.bool)[:, None]
        if state["list"] is None:
            seen = torch.where(ret, seen, near)
        else:
            lists = state["list"].long()
            c = torch.arange(lists.shape[2], device=k.device)
            lists = torch.where(c < state["count"].view(B, Hkv, 1), lists, N)
            chosen = torch.zeros(B, Hkv, N + 1, dtype=torch.bool, device=k.device).scatter_(2, lists, True)[..., :N]
            seen = near | (chosen & ret)
    last = (state["rows"] - 1).clamp(min=0)[:, None]
    q = _rotate(state["q"].float(), last, state["rope"], False, torch.float32).view(B, Hkv, G, D)
    s = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(D)
    s = torch.where(seen[:, :, None], s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return torch.matmul(p, v).view(B, case["Hq"], D)


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        x = s["x"] if case["order"] == "heads" else s["x"].transpose(1, 2)               # [B][H][T][d]
        pos = s["start"][:, None] + torch.arange(case["T"], device=x.device)
        z = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        for b in range(case["B"]):
            z[b] = _turn(x[b].double(), pos[b], s["rope"], -1.0 if case["transpose"] else 1.0)
        return z if case["order"] == "heads" else z.transpose(1, 2).contiguous()
    if case["op"] == "attend":
        return _exact_attend(s, case)
    if case["op"] == "append":
        out = torch.zeros((2,) + tuple(s["k"].shape), dtype=torch.float64, device="cuda")
        for b, n in enumerate(_rows(case)):
            if n == 0:
                continue
            pos = s["start"][b] + torch.arange(n, device="cuda")
            k = _turn(s["k"][b, :, :n].double(), pos, s["rope"], 1.0)
            v = s["v"][b, :, :n].double()
            if case["fmt"] == "int4":
                k, v = _in_4_bits(k, 8), _in_4_bits(v, 4)
            out[0, b, :, :n], out[1, b, :, :n] = k, v
        return out[0], out[1]
    out = torch.zeros((2,) + tuple(s["k_rows"].shape), dtype=torch.float64, device="cuda")
    for b, n in enumerate(_rows(case)):
        for g in range(case["Hkv"]):
            k, v = _one_head(s, case, b, g)
            out[0, b, g, :n], out[1, b, g, :n] = k[:n], v[:n]
    return out[0], out[1]


def _turn(x, pos, r, sign):
    """x [H][T][d] turned by complex numbers, pair by pair."""
    n = r["rot"]
    z = torch.complex(x[..., : n // 2], x[..., n // 2: n]) if r["layout"] == "half" else torch.view_as_complex(x[..., :n].reshape(*x.shape[:-1], n // 2, 2))
    theta = r["theta"] * (r["factor"] ** (n / (n - 2.0)) if r["scaling"] == "base" else 1.0)
    f = []
    for i in range(n // 2):
        w = math.exp(-2.0 * i / n * math.log(theta))
        if r["scaling"] == "linear":
            w /= r["factor"]
        elif r["scaling"] in ("bands", "ramp"):
            if r["scaling"] == "bands":
                mix = (w * r["orig_ctx"] / (2 * math.pi) - r["low"]) / (r["high"] - r["low"])
            else:
                first = max(0, math.floor(n / 2 * math.log(r["orig_ctx"] / (r["high"] * 2 * math.pi)) / math.log(theta)))
                last = max(0, math.ceil(n / 2 * math.log(r["orig_ctx"] / (r["low"] * 2 * math.pi)) / math.log(theta)))
                first, last = min(first, n - 1), min(last, n - 1)
                mix = 1 - (i - first) / (last - first if last > first else 0.001)
            mix = min(1.0, max(0.0, mix))
            w = w * mix + (1 - mix) * w / r["factor"]
        f.append(w)
    angle = pos.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    z = z * torch.polar(torch.full_like(angle, r.get("magnitude", 1.0)), sign * angle)
    y = x.clone()
    if r["layout"] == "half":
        y[..., : n // 2], y[..., n // 2: n] = z.real, z.imag
    else:
        y[..., 0:n:2], y[..., 1:n:2] = z.real, z.imag
    return y


def _in_4_bits(x, run):
    """The values that 4 bits keep of x [H][T][128], whose groups are runs of `run` dims, every fourth of them."""
    y = x.unflatten(-1, (-1, 4, run))                                                    # [H][T][128 / (4 run)][4][run]
    m, e = torch.frexp(y.abs().amax((-3, -1), keepdim=True) / 7)
    s = torch.ldexp(torch.round(m * 256), e - 8)                                         # 8 significant bits
    n = torch.where(s > 0, torch.round(y / torch.where(s > 0, s, 1.0)), 0.0)
    return (n.clamp(-7, 7) * s).flatten(-3)


def _one_head(s, case, b, g):
    """K and V of one KV head over its whole table, [positions][128] in 64 bits."""
    blk = s["pages"][s["table"][b].long(), g].flatten(0, 1)                              # [blocks][bytes]
    n = blk.shape[0]
    if case["fmt"] == "bf16":
        w = blk.view(torch.bfloat16).view(n, 2, 16, 16, 8).double()
        w = torch.stack([w[:, :, r, [c ^ (r % 8) for c in range(16)]] for r in range(16)], 2).view(n, 2, 16, D)
        return w[:, 0].reshape(-1, D), w[:, 1].reshape(-1, D)
    table = torch.tensor([[(x & 15) - 8, (x >> 4) - 8] for x in range(256)], dtype=torch.float64, device=blk.device)
    codes = table[blk[:, :2048].long()].view(n, 2, 16, D)
    sc = blk[:, 2048:].contiguous().view(torch.bfloat16).view(n, 16, 2, 4).double()
    k = codes[:, 0].view(n, 16, 4, 4, 8) * sc[:, :, 0][:, :, None, :, None]
    v = codes[:, 1].view(n, 16, 8, 4, 4) * sc[:, :, 1][:, :, None, :, None]
    return k.reshape(-1, D), v.reshape(-1, D)


def _exact_attend(s, case):
    G = case["Hq"] // case["Hkv"]
    ret = _retrieval(case)
    out = torch.zeros(case["B"], case["Hq"], D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_rows(case)):
        if n == 0:
            continue
        q = _turn(s["q"][b].double()[:, None], torch.tensor([n - 1], device="cuda"), s["rope"], 1.0)[:, 0]
        for g in range(case["Hkv"]):
            k, v = _one_head(s, case, b, g)
            if ret[g] and s["list"] is None:
                rows = torch.arange(n, device="cuda")
            else:
                lo = min(case["n_sink"], n)
                rows = torch.cat((torch.arange(lo, device="cuda"), torch.arange(max(lo, n - case["window"]), n, device="cuda")))
                if ret[g]:
                    rows = torch.cat((rows, s["list"][b, g, : int(s["count"][b * case["Hkv"] + g])].long()))
            w = torch.softmax(q[g * G: (g + 1) * G] @ k[rows].T / math.sqrt(D), -1)
            out[b, g * G: (g + 1) * G] = w @ v[rows]
    return out
