"""Rotary and paged-cache entry points: what is refused on the host, before any GPU is touched, and the
float64 model's own consistency.  No compute calls here."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import paged_model as M
from head_partitioned_sparse_b200 import binding as B


@pytest.fixture(scope="module", autouse=True)
def lib():
    from head_partitioned_sparse_b200 import build
    build.build()
    return B.load()


def refused(status, f, *a, **kw):
    with pytest.raises(B.SpaError) as e:
        f(*a, **kw)
    assert e.value.status == status and B.spa_last_error()


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=514), dict(rot_dim=-2), dict(layout=2), dict(layout=-1),
    dict(scaling=5), dict(scaling=-1), dict(theta=0.0), dict(theta=float("nan")), dict(theta=float("inf")),
    dict(magnitude=-1.0), dict(magnitude=float("nan")),
    dict(scaling=B.SPA_ROPE_LINEAR, factor=0.0), dict(scaling=B.SPA_ROPE_LINEAR, factor=float("inf")),
    dict(scaling=B.SPA_ROPE_BASE, rot_dim=2, factor=2.0),
    dict(scaling=B.SPA_ROPE_BANDS, factor=2.0, orig_ctx=0), dict(scaling=B.SPA_ROPE_BANDS, factor=2.0, orig_ctx=8, low=4.0),
    dict(scaling=B.SPA_ROPE_RAMP, factor=2.0, orig_ctx=8, low=0.0), dict(scaling=B.SPA_ROPE_RAMP, factor=2.0, orig_ctx=8, theta=1.0),
    dict(theta=5e-324, rot_dim=512),
])
def test_rope_config_refusals(kw):
    refused(B.SPA_ERR_INVALID_ARG, B.spa_rope_create, B.make_rope_config(**kw))


@pytest.fixture()
def rope():
    r = B.spa_rope_create(B.make_rope_config(rot_dim=64))
    yield r
    B.spa_rope_destroy(r)


def test_rope_apply_refusals(rope):
    X = 0x10000
    ok = dict(r=rope, x=X, y=X, B=1, T=1, n_heads=1, head_dim=64, dtype=B.SPA_BF16, start_pos=X)
    for status, kw in [
        (B.SPA_ERR_INVALID_ARG, dict(r=None)), (B.SPA_ERR_INVALID_ARG, dict(x=None)), (B.SPA_ERR_INVALID_ARG, dict(y=None)),
        (B.SPA_ERR_INVALID_ARG, dict(start_pos=None)), (B.SPA_ERR_INVALID_ARG, dict(positions=X)),
        (B.SPA_ERR_UNSUPPORTED, dict(dtype=2)), (B.SPA_ERR_INVALID_ARG, dict(x=X + 1)),
        (B.SPA_ERR_INVALID_ARG, dict(y=X + 2, dtype=B.SPA_F32)), (B.SPA_ERR_INVALID_ARG, dict(start_pos=X + 4)),
        (B.SPA_ERR_INVALID_ARG, dict(B=0)), (B.SPA_ERR_INVALID_ARG, dict(T=0)), (B.SPA_ERR_INVALID_ARG, dict(n_heads=0)),
        (B.SPA_ERR_INVALID_ARG, dict(head_dim=62)), (B.SPA_ERR_INVALID_ARG, dict(head_dim=65537)),
    ]:
        refused(status, B.spa_rope_apply, **{**ok, **kw})
    with pytest.raises(ValueError):
        B.spa_rope_apply(**{**ok, "x": torch.zeros(64)})     # host memory
    refused(B.SPA_ERR_INVALID_ARG, B.spa_rope_inv_freq, rope, 31)


def cfg(**kw):
    base = dict(max_batch=2, n_q_heads=8, n_kv_heads=2, kv_dtype=B.SPA_BF16, page_format=B.SPA_PAGE_INT4, page_size=64,
                n_pages=10, max_pages=4)
    return B.make_paged_config(**{**base, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=64), B.SPA_ERR_UNSUPPORTED), (dict(kv_dtype=3), B.SPA_ERR_UNSUPPORTED),
    (dict(page_format=2), B.SPA_ERR_UNSUPPORTED), (dict(n_kv_heads=65, n_q_heads=65), B.SPA_ERR_UNSUPPORTED),
    (dict(n_q_heads=18), B.SPA_ERR_UNSUPPORTED), (dict(n_q_heads=7), B.SPA_ERR_INVALID_ARG),
    (dict(max_batch=0), B.SPA_ERR_INVALID_ARG), (dict(max_batch=2049), B.SPA_ERR_INVALID_ARG),
    (dict(page_size=8), B.SPA_ERR_INVALID_ARG), (dict(page_size=24), B.SPA_ERR_INVALID_ARG),
    (dict(page_size=65552), B.SPA_ERR_INVALID_ARG), (dict(n_pages=0), B.SPA_ERR_INVALID_ARG),
    (dict(max_pages=0), B.SPA_ERR_INVALID_ARG), (dict(max_pages=(1 << 18) + 1), B.SPA_ERR_INVALID_ARG),
])
def test_paged_config_refusals(kw, status):
    refused(status, B.spa_paged_page_bytes, cfg(**kw))
    refused(status, B.spa_paged_create, cfg(**kw))


def test_page_bytes():
    assert B.spa_paged_page_bytes(cfg()) == 2 * 4 * 2304
    assert B.spa_paged_page_bytes(cfg(page_format=B.SPA_PAGE_BF16, page_size=16)) == 2 * 8192


def test_a_rotation_wider_than_the_head_is_refused():
    r = B.spa_rope_create(B.make_rope_config(rot_dim=256))
    refused(B.SPA_ERR_INVALID_ARG, B.spa_paged_create, cfg(), r)
    B.spa_rope_destroy(r)


def test_null_handles():
    X = 0x10000
    refused(B.SPA_ERR_INVALID_ARG, B.spa_kv_append_paged, None, X, X, X, 1, 1, X, X)
    refused(B.SPA_ERR_INVALID_ARG, B.spa_kv_read_paged, None, X, X, X, 1, 1, X, X)
    refused(B.SPA_ERR_INVALID_ARG, B.spa_attend_paged, None, X, X, X, X, 1, 0, X)
    refused(B.SPA_ERR_INVALID_ARG, B.spa_paged_status, None, 0)
    B.spa_paged_destroy(None)
    B.spa_rope_destroy(None)


def test_frequencies_match_the_model(rope):
    for scaling, name, kw in ((B.SPA_ROPE_PLAIN, "plain", {}), (B.SPA_ROPE_LINEAR, "linear", dict(factor=4.0)),
                              (B.SPA_ROPE_BASE, "base", dict(factor=8.0)),
                              (B.SPA_ROPE_BANDS, "bands", dict(factor=8.0, low=1.0, high=4.0, orig_ctx=8192)),
                              (B.SPA_ROPE_RAMP, "ramp", dict(factor=16.0, low=1.0, high=32.0, orig_ctx=4096))):
        r = B.spa_rope_create(B.make_rope_config(rot_dim=96, theta=10000.0, scaling=scaling, **kw))
        f = np.array(B.spa_rope_inv_freq(r, 48))
        assert np.allclose(f, M.frequencies(96, theta=10000.0, scaling=name, **kw), rtol=1e-13, atol=0)
        B.spa_rope_destroy(r)


@pytest.mark.parametrize("fmt", ["int4", "bf16"])
def test_model_pool_round_trip(fmt):
    rng = np.random.default_rng(0)
    pool = M.Pool(np.zeros((5, 2, 3, M.block_bytes(fmt)), np.uint8), fmt, 48)
    table = np.array([[3, 1], [0, 4]], np.int32)
    rows = {}
    for b, g, pos in ((0, 0, 0), (0, 1, 95), (1, 0, 47), (1, 1, 48), (0, 0, 17)):
        k, v = rng.standard_normal((2, 128))
        pool.put(table, b, g, pos, k, v)
        rows[b, g, pos] = (k, v)
    for (b, g, pos), (k, v) in rows.items():
        for x, y, grp in zip((k, v), pool.get(table, b, g, pos), (M.GROUP_K, M.GROUP_V)):
            if fmt == "bf16":
                assert np.array_equal(y, M.rne_bf16(x))
                continue
            # half a step of a group's scale: amax / 14, the scale itself off by 2^-9, the top level by as much
            amax = np.array([np.abs(x[grp == g2]).max() for g2 in range(4)])[grp]
            assert (np.abs(y - x) <= amax / 14 * (1 + 2.0 ** -8) + amax * 2.0 ** -9).all()


@pytest.mark.parametrize("n", [0, 1, 2, 4])
def test_strides_of_another_length_are_refused(rope, n):
    """Two strides would leave every head at the same place."""
    X, s = 0x10000, (64,) * n
    for kw in (dict(x_strides=s), dict(y_strides=s)):
        with pytest.raises(ValueError, match="strides"):
            B.spa_rope_apply(rope, X, X, 1, 1, 1, 64, B.SPA_BF16, start_pos=X, **kw)
    for f in (B.spa_kv_append_paged, B.spa_kv_read_paged):
        for kw in (dict(k_strides=s), dict(v_strides=s)):
            with pytest.raises(ValueError, match="strides"):
                f(None, X, X, X, 1, 1, X, X, **kw)


@pytest.mark.parametrize("private", [True, False])
def test_device_and_stream_without_torchs_private_functions(monkeypatch, private):
    class Stream:
        cuda_stream = 0x77
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream() if device == 1 else None)
    if private:
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x77, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(B, "_torch_cuda", None)
    assert B._device() == 1
    assert B._on(None, 1) == 0x77 and B._on(0x55, 1) == 0x55 and B._on(Stream(), 1) == 0x77


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
@pytest.mark.parametrize("name", ["spa_rope_config", "spa_paged_config"])
def test_config_layouts_match_the_header(tmp_path, name):
    """The ctypes mirrors have the C layout (size and every field offset)."""
    mirror = getattr(B, name)
    fields = [f for f, _ in mirror._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "spa.h"\nint main(void) {\n'
                   f'  printf("%zu", sizeof({name}));\n'
                   + "".join(f'  printf(" %zu", offsetof({name}, {f}));\n' for f in fields) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(mirror)] + [getattr(mirror, f).offset for f in fields]


def test_a_base_that_overflows_is_refused():
    """theta * factor^(rot_dim / (rot_dim - 2)) past 64 bits would leave every frequency but the first at 0."""
    ok = dict(scaling=B.SPA_ROPE_BASE, theta=1e4)
    r = B.spa_rope_create(B.make_rope_config(**ok, factor=1e290))
    f = np.array(B.spa_rope_inv_freq(r, 64))
    assert np.allclose(f, M.frequencies(128, theta=1e4, scaling="base", factor=1e290), rtol=1e-12, atol=0) and (f > 0).all()
    B.spa_rope_destroy(r)
    refused(B.SPA_ERR_INVALID_ARG, B.spa_rope_create, B.make_rope_config(**ok, factor=1e305))
