"""Refusals of the layers' entry points that need no GPU: the C ABI rejects bad arguments
before it touches the device, the binding rejects bad tensors before it calls the C ABI."""
import math

import pytest
import torch

import chunkwise_gated_delta_gdr_gb300 as gdr
from chunkwise_gated_delta_gdr_gb300 import build as gbuild

A = 1 << 20            # a fake, never dereferenced, aligned address
INV, UNS, ALI, WSP = (gdr.GDR_ERR_INVALID_ARG, gdr.GDR_ERR_UNSUPPORTED, gdr.GDR_ERR_ALIGNMENT,
                      gdr.GDR_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def layers():
    gbuild.build()
    from chunkwise_gated_delta_gdr_gb300 import layers as mod
    mod._lib()
    return mod


def test_package_exports_every_entry_point(layers):
    for name in gdr.LAYERS:
        assert getattr(gdr, name) is getattr(layers, name)
    with pytest.raises(AttributeError):
        gdr.no_such_entry_point


# ------------------------------------------------------------------ scan
def scan_dims(mod, **kw):
    base = dict(B=2, T=64, D=32, x_dtype=1, g_dtype=0, h_dtype=1, gated_input=0,
                x_stride_b=64 * 32, x_stride_t=32, g_stride_b=64 * 32, g_stride_t=32,
                dh_stride_b=64 * 32, dh_stride_t=32)
    base.update(kw)
    return mod.gdr_scan_dims(**base)


BAD_SCAN = [(dict(B=-1), INV), (dict(T=-1), INV), (dict(D=0), INV), (dict(x_dtype=2), INV),
            (dict(g_dtype=-1), INV), (dict(h_dtype=7), INV), (dict(x_stride_t=-1), INV),
            (dict(g_stride_b=-8), INV), (dict(dh_stride_t=-2), INV), (dict(B=65536), UNS)]


def scan_fwd(mod, d, x=A, g=A, s0=None, h=A, sT=None, ck=None):
    return mod._lib().gdr_linear_scan_fwd(x, g, s0, h, sT, ck, d, None)


def scan_bwd(mod, d, dh=A, x=A, g=A, ck=A, df=None, dx=A, dg=A, d0=None):
    return mod._lib().gdr_linear_scan_bwd(dh, x, g, ck, df, dx, dg, d0, d, None)


@pytest.mark.parametrize("kw,want", BAD_SCAN)
def test_scan_sizes(layers, kw, want):
    d = scan_dims(layers, **kw)
    assert scan_fwd(layers, d) == want and scan_bwd(layers, d) == want
    assert layers._lib().gdr_linear_scan_checkpoints_size(d) == 0


def test_scan_pointers(layers):
    d = scan_dims(layers)
    for name in ("x", "g", "h"):
        assert scan_fwd(layers, d, **{name: None}) == INV
    for name in ("dh", "x", "g", "ck", "dx", "dg"):
        assert scan_bwd(layers, d, **{name: None}) == INV
    for name, off in (("x", 1), ("g", 2), ("h", 8), ("s0", 4), ("sT", 4), ("ck", 4)):
        assert scan_fwd(layers, d, **{name: A + off}) == ALI, name
    for name, off in (("dh", 1), ("x", 1), ("g", 2), ("ck", 8), ("df", 4), ("dx", 2), ("dg", 4),
                      ("d0", 4)):
        assert scan_bwd(layers, d, **{name: A + off}) == ALI, name
    assert scan_fwd(layers, None) == INV
    empty = scan_dims(layers, B=0)
    assert scan_fwd(layers, empty, x=None, g=None, h=None) == gdr.GDR_OK
    assert scan_bwd(layers, empty, dh=None, x=None, g=None, ck=None, dx=None, dg=None) == gdr.GDR_OK


def test_scan_checkpoints_size(layers):
    size = layers._lib().gdr_linear_scan_checkpoints_size
    assert size(scan_dims(layers)) == 2 * 1 * 32 * 4
    assert size(scan_dims(layers, T=65)) == 2 * 2 * 32 * 4
    assert size(scan_dims(layers, T=0)) == 0
    assert tuple(gdr.linear_scan_checkpoints(torch.empty(2, 65, 32)).shape) == (2, 2, 32)


# ------------------------------------------------------------------ norm and rotation
def qk_dims(mod, **kw):
    base = dict(B=2, T=3, HQ=4, HK=2, D=128, R=64, in_dtype=1, out_dtype=1, interleaved=0,
                position_bits=32, table_rows=10, eps=1e-6, q_stride_b=3 * 512, q_stride_t=512,
                q_stride_h=128, k_stride_b=3 * 256, k_stride_t=256, k_stride_h=128,
                v_stride_b=3 * 256, v_stride_t=256, v_stride_h=128)
    base.update(kw)
    return mod.gdr_qk_dims(**base)


def cache_dims(mod, **kw):
    base = dict(num_pages=9, page_size=16, HK=2, D=128, dtype=1, max_pages=4,
                page_stride=16 * 256, token_stride=256, head_stride=128)
    base.update(kw)
    return mod.gdr_paged_cache(**base)


def qk_fwd(mod, d, q=A, k=A, wq=A, wk=A, cos=A, sin=A, pos=A, qo=A, ko=A):
    return mod._lib().gdr_qk_norm_rope(q, k, wq, wk, cos, sin, pos, qo, ko, d, None)


def qk_bwd(mod, d, dqo=A, dko=A, q=A, k=A, wq=A, wk=A, cos=A, sin=A, pos=A, dq=A, dk=A, dwq=A,
           dwk=A, ws=A, n=1 << 40):
    return mod._lib().gdr_qk_norm_rope_bwd(dqo, dko, q, k, wq, wk, cos, sin, pos, dq, dk, dwq,
                                           dwk, d, ws, n, None)


def append(mod, d, c, q=A, k=A, v=A, cos=A, pos=A, qo=A, kc=A, vc=A, table=A):
    return mod._lib().gdr_qk_norm_rope_append(q, k, v, A, A, cos, A, pos, qo, kc, vc, table, d, c,
                                              None)


BAD_QK = [(dict(B=-1), INV), (dict(T=-1), INV), (dict(HQ=0), INV), (dict(HK=0), INV),
          (dict(D=0, R=0), INV), (dict(R=63), INV), (dict(R=130), INV), (dict(R=-2), INV),
          (dict(in_dtype=3), INV), (dict(out_dtype=-1), INV), (dict(position_bits=16), INV),
          (dict(table_rows=-1), INV), (dict(eps=0.0), INV), (dict(eps=math.nan), INV),
          (dict(eps=math.inf), INV), (dict(q_stride_t=-1), INV), (dict(k_stride_h=-1), INV),
          (dict(v_stride_b=-1), INV), (dict(D=257), UNS)]


@pytest.mark.parametrize("kw,want", BAD_QK)
def test_qk_sizes(layers, kw, want):
    d = qk_dims(layers, **kw)
    assert qk_fwd(layers, d) == want and qk_bwd(layers, d) == want
    assert append(layers, d, cache_dims(layers)) == want
    assert layers._lib().gdr_qk_norm_rope_bwd_workspace_size(d) == 0


def test_qk_pointers(layers):
    d = qk_dims(layers)
    for name in ("q", "k", "cos", "sin", "pos", "qo", "ko"):
        assert qk_fwd(layers, d, **{name: None}) == INV, name
    for name in ("q", "k", "cos", "sin", "pos", "dqo", "dko", "dq", "dk"):
        assert qk_bwd(layers, d, **{name: None}) == INV, name
    for name, off in (("q", 1), ("k", 1), ("wq", 4), ("wk", 8), ("cos", 4), ("sin", 4), ("pos", 2),
                      ("qo", 8), ("ko", 2)):
        assert qk_fwd(layers, d, **{name: A + off}) == ALI, name
    for name, off in (("dqo", 2), ("dko", 8), ("dq", 4), ("dk", 2), ("dwq", 4), ("dwk", 4),
                      ("ws", 16)):
        assert qk_bwd(layers, d, **{name: A + off}) == ALI, name
    need = layers._lib().gdr_qk_norm_rope_bwd_workspace_size(d)
    assert need > 0
    assert qk_bwd(layers, d, ws=None) == WSP and qk_bwd(layers, d, n=need - 1) == WSP
    empty = qk_dims(layers, B=0)
    assert qk_fwd(layers, empty, q=None, k=None, qo=None, ko=None) == gdr.GDR_OK


def test_append_arguments(layers):
    d, c = qk_dims(layers), cache_dims(layers)
    for name in ("q", "k", "v", "cos", "pos", "qo", "kc", "vc", "table"):
        assert append(layers, d, c, **{name: None}) == INV, name
    assert append(layers, qk_dims(layers, R=0), c, pos=None) == INV
    for name, off in (("v", 1), ("kc", 8), ("vc", 2), ("table", 2), ("qo", 4)):
        assert append(layers, d, c, **{name: A + off}) == ALI, name
    for kw in (dict(HK=3), dict(D=64), dict(num_pages=-1), dict(page_size=0), dict(max_pages=-1),
               dict(dtype=4), dict(token_stride=-1)):
        assert append(layers, d, cache_dims(layers, **kw)) == INV, kw


# ------------------------------------------------------------------ paged attention
def attn_dims(mod, **kw):
    base = dict(B=2, HQ=8, q_dtype=1, out_dtype=1, window=0, scale=0.1, q_stride_b=1024,
                q_stride_h=128)
    base.update(kw)
    return mod.gdr_attn_dims(**base)


def attn(mod, d, c, q=A, kc=A, vc=A, table=A, lens=A, out=A, lse=None, ws=A, n=1 << 40):
    return mod._lib().gdr_paged_decode_attn(q, kc, vc, table, lens, out, lse, d, c, ws, n, None)


BAD_ATTN = [(dict(B=-1), {}, INV), (dict(HQ=0), {}, INV), (dict(HQ=7), {}, INV),
            (dict(q_dtype=2), {}, INV), (dict(out_dtype=2), {}, INV), (dict(window=-1), {}, INV),
            (dict(scale=0.0), {}, INV), (dict(scale=math.nan), {}, INV),
            (dict(q_stride_h=-1), {}, INV), ({}, dict(D=0), INV), ({}, dict(D=300), UNS),
            ({}, dict(page_size=0), INV), ({}, dict(num_pages=-2), INV),
            ({}, dict(head_stride=-1), INV)]


@pytest.mark.parametrize("dk,ck,want", BAD_ATTN)
def test_attn_sizes(layers, dk, ck, want):
    d, c = attn_dims(layers, **dk), cache_dims(layers, **ck)
    assert attn(layers, d, c) == want
    assert layers._lib().gdr_paged_decode_attn_workspace_size(d, c) == 0


def test_attn_pointers(layers):
    d, c = attn_dims(layers), cache_dims(layers, max_pages=1000)
    for name in ("q", "kc", "vc", "table", "lens", "out"):
        assert attn(layers, d, c, **{name: None}) == INV, name
    for name, off in (("q", 1), ("kc", 8), ("vc", 8), ("table", 2), ("lens", 1), ("out", 2),
                      ("lse", 4), ("ws", 128)):
        assert attn(layers, d, c, **{name: A + off}) == ALI, name
    need = layers._lib().gdr_paged_decode_attn_workspace_size(d, c)
    assert attn(layers, d, c, ws=None) == WSP and attn(layers, d, c, n=need - 1) == WSP
    assert attn(layers, attn_dims(layers, B=0), c, q=None) == gdr.GDR_OK


# ------------------------------------------------------------------ the binding
def test_binding_refuses_host_tensors(layers):
    x = torch.zeros(1, 4, 8)
    for call in (lambda: gdr.linear_scan_fwd(x, x),
                 lambda: gdr.linear_scan_bwd(x, x, x, gdr.linear_scan_checkpoints(x)),
                 lambda: gdr.qk_norm_rope(x[..., None], x[..., None]),
                 lambda: gdr.paged_decode_attn(x, x[None], x[None],
                                               torch.zeros(1, 1, dtype=torch.int32),
                                               torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_checks_of_tensors(layers):
    cpu = torch.device("cpu")
    t = torch.zeros(2, 3, 8)
    assert layers._dense("t", None, (1,), cpu) is None
    assert layers._dense("t", t, (2, 3, 8), cpu) == t.data_ptr()
    with pytest.raises(ValueError, match="shape"):
        layers._dense("t", t, (2, 3, 9), cpu)
    with pytest.raises(ValueError, match="contiguous"):
        layers._dense("t", t.transpose(0, 1), (3, 2, 8), cpu)
    with pytest.raises(TypeError):
        layers._dense("t", t.double(), (2, 3, 8), cpu)
    layers._view("t", t[:, :, 1:5], (2, 3, 4), cpu)
    with pytest.raises(ValueError, match="last dimension"):
        layers._view("t", t.transpose(1, 2), (2, 8, 3), cpu)
    with pytest.raises(ValueError, match="shape"):
        layers._view("t", t, (2, 3, 4), cpu)
    with pytest.raises(TypeError):
        layers._code("t", t.half())


def test_binding_checks_of_the_caches(layers):
    cpu = torch.device("cpu")
    k = torch.zeros(5, 16, 2, 64)
    table = torch.zeros(3, 4, dtype=torch.int32)
    c = layers._cache_dims(k, k, table, 3, cpu)
    assert (c.num_pages, c.page_size, c.HK, c.D, c.max_pages) == (5, 16, 2, 64, 4)
    with pytest.raises(ValueError, match="one layout"):
        layers._cache_dims(k, torch.zeros(5, 2, 16, 64).transpose(1, 2), table, 3, cpu)
    with pytest.raises(ValueError, match="shape"):
        layers._cache_dims(k, k[:, :, :1], table, 3, cpu)
    with pytest.raises(TypeError):
        layers._cache_dims(k, k, table.long(), 3, cpu)
    q = torch.zeros(3, 4, 1, 64).squeeze(2)
    dims, _ = layers._attn_dims(q, k, k, table, None, 0, 0)
    assert dims.scale == pytest.approx(0.125)
    with pytest.raises(ValueError):
        layers._attn_dims(q[..., :32], k, k, table, None, 0, 0)


def test_binding_checks_of_the_rotation(layers):
    q, k = torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 2, 64)
    cos, pos = torch.zeros(10, 32), torch.zeros(2, 3, dtype=torch.int64)
    d = layers._qk_dims(q, k, None, cos, cos, pos, 1e-6, False, 0)
    assert (d.R, d.table_rows, d.position_bits, d.q_stride_h) == (64, 10, 64, 64)
    with pytest.raises(ValueError, match="together"):
        layers._qk_dims(q, k, None, cos, None, pos, 1e-6, False, 0)
    with pytest.raises(ValueError, match="positions"):
        layers._qk_dims(q, k, None, cos, cos, None, 1e-6, False, 0)
    with pytest.raises(TypeError):
        layers._qk_dims(q, k, None, cos, cos, pos.short(), 1e-6, False, 0)
    with pytest.raises(TypeError):
        layers._qk_dims(q, k.double(), None, cos, cos, pos, 1e-6, False, 0)
    with pytest.raises(ValueError, match="shape"):
        layers._qk_dims(q, k[:, :2], None, cos, cos, pos, 1e-6, False, 0)


def test_binding_refuses_sizes_past_32_bits(layers):
    for v in (1 << 31, 1 << 32, -(1 << 31) - 1):
        with pytest.raises(ValueError, match="out of range"):
            layers._struct(layers.gdr_scan_dims, 1, v, 1, 0, 0, 0, False, 0, 0, 0, 0, 0, 0)
    s = layers._struct(layers.gdr_scan_dims, 1, (1 << 31) - 1, 1, 0, 0, 0, True, 1 << 40, 0, 0, 0,
                       0, 0)
    assert s.T == (1 << 31) - 1 and s.gated_input == 1 and s.x_stride_b == 1 << 40
