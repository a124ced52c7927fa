"""Refusals of the norms around a layer and of the attention behind a shared prompt that need
no GPU: the C ABI rejects bad arguments before it touches the device, the binding rejects bad
tensors before it calls the C ABI."""
import math

import pytest
import torch

import chunkwise_gated_delta_gdr_gb300 as gdr
from chunkwise_gated_delta_gdr_gb300 import build as gbuild

A = 1 << 20            # a fake, never dereferenced, aligned address
INV, UNS, ALI, WSP = (gdr.GDR_ERR_INVALID_ARG, gdr.GDR_ERR_UNSUPPORTED, gdr.GDR_ERR_ALIGNMENT,
                      gdr.GDR_ERR_WORKSPACE)
OK = gdr.GDR_OK


@pytest.fixture(scope="module")
def layers():
    gbuild.build()
    from chunkwise_gated_delta_gdr_gb300 import layers as mod
    mod._lib()
    return mod


# ------------------------------------------------------------------ gated norm
def gated_dims(mod, **kw):
    base = dict(B=2, T=3, H=4, D=128, in_dtype=1, out_dtype=1, activation=2, gate_first=0,
                weight_per_head=0, eps=1e-6, x_stride_b=3 * 512, x_stride_t=512, x_stride_h=128,
                gate_stride_b=3 * 512, gate_stride_t=512, gate_stride_h=128)
    base.update(kw)
    return mod.gdr_gated_dims(**base)


def gated(mod, d, x=A, z=A, w=A, y=A):
    return mod._lib().gdr_gated_norm(x, z, w, y, d, None)


def gated_bwd(mod, d, dy=A, x=A, z=A, w=A, dx=A, dz=A, dw=A, ws=A, n=1 << 40):
    return mod._lib().gdr_gated_norm_bwd(dy, x, z, w, dx, dz, dw, d, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(H=0), INV), (dict(D=0), INV),
    (dict(in_dtype=2), INV), (dict(out_dtype=-1), INV), (dict(activation=3), INV),
    (dict(activation=-1), INV), (dict(eps=0.0), INV), (dict(eps=-1.0), INV),
    (dict(eps=math.nan), INV), (dict(eps=math.inf), INV), (dict(x_stride_t=-1), INV),
    (dict(gate_stride_h=-1), INV), (dict(D=16385), UNS), (dict(B=1 << 16, T=1 << 16), UNS),
    (dict(H=1 << 21), UNS), (dict(H=1 << 20, D=2048), UNS)])
def test_gated_sizes(layers, kw, want):
    d = gated_dims(layers, **kw)
    assert gated(layers, d) == want and gated_bwd(layers, d) == want
    assert layers._lib().gdr_gated_norm_bwd_workspace_size(d) == 0


def test_gated_pointers(layers):
    d = gated_dims(layers)
    for name in ("x", "z", "y"):
        assert gated(layers, d, **{name: None}) == INV, name
    for name in ("dy", "x", "z", "dx", "dz"):
        assert gated_bwd(layers, d, **{name: None}) == INV, name
    for name, off in (("x", 1), ("z", 1), ("w", 4), ("y", 8)):
        assert gated(layers, d, **{name: A + off}) == ALI, name
    for name, off in (("dy", 2), ("x", 1), ("z", 1), ("w", 8), ("dx", 4), ("dz", 2), ("dw", 4),
                      ("ws", 16)):
        assert gated_bwd(layers, d, **{name: A + off}) == ALI, name
    need = layers._lib().gdr_gated_norm_bwd_workspace_size(d)
    assert need > 0
    assert gated_bwd(layers, d, ws=None) == WSP and gated_bwd(layers, d, n=need - 1) == WSP
    assert gated(layers, None) == INV
    assert gated(layers, gated_dims(layers, B=0), x=None, z=None, y=None) == OK
    assert gated_bwd(layers, gated_dims(layers, T=0), dy=None, x=None, z=None, dx=None, dz=None,
                     dw=None) == OK


# ------------------------------------------------------------------ residual add and norm
def residual_dims(mod, **kw):
    base = dict(B=2, T=3, D=128, residual_dtype=0, y_dtype=1, out_dtype=1, activation=1,
                post_norm=1, eps=1e-6, scale=1.0, residual_stride_b=384, residual_stride_t=128,
                y_stride_b=384, y_stride_t=128, gate_stride_b=384, gate_stride_t=128)
    base.update(kw)
    return mod.gdr_residual_dims(**base)


def residual(mod, d, r=A, y=A, z=A, w=A, wp=A, s=A, ro=A, out=A):
    return mod._lib().gdr_residual_norm(r, y, z, w, wp, s, ro, out, d, None)


def residual_bwd(mod, d, do=A, dro=A, r=A, y=A, z=A, w=A, wp=A, s=A, dr=A, dy=A, dz=A, dw=A,
                 dwp=A, ds=A, ws=A, n=1 << 40):
    return mod._lib().gdr_residual_norm_bwd(do, dro, r, y, z, w, wp, s, dr, dy, dz, dw, dwp, ds, d,
                                            ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(D=0), INV), (dict(residual_dtype=2), INV),
    (dict(y_dtype=2), INV), (dict(out_dtype=-1), INV), (dict(activation=9), INV),
    (dict(eps=0.0), INV), (dict(eps=math.nan), INV), (dict(scale=math.inf), INV),
    (dict(scale=math.nan), INV), (dict(residual_stride_t=-1), INV), (dict(y_stride_b=-1), INV),
    (dict(gate_stride_t=-1), INV), (dict(D=16385), UNS), (dict(B=1 << 16, T=1 << 16), UNS)])
def test_residual_sizes(layers, kw, want):
    d = residual_dims(layers, **kw)
    assert residual(layers, d) == want and residual_bwd(layers, d) == want
    assert layers._lib().gdr_residual_norm_bwd_workspace_size(d) == 0


def test_residual_pointers(layers):
    d, plain = residual_dims(layers), residual_dims(layers, post_norm=0)
    for name in ("r", "y", "ro", "out"):
        assert residual(layers, d, **{name: None}) == INV, name
    # Without y: no gate, post norm, scale per channel or result.
    alone = dict(y=None, z=None, wp=None, s=None, ro=None)
    for name in ("z", "wp", "s", "ro"):
        assert residual(layers, plain, **{**alone, name: A}) == INV, name
    assert residual(layers, d, **alone) == INV
    assert residual(layers, plain) == INV                  # post_weight without post_norm
    for name in ("do", "r", "y", "dr", "dy", "z", "dz"):
        assert residual_bwd(layers, d, **{name: None}) == INV, name
    assert residual_bwd(layers, d, s=None) == INV          # d_scale of a number
    assert residual_bwd(layers, plain, wp=None) == INV     # d_post_weight without post_norm
    for name, off in (("r", 2), ("y", 1), ("z", 1), ("w", 4), ("wp", 8), ("s", 4), ("ro", 8),
                      ("out", 2)):
        assert residual(layers, d, **{name: A + off}) == ALI, name
    for name, off in (("do", 2), ("dro", 4), ("r", 2), ("y", 1), ("z", 1), ("w", 4), ("wp", 4),
                      ("s", 4), ("dr", 8), ("dy", 8), ("dz", 8), ("dw", 4), ("dwp", 4), ("ds", 8),
                      ("ws", 16)):
        assert residual_bwd(layers, d, **{name: A + off}) == ALI, name
    need = layers._lib().gdr_residual_norm_bwd_workspace_size(d)
    assert residual_bwd(layers, d, ws=None) == WSP and residual_bwd(layers, d, n=need - 1) == WSP
    assert residual(layers, None) == INV
    assert residual(layers, residual_dims(layers, B=0), r=None, y=None, ro=None, out=None) == OK
    assert residual_bwd(layers, residual_dims(layers, T=0), dw=None, dwp=None, ds=None) == OK


# ------------------------------------------------------------------ shared prompt
def cache_dims(mod, **kw):
    base = dict(num_pages=9, page_size=16, HK=2, D=128, dtype=1, max_pages=4,
                page_stride=16 * 256, token_stride=256, head_stride=128)
    base.update(kw)
    return mod.gdr_paged_cache(**base)


def attn_dims(mod, **kw):
    base = dict(B=2, HQ=8, q_dtype=1, out_dtype=1, window=0, scale=0.1, q_stride_b=1024,
                q_stride_h=128)
    base.update(kw)
    return mod.gdr_attn_dims(**base)


def prefix(mod, d, c, pages=5, n=70, q=A, kc=A, vc=A, px=A, table=A, lens=A, out=A, lse=None, ws=A,
           size=1 << 50):
    return mod._lib().gdr_paged_prefix_attn(q, kc, vc, px, pages, n, table, lens, out, lse, d, c,
                                            ws, size, None)


@pytest.mark.parametrize("dk,ck,pk,want", [
    (dict(B=-1), {}, {}, INV), (dict(HQ=0), {}, {}, INV), (dict(HQ=7), {}, {}, INV),
    (dict(q_dtype=2), {}, {}, INV), (dict(out_dtype=2), {}, {}, INV), (dict(window=3), {}, {}, INV),
    (dict(scale=0.0), {}, {}, INV), (dict(scale=math.nan), {}, {}, INV),
    (dict(q_stride_h=-1), {}, {}, INV), ({}, dict(D=0), {}, INV), ({}, dict(D=300), {}, UNS),
    ({}, dict(page_size=0), {}, INV), ({}, dict(num_pages=-2), {}, INV),
    ({}, dict(head_stride=-1), {}, INV), ({}, {}, dict(pages=-1), INV), ({}, {}, dict(n=-1), INV),
    ({}, {}, dict(n=81), INV), ({}, {}, dict(pages=0, n=1), INV),
    ({}, {}, dict(pages=1 << 27, n=(1 << 30) + 1), UNS), (dict(B=1 << 28), {}, {}, UNS),
    (dict(B=1 << 26), {}, dict(pages=1 << 26, n=1 << 30), UNS)])
def test_prefix_sizes(layers, dk, ck, pk, want):
    d, c = attn_dims(layers, **dk), cache_dims(layers, **ck)
    assert prefix(layers, d, c, **pk) == want
    pk = {"pages": 5, "n": 70, **pk}
    assert layers._lib().gdr_paged_prefix_attn_workspace_size(d, c, pk["pages"], pk["n"]) == 0


def test_prefix_pointers(layers):
    d, c = attn_dims(layers), cache_dims(layers)
    for name in ("q", "kc", "vc", "px", "table", "lens", "out"):
        assert prefix(layers, d, c, **{name: None}) == INV, name
    for name, off in (("q", 1), ("kc", 8), ("vc", 8), ("px", 2), ("table", 2), ("lens", 1),
                      ("out", 2), ("lse", 4), ("ws", 128)):
        assert prefix(layers, d, c, **{name: A + off}) == ALI, name
    size = layers._lib().gdr_paged_prefix_attn_workspace_size
    need = size(d, c, 5, 70)
    assert need > size(d, c, 5, 0) > 0
    assert prefix(layers, d, c, ws=None) == WSP and prefix(layers, d, c, size=need - 1) == WSP
    assert prefix(layers, attn_dims(layers, B=0), c, q=None) == OK


@pytest.mark.parametrize("dtype,D", [(1, 128), (1, 256), (1, 40), (0, 128)])
def test_scratch_of_no_tokens(layers, dtype, D):
    """The binding asks for the scratch's size before the call: an empty batch has one, too,
    whichever kernels its sizes and types would take."""
    lib = layers._lib()
    c = cache_dims(layers, dtype=dtype, D=D, page_stride=32 * D, token_stride=2 * D, head_stride=D)
    for n in (0, 1, 70, 80):
        d = attn_dims(layers, B=0, q_dtype=dtype)
        assert lib.gdr_paged_prefix_attn_workspace_size(d, c, 5, n) > 0
        assert prefix(layers, d, c, n=n, q=None) == OK
    for kw in (dict(B=0), dict(T=0), dict(B=0, T=0)):
        for D in (D, D + 1, 5000):
            d = gated_dims(layers, in_dtype=dtype, D=D, **kw)
            assert lib.gdr_gated_norm_bwd_workspace_size(d) > 0
            d = residual_dims(layers, residual_dtype=dtype, D=D, **kw)
            assert lib.gdr_residual_norm_bwd_workspace_size(d) > 0


# ------------------------------------------------------------------ the binding
def test_binding_refuses_host_tensors(layers):
    x = torch.zeros(1, 4, 2, 8)
    r, i = x[:, :, 0], torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda: gdr.gated_norm(x, x), lambda: gdr.gated_norm_bwd(x, x, x),
                 lambda: gdr.residual_norm(r, r), lambda: gdr.residual_norm_bwd(r, r, r, r),
                 lambda: gdr.paged_prefix_attn(r, x, x, i[0], 1, i, i[0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_checks(layers):
    x = torch.zeros(2, 3, 4, 8)
    d, w, shape = layers._gated_dims(x, x, None, "silu", False, 1e-6, 0)
    assert (d.H, d.activation, d.weight_per_head, d.x_stride_t) == (4, 2, 0, 32)
    assert w is None and shape == (8,)
    assert layers._gated_dims(x, x, torch.ones(4, 8), "none", True, 1e-6, 0)[2] == (4, 8)
    for bad in (lambda: layers._gated_dims(x[0], x[0], None, "silu", False, 1e-6, 0),
                lambda: layers._gated_dims(x, x[:, :2], None, "silu", False, 1e-6, 0),
                lambda: layers._gated_dims(x, x, torch.ones(4), "silu", False, 1e-6, 0),
                lambda: layers._gated_dims(x, x, None, "tanh", False, 1e-6, 0),
                lambda: layers._gated_dims(x, x.transpose(2, 3), None, "silu", False, 1e-6, 0)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        layers._gated_dims(x, x.bfloat16(), None, "silu", False, 1e-6, 0)

    r = x[:, :, 0]
    base = dict(y=None, gate=None, weight=None, post_norm=False, post_weight=None, scale=1.0,
                activation="silu", eps=1e-6, out_code=0)
    d, ptrs = layers._residual_dims(r, **{**base, "y": r, "scale": 0.5})
    assert (d.D, d.scale, d.residual_stride_t, ptrs[4]) == (8, 0.5, 32, None)
    d, ptrs = layers._residual_dims(r, **{**base, "y": r, "scale": torch.ones(8)})
    assert d.scale == 1.0 and ptrs[4]
    for kw in (dict(gate=r), dict(post_norm=True), dict(scale=torch.ones(8)),
               dict(y=r, post_weight=torch.ones(8)), dict(y=r[:, :1]), dict(weight=torch.ones(7)),
               dict(y=r, scale=torch.ones(2)), dict(y=r, gate=r[:1])):
        with pytest.raises(ValueError):
            layers._residual_dims(r, **{**base, **kw})

    cpu, px = torch.device("cpu"), torch.zeros(5, dtype=torch.int32)
    assert layers._prefix_args(px, 7, cpu)[1:] == (5, 7)
    for args in ((px[None], 7), (px, -1), (px, 7.0), (px, 1 << 31), (px[::2], 7)):
        with pytest.raises(ValueError):
            layers._prefix_args(*args, cpu)
    with pytest.raises(TypeError):
        layers._prefix_args(px.long(), 7, cpu)
