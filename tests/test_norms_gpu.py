"""GPU numerics of the gated norm and of the residual add with norm, against plain 64-bit
implementations differentiated by autograd.

Tolerances. e = 2^-24 is fp32's rounding unit. A row's sum of squares is within 40 e of itself
(at most 32 terms in a row per thread, then a tree), its inverse root within 22 e; exp of an
argument |z| <= 8 is within 16 e, so that a gate is within 24 e and its slope, a product
g (1 - g) with 1 - g off by 24 e of 1, within 48 e of 1 (of 1 + |z| for z g). With a handful of products and the mean of D such terms a result is within 130 e = 8e-6 of the
size of the terms that make it up; 1e-5 is used. Those sizes are the ``size`` tensors below. A
weight gradient is a sum of such terms, in strands of at most 64 that meet in a tree: 1e-5 of
the sum of their sizes too. A bf16 result has to be the rounding of a value within that.
"""
import pytest
import torch

import chunkwise_gated_delta_gdr_gb300 as gdr

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"
TOL, EPS = 1e-5, 1e-6


def rnd(gen, *shape, dtype=F32):
    return torch.randn(*shape, generator=gen, dtype=F32).to(dtype).to(DEV)


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


def check(got, ref, size, tol=TOL):
    """got is (the rounding of) a value within tol * size of ref, element by element."""
    assert got.shape == ref.shape
    lo, hi = ((ref + s * tol * size).to(got.dtype).double() for s in (-1, 1))
    over = torch.maximum(got.double() - hi, lo - got.double())
    assert not torch.isnan(over).any()
    assert over.max().item() <= 0, f"exceeds its bound by {over.max().item():.3e}"


def act(z, kind):
    g = torch.sigmoid(z)
    return z if kind == "none" else g if kind == "sigmoid" else z * g


def rms(x):
    return torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS)


# ------------------------------------------------------------------ gated norm
def gated_ref(x, z, w, d, kind, first):
    """(y, dx, dz, dw) and their sizes."""
    x, z = (t.double().requires_grad_(True) for t in (x, z))
    shape = x.shape[-1:] if w is None else w.shape
    w = (torch.ones(shape, dtype=torch.float64, device=DEV) if w is None else w.double())
    w.requires_grad_(True)
    a = act(z, kind)
    y = x * a / rms(x * a) * w if first else x / rms(x) * w * a
    d = d.double()
    grads = torch.autograd.grad(y, (x, z, w), d)
    with torch.no_grad():
        big = (1 + z.abs()) if kind != "sigmoid" else torch.ones_like(z)   # of a' and of a
        v = x * a if first else x
        u, c = (v / rms(v)).abs(), (d * w).abs() * (1 if first else a.abs())
        dv = (c + u * (c * u).mean(-1, keepdim=True)) / rms(v)
        sizes = [y.abs() + 1e-30, dv * (a.abs() if first else 1),
                 (dv * x.abs() if first else (d * w).abs() * u) * big,
                 (d.abs() * u * (1 if first else a.abs())).sum((0, 1) if w.dim() == 2 else (0, 1, 2))]
    return (y.detach(), *grads), [s + 1e-30 for s in sizes]


def gated_check(x, z, w, d, kind="silu", first=False):
    kw = dict(activation=kind, gate_first=first, eps=EPS)
    y = gdr.gated_norm(x, z, w, **kw)
    got = (y, *gdr.gated_norm_bwd(d, x, z, w, **kw))
    for g, r, s in zip(got, *gated_ref(x, z, w, d, kind, first)):
        check(g, r, s)
    return got


def gated_inputs(B, T, H, D, dtype=F32, seed=0, weight="one"):
    gen = gen_of(seed)
    x, z, d = (rnd(gen, B, T, H, D, dtype=dtype) for _ in range(3))
    w = None if weight == "none" else 1 + 0.2 * rnd(gen, *((H, D) if weight == "head" else (D,)))
    return x, z.mul(1.5), w, d


GATED = [(1, 1, 1, 1), (2, 3, 2, 7), (3, 5, 2, 64), (2, 7, 3, 80), (1, 33, 4, 128), (2, 3, 2, 256),
         (1, 5, 2, 257), (1, 6, 3, 264), (2, 1, 1, 1536), (1, 3, 2, 4096), (1, 2, 1, 8200),
         (1, 1, 2, 9001), (1, 2, 1, 16384)]


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", GATED)
def test_gated_shapes(shape, dtype, first):
    for i, (kind, weight) in enumerate([("silu", "one"), ("sigmoid", "head"), ("none", "none")]):
        gated_check(*gated_inputs(*shape, dtype=dtype, seed=i, weight=weight), kind, first)


@pytest.mark.parametrize("weight", ["one", "head"])
@pytest.mark.parametrize("shape", [(1, 20000, 1, 8), (2, 3000, 3, 64), (1, 5001, 5, 96),
                                   (3, 701, 7, 200), (2, 600, 2, 1024), (1, 1500, 3, 33),
                                   (1, 400, 1, 8192), (1, 310, 1, 16000)])
def test_gated_many_rows_per_group(shape, weight):
    gated_check(*gated_inputs(*shape, dtype=BF, seed=3, weight=weight), "silu", False)


def test_gated_more_heads_than_groups():
    gated_check(*gated_inputs(1, 2, 9001, 64, seed=4, weight="head"), "silu", False)
    gated_check(*gated_inputs(1, 1, 1300, 300, seed=4, weight="one"), "sigmoid", True)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_gated_views(offset, dtype):
    """Slices of a projection, transposed layouts and a broadcast gate."""
    gen, B, T, H, D = gen_of(5), 2, 9, 3, 64
    wide = rnd(gen, B, T, 2 * H * D + 16, dtype=dtype)
    x = wide[..., offset:offset + H * D].unflatten(-1, (H, D))
    z = wide[..., H * D + offset:2 * H * D + offset].unflatten(-1, (H, D))
    w, d = 1 + 0.2 * rnd(gen, D), rnd(gen, B, T, H, D, dtype=dtype)
    gated_check(x, z, w, d)
    gated_check(rnd(gen, H, T, B, D, dtype=dtype).permute(2, 1, 0, 3), z, w, d, "sigmoid", True)
    gated_check(x, rnd(gen, B, 1, 1, D, dtype=dtype).expand(B, T, H, D), w, d)


@pytest.mark.parametrize("dtype,out", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("D", [128, 129, 1040])
def test_gated_other_output_type(D, dtype, out):
    x, z, w, d = gated_inputs(2, 5, 3, D, dtype=dtype, seed=6)
    d = d.to(out)
    y = gdr.gated_norm(x, z, w, out_dtype=out)
    got = (y, *gdr.gated_norm_bwd(d, x, z, w))
    assert y.dtype == out and got[1].dtype == dtype
    for g, r, s in zip(got, *gated_ref(x, z, w, d, "silu", False)):
        check(g, r, s)


@pytest.mark.parametrize("D", [64, 513])
def test_gated_zero_rows_large_gates_and_nan(D):
    """Rows of zeros, gates that are fully open or shut, and a NaN that stays in its row."""
    x, z, w, d = gated_inputs(1, 6, 2, D, seed=7)
    x[0, 1] = 0
    z[0, 2], z[0, 3] = 60.0, -60.0
    for first in (False, True):
        y = gdr.gated_norm(x, z, w, gate_first=first)
        dx, dz, dw = gdr.gated_norm_bwd(d, x, z, w, gate_first=first)
        assert all(torch.isfinite(t).all() for t in (y, dx, dz, dw))
        assert (y[0, 1] == 0).all()
    bad = x.clone()
    bad[0, 4, 1, 0] = float("nan")
    again = gdr.gated_norm(bad, z, w, gate_first=True)
    keep = torch.ones(1, 6, 2, dtype=torch.bool, device=DEV)
    keep[0, 4, 1] = False
    assert torch.equal(again[keep], y[keep]) and torch.isnan(again[~keep]).all()


def test_gated_gradient_against_differences():
    """Central differences of the forward call along random directions. The call's fp32 error
    is 1e-5 of a sum of n terms of size 1, random in sign: 1e-5 sqrt(n) / (2 h) of a
    derivative, h = 1e-2, and the third derivative adds about h^2 sqrt(n)."""
    x, z, w, d = gated_inputs(2, 9, 3, 64, seed=8)
    gen = gen_of(9)
    for first in (False, True):
        kw = dict(activation="silu", gate_first=first)
        grads = gdr.gated_norm_bwd(d, x, z, w, **kw)
        for i, g in enumerate(grads):
            v, h = rnd(gen, *g.shape), 1e-2
            at = [[t + s * h * v if j == i else t for j, t in enumerate((x, z, w))] for s in (1, -1)]
            hi, lo = ((gdr.gated_norm(*p, **kw).double() * d.double()).sum() for p in at)
            n = x.numel() ** 0.5
            assert abs((hi - lo) / (2 * h) - (g.double() * v.double()).sum()) <= n * (5e-4 + 1e-3)


# ------------------------------------------------------------------ residual add and norm
def residual_ref(r, y, w, z, wp, s, d, dr, kind, post, stored):
    """(out, r') and, from the residual as it was stored, every gradient; and their sizes."""
    D = r.shape[-1]
    ones = torch.ones(D, dtype=torch.float64, device=DEV)
    leaf = lambda t: t.detach().double().requires_grad_(True)  # noqa: E731
    w = leaf(ones if w is None else w)
    res = r.double()
    parts = {}
    if y is not None:
        y, wp = leaf(y), leaf(ones if wp is None else wp)
        z = None if z is None else leaf(z)
        s = leaf(s if isinstance(s, torch.Tensor) else ones * s)
        p = y / rms(y) * wp if post else y
        a = torch.ones_like(y) if z is None else act(z, kind)
        t = s * a * p
        res = res + t.detach()
    out = res / rms(res) * w.detach()
    x = leaf(stored)
    g, dw = torch.autograd.grad(x / rms(x) * w, (x, w), d.double())
    g = g + (0 if dr is None else dr.double())
    with torch.no_grad():
        u, c = (x / rms(x)).abs(), (d.double() * w).abs()
        gs = (c + u * (c * u).mean(-1, keepdim=True)) / rms(x) + (0 if dr is None else dr.abs())
        size_r = r.double().abs() + (t.abs() if y is not None else 0)
        # An error of the sum shows in out at the same relative size, and through the mean.
        parts["out"] = (out, (size_r + res.abs()) / rms(res) * w.abs())
        parts["dr"] = (g, gs)
        parts["dw"] = (dw, (d.double().abs() * u).sum((0, 1)))
        if y is not None:
            parts["r"] = (res, size_r)
    if y is not None:
        want = [n for n in (y, z, wp if post else None, s) if n is not None]
        got = dict(zip(map(id, want), torch.autograd.grad(t, want, g)))
        with torch.no_grad():
            dp, uy = gs * (s * a).abs(), (y / rms(y)).abs()
            q = dp * wp.abs()
            size_y = (q + uy * (q * uy).mean(-1, keepdim=True)) / rms(y) if post else dp
            parts["dy"] = (got[id(y)], size_y)
            if z is not None:
                parts["dz"] = (got[id(z)], gs * (s * p).abs() * (1 + z.abs()))
            if post:
                parts["dwp"] = (got[id(wp)], (dp * uy).sum((0, 1)))
            parts["ds"] = (got[id(s)], (gs * (a * p).abs()).sum((0, 1)))
    return parts


def residual_check(r, y, w=None, z=None, wp=None, s=1.0, d=None, dr=None, kind="sigmoid",
                   post=False, out_dtype=None):
    kw = dict(gate=z, activation=kind, post_norm=post, post_weight=wp, scale=s, eps=EPS)
    out, res = gdr.residual_norm(r, y, w, out_dtype=out_dtype, **kw)
    d = d.to(out.dtype)
    grads = gdr.residual_norm_bwd(d, dr, res, y, w, **kw)
    ref = residual_ref(r, y, w, z, wp, s, d, dr, kind, post, res)
    got = dict(zip(("dr", "dy", "dz", "dw", "dwp", "ds"), grads), out=out)
    if y is not None:
        got["r"] = res
    else:
        assert res is r
    vector = isinstance(s, torch.Tensor)
    for name, g in got.items():
        if g is None:
            assert name not in ref or (name == "ds" and not vector)
        else:
            check(g, *[t + (1e-30 if i else 0) for i, t in enumerate(ref[name])])
    return got


def residual_inputs(B, T, D, rt=F32, yt=F32, seed=0):
    gen = gen_of(seed)
    r = rnd(gen, B, T, D).mul_(3).to(rt)
    y, z, d = (rnd(gen, B, T, D, dtype=yt) for _ in range(3))
    w, wp, s = (1 + 0.2 * rnd(gen, D) for _ in range(3))
    return r, y, z, d, rnd(gen, B, T, D, dtype=rt), w, wp, s * 0.5


RESIDUAL = [(1, 1, 1), (2, 3, 7), (3, 5, 64), (2, 1, 200), (1, 9, 777), (2, 2, 1536), (1, 3, 2048),
            (1, 2, 4096), (1, 2, 8192), (1, 2, 8200), (1, 1, 16384), (1, 1, 12345)]


@pytest.mark.parametrize("rt,yt", [(F32, F32), (BF, BF), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("shape", RESIDUAL)
def test_residual_shapes(shape, rt, yt):
    r, y, z, d, dr, w, wp, s = residual_inputs(*shape, rt, yt)
    residual_check(r, y, w, d=d, dr=dr)
    residual_check(r, y, w, z, wp, s, d, dr, "silu", True)
    residual_check(r, y, None, z, None, 0.25, d, None, "sigmoid", False)
    residual_check(r, None, w, d=d, dr=dr)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "none", "sigmoid", "silu"])
@pytest.mark.parametrize("scale", [1.0, -0.5, "vector"])
def test_residual_every_form(scale, gate, post):
    r, y, z, d, dr, w, wp, s = residual_inputs(2, 5, 320, F32, BF, seed=1)
    scale = s if scale == "vector" else scale
    for weight in (None, wp) if post else (None,):
        residual_check(r, y, w, z if gate else None, weight, scale, d, dr, gate or "sigmoid", post)


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("shape,rt,yt", [((2, 5000, 64), F32, BF), ((1, 3001, 96), BF, BF),
                                         ((3, 700, 1000), F32, F32), ((1, 900, 777), BF, BF),
                                         ((2, 600, 4096), BF, BF), ((1, 400, 8192), F32, F32),
                                         ((1, 330, 9000), F32, BF), ((1, 400, 4097), F32, F32)])
def test_residual_many_rows_per_block(shape, rt, yt, full):
    r, y, z, d, dr, w, wp, s = residual_inputs(*shape, rt, yt, seed=2)
    if full:
        residual_check(r, y, w, z, wp, s, d, dr, "silu", True)
    else:
        residual_check(r, y, w, d=d, dr=dr, s=0.5)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_residual_views(offset, dtype):
    gen, B, T, D = gen_of(3), 2, 9, 96
    wide = rnd(gen, B, T, 3 * D + 16, dtype=dtype)
    r, y, z = (wide[..., i * D + offset:(i + 1) * D + offset] for i in range(3))
    d, dr, w = rnd(gen, B, T, D, dtype=dtype), rnd(gen, B, T, D, dtype=dtype), rnd(gen, D)
    residual_check(r, y, w, z, None, 1.0, d, dr, "silu", True)
    turned = rnd(gen, T, B, D, dtype=dtype).transpose(0, 1)
    residual_check(turned, y, w, d=d, dr=dr)
    residual_check(r, y, w, rnd(gen, B, 1, D, dtype=dtype).expand(B, T, D), None, 1.0, d, dr,
                   "none")


@pytest.mark.parametrize("D", [256, 250])
def test_residual_output_type(D):
    r, y, _, d, dr, w, _, _ = residual_inputs(2, 4, D, F32, BF, seed=4)
    for out in (BF, F32):
        got = residual_check(r, y, w, d=d, dr=dr, out_dtype=out)
        assert got["out"].dtype == out and got["r"].dtype == F32
        assert residual_check(r, None, w, d=d, dr=dr, out_dtype=out)["out"].dtype == out


@pytest.mark.parametrize("D", [128, 131, 4096])
@pytest.mark.parametrize("rt", [F32, BF])
def test_residual_in_place(D, rt):
    r, y, z, _, _, w, wp, s = residual_inputs(2, 600, D, rt, BF, seed=5)
    kw = dict(gate=z, post_norm=True, post_weight=wp, scale=s)
    out, res = gdr.residual_norm(r, y, w, **kw)
    mine = r.clone()
    out2, res2 = gdr.residual_norm(mine, y, w, **kw, residual_out=mine)
    assert res2 is mine and torch.equal(out, out2) and torch.equal(res, mine)


def test_residual_gradient_against_differences():
    """As for the gated norm; a loss of both results."""
    r, y, z, d, dr, w, wp, s = residual_inputs(2, 9, 128, seed=6)
    gen = gen_of(10)
    ins = [r, y, z, w, wp, s]

    def call(r, y, z, w, wp, s):
        return gdr.residual_norm(r, y, w, gate=z, activation="silu", post_norm=True, post_weight=wp,
                                 scale=s)

    def loss(*ins):
        out, res = call(*ins)
        return (out.double() * d.double()).sum() + (res.double() * dr.double()).sum()

    grads = gdr.residual_norm_bwd(d, dr, call(*ins)[1], y, w, gate=z, activation="silu",
                                  post_norm=True, post_weight=wp, scale=s)
    for i, g in enumerate(grads):
        v, h = rnd(gen, *g.shape), 1e-2
        at = [[t + k * h * v if j == i else t for j, t in enumerate(ins)] for k in (1, -1)]
        slope = (loss(*at[0]) - loss(*at[1])) / (2 * h)
        n = r.numel() ** 0.5
        assert abs(slope - (g.double() * v.double()).sum()) <= n * (3 * 5e-4 + 3e-3)


# ------------------------------------------------------------------ both
def calls(seed=0):
    x, z, w, d = gated_inputs(2, 40, 4, 128, BF, seed)
    r, y, g, do, dr, wr, wp, s = residual_inputs(2, 40, 512, F32, BF, seed)
    kw = dict(gate=g, post_norm=True, post_weight=wp, scale=s)

    def run(**stream):
        a = gdr.gated_norm(x, z, w, **stream)
        b = gdr.gated_norm_bwd(d, x, z, w, **stream)
        c = gdr.residual_norm(r, y, wr, **kw, **stream)
        e = gdr.residual_norm_bwd(do, dr, c[1], y, wr, **kw, **stream)
        return (a, *b, *c, *e)

    return run, (x, z, d, r, y, g, do, dr)


def test_runs_are_equal():
    run, _ = calls()
    for a, b in zip(run(), run()):
        assert torch.equal(a, b)


def test_no_tokens():
    for shape in ((0, 3, 2, 64), (2, 0, 2, 64)):
        x = torch.empty(*shape, device=DEV)
        y = gdr.gated_norm(x, x)
        dx, dz, dw = gdr.gated_norm_bwd(y, x, x)
        assert y.shape == dx.shape == dz.shape == x.shape and (dw == 0).all()
        r = x[:, :, 0]
        out, res = gdr.residual_norm(r, r.clone(), post_norm=True, scale=torch.ones(64, device=DEV))
        grads = gdr.residual_norm_bwd(out, None, res, r.clone(), post_norm=True,
                                      scale=torch.ones(64, device=DEV))
        assert out.shape == r.shape and all((g == 0).all() for g in grads[3:])


def test_another_stream():
    run, _ = calls(1)
    want = run()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        inside = run()
    named = run(stream=stream)
    stream.synchronize()
    for a, b, c in zip(want, inside, named):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_capture_and_replay_on_new_inputs():
    run, ins = calls(2)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    gen = gen_of(11)
    for _ in range(2):
        for t in ins:
            t.copy_(rnd(gen, *t.shape))
        graph.replay()
        for a, b in zip(got, run()):
            assert torch.equal(a, b)


def test_compiled_and_python_calls_agree(monkeypatch):
    from chunkwise_gated_delta_gdr_gb300 import layers
    run, _ = calls(3)
    assert layers._host is not None
    want = run()
    monkeypatch.setattr(layers, "_host", None)
    for a, b in zip(want, run()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("compiled", [True, False])
def test_refusals_on_the_gpu(compiled, monkeypatch):
    from chunkwise_gated_delta_gdr_gb300 import layers
    if not compiled:
        monkeypatch.setattr(layers, "_host", None)
    x = torch.randn(2, 3, 2, 64, device=DEV)
    r = x[:, :, 0].contiguous()
    w = torch.ones(64, device=DEV)
    for error, call in [
            (ValueError, lambda: gdr.gated_norm(x, x, activation="relu")),
            (ValueError, lambda: gdr.gated_norm(x, x[:, :2])),
            (ValueError, lambda: gdr.gated_norm(x, x.cpu())),
            (ValueError, lambda: gdr.gated_norm(x, x, w[:32])),
            (ValueError, lambda: gdr.gated_norm(r, r)),
            (TypeError, lambda: gdr.gated_norm(x, x.bfloat16())),
            (TypeError, lambda: gdr.gated_norm(x.half(), x.half())),
            (TypeError, lambda: gdr.gated_norm(x, x, w.bfloat16())),
            (TypeError, lambda: gdr.gated_norm(x, x, out_dtype=BF, out=x.clone())),
            (gdr.GdrError, lambda: gdr.gated_norm(x, x, eps=0.0)),
            (ValueError, lambda: gdr.gated_norm(x.transpose(2, 3), x.transpose(2, 3))),
            (ValueError, lambda: gdr.gated_norm_bwd(x.transpose(0, 1), x, x)),
            (gdr.GdrError, lambda: gdr.gated_norm_bwd(x, x, x, workspace=torch.empty(
                16, dtype=torch.uint8, device=DEV))),
            (ValueError, lambda: gdr.residual_norm(x, x)),
            (ValueError, lambda: gdr.residual_norm(r, None, post_norm=True)),
            (ValueError, lambda: gdr.residual_norm(r, None, gate=r)),
            (ValueError, lambda: gdr.residual_norm(r, None, scale=w)),
            (ValueError, lambda: gdr.residual_norm(r, None, residual_out=r.clone())),
            (ValueError, lambda: gdr.residual_norm(r, r, post_weight=w)),
            (TypeError, lambda: gdr.residual_norm(r, r, gate=r.bfloat16())),
            (ValueError, lambda: gdr.residual_norm(r, r, scale=w[:3])),
            (gdr.GdrError, lambda: gdr.residual_norm(r, r, scale=float("inf"))),
            (ValueError, lambda: gdr.residual_norm_bwd(r, r, r, d_gate=r)),
            (TypeError, lambda: gdr.residual_norm_bwd(r, r.bfloat16(), r, r)),
            (gdr.GdrError, lambda: gdr.residual_norm(torch.empty(1, 1, 16385, device=DEV)))]:
        with pytest.raises(error):
            call()
    gdr.gated_norm(x, x)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rt,yt", [(F32, F32), (BF, BF), (F32, BF)])
@pytest.mark.parametrize("D", [9, 65, 777, 1001, 3190, 6547, 8185, 8186])
def test_residual_odd_rows(D, rt, yt):
    """Rows that start anywhere against 16 bytes, more of them than blocks; a neighbour's NaN
    next to a row's ends stays out of it, and rows next to a slice are left as they were."""
    T = 1300 if D < 1000 else 700
    r, y, z, d, dr, w, wp, s = residual_inputs(1, T, D, rt, yt, seed=12)
    residual_check(r, y, w, z, wp, s, d, dr, "silu", True)
    residual_check(r, y, w, d=d, dr=dr, s=0.5)
    out, res = gdr.residual_norm(r, y, w)
    bad = y.clone()
    bad[0, 3::7] = float("nan")
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[3::7] = False
    out2, res2 = gdr.residual_norm(r, bad, w)
    assert torch.equal(out2[0, keep], out[0, keep]) and torch.isnan(out2[0, ~keep]).all()
    pool = torch.full((T + 2, D), 7.0, dtype=rt, device=DEV)
    row = 16 // torch.finfo(rt).bits * 8          # a slice that starts on 16 bytes
    mine = pool.view(-1)[8 * row:8 * row + 8 * D].view(1, 8, D)
    gdr.residual_norm(r[:, :8], y[:, :8], w, residual_out=mine)
    assert torch.equal(mine, res[:, :8])
    flat = pool.view(-1)
    assert (flat[:8 * row] == 7).all() and (flat[8 * row + 8 * D:] == 7).all()


@pytest.mark.parametrize("weight", ["one", "head"])
@pytest.mark.parametrize("shape", [(2, 900, 3, 9), (1, 1100, 5, 57), (3, 701, 7, 100), (2, 500, 4, 173),
                                   (2, 700, 3, 250), (1, 900, 2, 335), (1, 30, 2, 8185)])
def test_gated_odd_rows(shape, weight):
    for dtype in (BF, F32):
        x, z, w, d = gated_inputs(*shape, dtype=dtype, seed=13, weight=weight)
        gated_check(x, z, w, d, "silu", False)
        gated_check(x, z, w, d, "sigmoid", True)


def test_odd_rows_of_views_with_even_steps():
    """Views whose strides differ from the dense ones by multiples of 8 elements."""
    gen, B, T, H, D = gen_of(14), 2, 40, 3, 77
    for dtype in (BF, F32):
        x = rnd(gen, B, T, H * D + 16, dtype=dtype)[..., :H * D].unflatten(-1, (H, D))
        z = rnd(gen, B, T + 8, H * D, dtype=dtype)[:, :T].unflatten(-1, (H, D))
        w, d = rnd(gen, H, D), rnd(gen, B, T, H, D, dtype=dtype)
        gated_check(x, z, w, d)
        residual_check(x[:, :, 0], z[:, :, 0], w[0].contiguous(), d=d[:, :, 0].contiguous(),
                       dr=d[:, :, 1].contiguous())


@pytest.mark.parametrize("D", [5, 8, 57, 58, 64, 72, 100, 128, 200, 249, 250, 256, 264])
@pytest.mark.parametrize("rt,yt", [(F32, BF), (F32, F32)])
def test_residual_short_rows(D, rt, yt):
    """Several rows per warp: more of them than groups, and too few for one block."""
    for T in (3, 20011 if D < 100 else 9001):
        r, y, z, d, dr, w, wp, s = residual_inputs(1, T, D, rt, yt, seed=15)
        residual_check(r, y, w, z, wp, s, d, dr, "silu", True)
        residual_check(r, y, w, d=d, dr=dr, s=0.5)
    wide = torch.cat([r, r], -1)                 # rows that are not aligned at all
    residual_check(wide[..., 1:D + 1], y, w, d=d, dr=dr)


@pytest.mark.parametrize("dtype,out", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("D", [24, 100, 200, 333, 400])
def test_gated_other_output_type_of_short_rows(D, dtype, out):
    x, z, w, d = gated_inputs(2, 300, 3, D, dtype=dtype, seed=16)
    y = gdr.gated_norm(x, z, w, out_dtype=out)
    got = (y, *gdr.gated_norm_bwd(d.to(out), x, z, w))
    for g, r, s in zip(got, *gated_ref(x, z, w, d.to(out), "silu", False)):
        check(g, r, s)


def test_single_tokens_of_a_batch():
    """T = 1 with batch rows any stride apart, and with one row for all of them."""
    gen, B, H, D = gen_of(17), 300, 2, 72
    for dtype in (BF, F32):
        x = rnd(gen, B, 5, H, D, dtype=dtype)[:, 2:3]
        z = rnd(gen, 1, 1, H, D, dtype=dtype).expand(B, 1, H, D)
        w, d = rnd(gen, D), rnd(gen, B, 1, H, D, dtype=dtype)
        gated_check(x, z, w, d)
        residual_check(x[:, :, 0], z[:, :, 1], w, d=d[:, :, 0].contiguous(),
                       dr=d[:, :, 1].contiguous())


@pytest.mark.parametrize("D", [64, 513, 1024])
def test_infinite_gate_without_activation(D):
    """Its slope is 1, so its gradient d u w does not depend on it: with one row's gates infinite
    every row's is what it is with finite ones, bit by bit."""
    x, z, w, d = gated_inputs(1, 3, 2, D, seed=60)
    _, want, _ = gdr.gated_norm_bwd(d, x, z, w, activation="none")
    z[0, 1, 1] = float("inf")
    _, got, _ = gdr.gated_norm_bwd(d, x, z, w, activation="none")
    assert torch.equal(got, want)
    r, y, z, d, dr, w, _, _ = residual_inputs(1, 3, D, seed=61)
    kw = dict(activation="none", scale=0.5)
    want = gdr.residual_norm_bwd(d, dr, r, y, w, gate=z, **kw)[2]
    z[0, 1] = float("-inf")
    assert torch.equal(gdr.residual_norm_bwd(d, dr, r, y, w, gate=z, **kw)[2], want)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D", [301, 2047, 2049, 4075, 4097, 8191, 9000])
def test_long_rows_from_anywhere(D, dtype):
    """Slices that start one element behind a boundary: no row is aligned."""
    gen, B, T, H = gen_of(70), 2, 5, 2
    x, z, w, d = gated_inputs(B, T, H, D, dtype=dtype, seed=71, weight="head")
    wide = rnd(gen, B, T, 2 * H * D + 3, dtype=dtype)
    gated_check(x, wide[..., 1:1 + H * D].unflatten(-1, (H, D)), w, d, "silu", False)
    gated_check(wide[..., 1 + H * D:1 + 2 * H * D].unflatten(-1, (H, D)), z, w, d, "sigmoid", True)
    r, y, _, d, dr, w, wp, s = residual_inputs(B, T, D, rt=F32, yt=dtype, seed=72)
    gate = wide[..., 1:1 + D]
    residual_check(r, y, w, gate, wp, s, d, dr, "silu", True)
    residual_check(r, wide[..., 1:1 + D], w, d=d, dr=dr)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D", [40, 64, 513, 1024, 4096])
def test_infinite_gate_before_the_norm(D, dtype):
    """An infinite gate without activation makes its row's root mean square infinite: that channel
    is inf / inf, the row's others are 0, its gradients are NaN; every other row, and the weights'
    gradients of the other channels, have the bits that they have without it."""
    x, z, w, d = gated_inputs(2, 3, 2, D, dtype=dtype, seed=62)
    x[1, 1, 0, 7] = 2.0
    kw = dict(activation="none", gate_first=True)
    without = d.clone()
    without[1, 1, 0] = 0
    y = gdr.gated_norm(x, z, w, **kw)
    dx, dz, _ = gdr.gated_norm_bwd(d, x, z, w, **kw)
    dw = gdr.gated_norm_bwd(without, x, z, w, **kw)[2]
    z[1, 1, 0, 7] = float("inf")
    y2 = gdr.gated_norm(x, z, w, **kw)
    dx2, dz2, dw2 = gdr.gated_norm_bwd(d, x, z, w, **kw)
    keep = torch.ones(2, 3, 2, dtype=torch.bool, device=DEV)
    keep[1, 1, 0] = False
    for a, b in ((y, y2), (dx, dx2), (dz, dz2)):
        assert torch.equal(a[keep], b[keep])
    others = torch.arange(D, device=DEV) != 7
    assert torch.isnan(y2[1, 1, 0, 7]) and (y2[1, 1, 0][others] == 0).all()
    assert torch.isnan(dx2[1, 1, 0]).all() and torch.isnan(dz2[1, 1, 0]).all()
    assert torch.isnan(dw2[7]) and torch.equal(dw2[others], dw[others])


def _many(rows, D, seed):
    """rows x D elements, more than 2^31, bf16; the last ones are compared."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(rows, D, generator=gen, dtype=BF, device=DEV)


@pytest.mark.parametrize("H,D,offset", [(8, 128, 0), (2, 1000, 0), (3, 1001, 0), (2, 700, 1)])
def test_gated_offsets_beyond_32_bits(H, D, offset):
    """Tensors of more than 2^31 elements: rows at the end have the bits that they have in a call
    of their own, and the weights' gradient, from those rows alone, is the same sum."""
    T, n = (1 << 31) // (H * D) + 40, 9
    x, z = (_many(T, H * D + offset, seed)[:, offset:].view(1, T, H, D) for seed in (1, 2))
    w = 1 + 0.2 * rnd(gen_of(3), D)
    d = torch.zeros(1, T, H, D, dtype=BF, device=DEV)
    d[:, -n:] = rnd(gen_of(4), 1, n, H, D, dtype=BF)
    small = [t[:, -n:].clone() for t in (x, z, d)]
    assert torch.equal(gdr.gated_norm(x, z, w)[:, -n:], gdr.gated_norm(*small[:2], w))
    dx, dz, dw = gdr.gated_norm_bwd(d, x, z, w)
    assert not dx[:, :-n].any() and not dz[:, :-n].any()
    for g, e in zip((dx, dz), gdr.gated_norm_bwd(small[2], *small[:2], w)):
        assert torch.equal(g[:, -n:], e)
    (_, _, _, ref), sizes = gated_ref(*small[:2], w, small[2], "silu", False)
    check(dw, ref, sizes[3])


@pytest.mark.parametrize("D,offset", [(4096, 0), (4099, 0), (200, 0), (4096, 1)])
def test_residual_offsets_beyond_32_bits(D, offset):
    """The same for the residual's add and norm, in place where it is dense."""
    T, n = (1 << 31) // D + 40, 9
    r, y = (_many(T, D + offset, seed)[:, offset:].view(1, T, D) for seed in (5, 6))
    w, s = (1 + 0.2 * rnd(gen_of(seed), D) for seed in (7, 8))
    small = [t[:, -n:].clone() for t in (r, y)]
    want, stored = gdr.residual_norm(*small, w, scale=s, out_dtype=BF)
    out, res = gdr.residual_norm(r, y, w, scale=s, out_dtype=BF, residual_out=None if offset else r)
    assert torch.equal(out[:, -n:], want) and torch.equal(res[:, -n:], stored)
    out.zero_()
    d = out
    d[:, -n:] = rnd(gen_of(9), 1, n, D, dtype=BF)
    dr, dy, _, dw, _, ds = gdr.residual_norm_bwd(d, None, res, y, w, scale=s)
    assert not dr[:, :-n].any() and not dy[:, :-n].any()
    dn = d[:, -n:].clone()
    e = gdr.residual_norm_bwd(dn, None, stored, small[1], w, scale=s)
    assert torch.equal(dr[:, -n:], e[0]) and torch.equal(dy[:, -n:], e[1])
    ref = residual_ref(*small, w, None, None, s, dn, None, "sigmoid", False, stored)
    check(dw, *ref["dw"])
    check(ds, *ref["ds"])
