"""GPU numerics of the gated linear recurrence, the q/k norm with rotation and the paged
decode attention, against plain 64-bit implementations written here.

Tolerances. e = 2^-24 is fp32's rounding unit, u = 2^-8 bf16's (8 significant bits). A bf16
result has to be the rounding of a value within the fp32 tolerance of the reference.
- Scan: a step rounds exp(g) (1 ulp), one product and one sum, at most 4 e |h|max, and an
  error lives for 1 / (1 - a) tokens. Gates here keep that below about 60 tokens:
  4 e 60 = 1.5e-5 of the largest |h|; 2e-5 is used.
- Norm and rotation: a sum of at most 256 squares, rsqrt and three products: below 64 e of
  the row's largest value; 4e-6 is used. Weight gradients sum n rows of such terms: 4e-6 of
  the sum of the terms' magnitudes.
- Attention: fp32 scores of |s| < 40 are within 40 * 16 e < 4e-5 of themselves, and so is
  every weight; on the tensor cores a weight is also rounded to bf16 (u), or where the
  result is fp32 to two of them (u^2): (4e-5 [+ u or u^2]) sum p |v| / sum p.
"""
import math

import pytest
import torch

import chunkwise_gated_delta_gdr_gb300 as gdr

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -8
DEV = "cuda:0"


def rnd(gen, *shape, dtype=F32):
    return torch.randn(*shape, generator=gen, dtype=F32).to(dtype).to(DEV)


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


def check(got, ref, tol, scale=None):
    """got is (the rounding of) a value within tol * scale of ref (default: the largest |ref|)."""
    assert got.shape == ref.shape
    scale = ref.abs().max() if scale is None else scale
    lo, hi = ((ref + s * tol * scale).to(got.dtype).double() for s in (-1, 1))
    over = torch.maximum(got.double() - hi, lo - got.double())
    assert not torch.isnan(over).any()
    assert over.max().item() <= 0, f"exceeds its bound by {over.max().item():.3e}"


# ------------------------------------------------------------------ gated linear recurrence
def scan_ref(x, g, h0, gated, dh=None, dfinal=None):
    x, g = x.double(), g.double()
    a = g.exp()
    m = 1 - a if gated else torch.ones_like(a)
    B, T, D = x.shape
    s = torch.zeros(B, D, dtype=torch.float64, device=x.device) if h0 is None else h0.double()
    before, h = [], []
    for t in range(T):
        before.append(s)
        s = a[:, t] * s + m[:, t] * x[:, t]
        h.append(s)
    h = torch.stack(h, 1)
    if dh is None:
        return h, s
    lam = torch.zeros_like(s) if dfinal is None else dfinal.double()
    dx, dg = torch.empty_like(x), torch.empty_like(x)
    for t in reversed(range(T)):
        lam = lam + dh[:, t].double()
        dx[:, t] = lam * m[:, t]
        dg[:, t] = lam * a[:, t] * (before[t] - (x[:, t] if gated else 0))
        lam = lam * a[:, t]
    return h, s, dx, dg, lam


def scan_inputs(B, T, D, xd, gd, seed, state=True):
    gen = gen_of(seed)
    x = rnd(gen, B, T, D, dtype=xd)
    g = torch.nn.functional.logsigmoid(rnd(gen, B, T, D) + 3.0).clamp_max(-1 / 60).to(gd)
    h0 = rnd(gen, B, D) if state else None
    dh = rnd(gen, B, T, D, dtype=xd)
    dfinal = rnd(gen, B, D) if state else None
    return x, g, h0, dh, dfinal


def scan_both(x, g, h0, dh, dfinal, gated):
    ck = gdr.linear_scan_checkpoints(x)
    h, s = gdr.linear_scan_fwd(x, g, h0, gated_input=gated, checkpoints=ck)
    dx, dg, dh0 = gdr.linear_scan_bwd(dh, x, g, ck, dfinal, gated_input=gated)
    return h, s, dx, dg, dh0


def scan_check(x, g, h0, dh, dfinal, gated):
    got = scan_both(x, g, h0, dh, dfinal, gated)
    ref = scan_ref(x, g, h0, gated, dh, dfinal)
    scales = [ref[0].abs().max()] * 2 + [ref[2].abs().max(), None, None]
    # dg and dh0 multiply a gradient and a state, each within its own tolerance.
    scales[3] = ref[2].abs().max() * (ref[0].abs().max() + x.double().abs().max() + 1)
    scales[4] = ref[2].abs().max() if not gated else ref[4].abs().max() + ref[2].abs().max() * 60
    for y, r, sc in zip(got, ref, scales):
        check(y, r, 2e-5, sc)


SCAN_SHAPES = [(1, 1, 1), (64, 1, 96), (2, 2, 34), (1, 63, 33), (1, 64, 64), (2, 65, 130),
               (3, 127, 7), (1, 128, 62), (2, 300, 512), (1, 1000, 96), (5, 17, 66),
               (1, 2065, 64), (2, 5000, 34), (1, 4096, 200), (33, 70, 258)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("shape", SCAN_SHAPES)
def test_scan_shapes(shape, gated):
    scan_check(*scan_inputs(*shape, F32, F32, 1, state=shape[1] % 2 == 1), gated)


@pytest.mark.parametrize("xd,gd", [(BF, F32), (BF, BF), (F32, BF)])
@pytest.mark.parametrize("shape", [(2, 1, 34), (1, 777, 33), (2, 1300, 128), (1, 900, 130)])
def test_scan_types(shape, xd, gd):
    scan_check(*scan_inputs(*shape, xd, gd, 2), True)
    scan_check(*scan_inputs(*shape, xd, gd, 3), False)


@pytest.mark.parametrize("shape", [(2, 1, 33), (2, 500, 64)])
def test_scan_fp32_output_of_bf16_input(shape):
    x, g, h0, _, _ = scan_inputs(*shape, BF, F32, 4)
    h, s = gdr.linear_scan_fwd(x, g, h0, out_dtype=F32)
    ref = scan_ref(x, g, h0, False)
    assert h.dtype == F32
    check(h, ref[0], 2e-5)
    check(s, ref[1], 2e-5, ref[0].abs().max())


@pytest.mark.parametrize("T", [1, 9, 700])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_scan_views(T, offset):
    """x, g and dh as slices of wider tensors, odd offsets and strides included."""
    gen, B, D = gen_of(5), 2, 66
    wide = rnd(gen, B, T, 2 * D + 5)
    x, dh = wide[..., offset:offset + D], wide[..., D + offset:2 * D + offset]
    g = -rnd(gen, T, B, D).abs().clamp_min(1 / 60).transpose(0, 1)
    scan_check(x, g, rnd(gen, B, D), dh, None, True)


def test_scan_broadcast_gate():
    """One gate row for every token and sequence (strides of zero)."""
    gen, B, T, D = gen_of(6), 3, 210, 64
    g = -rnd(gen, 1, 1, D).abs().clamp_min(1 / 60).expand(B, T, D)
    scan_check(rnd(gen, B, T, D), g, None, rnd(gen, B, T, D), rnd(gen, B, D), False)


@pytest.mark.parametrize("gated", [False, True])
def test_scan_restart(gated):
    """exp(-inf) = 0 restarts a channel; nothing before it reaches later states."""
    x, g, h0, dh, dfinal = scan_inputs(1, 400, 64, F32, F32, 7)
    g[:, ::37] = -math.inf
    g[:, 200] = -math.inf
    scan_check(x, g, h0, dh, dfinal, gated)
    x2 = x.clone()
    x2[:, :200] *= 3
    y, y2 = (gdr.linear_scan_fwd(v, g, h0, gated_input=gated)[0] for v in (x, x2))
    assert torch.equal(y[:, 200:], y2[:, 200:])


def test_scan_long_memory():
    """g = 0 keeps everything: h is a running sum, 3000 equal steps exact in fp32."""
    x = torch.ones(1, 3000, 66, device=DEV)
    h, s = gdr.linear_scan_fwd(x, torch.zeros_like(x))
    assert torch.equal(h[0, :, 5], torch.arange(1, 3001, device=DEV, dtype=F32))
    assert torch.equal(s, torch.full((1, 66), 3000.0, device=DEV))


@pytest.mark.parametrize("T", [0, 1, 5, 300])
def test_scan_state_in_place(T):
    x, g, h0, dh, dfinal = scan_inputs(2, T, 64, BF, F32, 8)
    h, s = gdr.linear_scan_fwd(x, g, h0)
    state = h0.clone()
    h2, s2 = gdr.linear_scan_fwd(x, g, state, final_state=state)
    assert s2 is state and torch.equal(s, state) and torch.equal(h, h2)
    ck = gdr.linear_scan_checkpoints(x)
    gdr.linear_scan_fwd(x, g, h0, checkpoints=ck)
    grads = gdr.linear_scan_bwd(dh, x, g, ck, dfinal)
    again = dfinal.clone()
    grads2 = gdr.linear_scan_bwd(dh, x, g, ck, again, d_initial_state=again)
    assert all(torch.equal(p, q) for p, q in zip(grads, grads2))
    if T == 0:
        assert torch.equal(s, h0) and torch.equal(grads[2], dfinal)
        assert not gdr.linear_scan_fwd(x, g)[1].any()


def test_scan_no_batch():
    x = torch.empty(0, 5, 8, device=DEV)
    h, s = gdr.linear_scan_fwd(x, x)
    assert h.shape == (0, 5, 8) and s.shape == (0, 8)


def test_scan_steps_continue_a_prefill():
    x, g, h0, _, _ = scan_inputs(3, 131, 64, BF, F32, 9)
    h, s = gdr.linear_scan_fwd(x, g, h0, out_dtype=F32)
    _, state = gdr.linear_scan_fwd(x[:, :120], g[:, :120], h0)
    for t in range(120, 131):
        step, _ = gdr.linear_scan_fwd(x[:, t:t + 1], g[:, t:t + 1], state, final_state=state,
                                      out_dtype=F32)
        check(step[:, 0], h[:, t].double(), 4e-5, h.abs().max().double())
    check(state, s.double(), 4e-5, h.abs().max().double())


def test_scan_runs_are_equal():
    args = scan_inputs(2, 3000, 128, BF, F32, 10)
    first = scan_both(*args, True)
    assert all(torch.equal(p, q) for p, q in zip(first, scan_both(*args, True)))


@pytest.mark.parametrize("gated", [False, True])
def test_scan_gradient_against_differences(gated):
    """Central differences along random directions; their fp32 noise is about
    e sqrt(n) |h| / step of a sum of n terms."""
    x, g, h0, dh, dfinal = scan_inputs(1, 150, 40, F32, F32, 11)
    _, _, dx, dg, dh0 = scan_both(x, g, h0, dh, dfinal, gated)
    gen, eps = gen_of(12), 1e-2

    def loss(x, g, h0):
        h, s = gdr.linear_scan_fwd(x, g, h0, gated_input=gated)
        return ((h.double() * dh).sum() + (s.double() * dfinal).sum()).item()

    for which, grad in enumerate((dx, dg, dh0)):
        args = [x, g, h0]
        v = rnd(gen, *args[which].shape) * 0.1
        vals = []
        for sign in (1, -1):
            moved = list(args)
            moved[which] = args[which] + sign * eps * v
            vals.append(loss(*moved))
        diff, dot = (vals[0] - vals[1]) / (2 * eps), (grad.double() * v).sum().item()
        size = (grad.double() * v).norm().item() * math.sqrt(grad.numel())
        assert abs(diff - dot) <= 2e-3 * size / math.sqrt(grad.numel()) + 1e-3 * abs(dot)


# ------------------------------------------------------------------ q/k norm and rotation
def tables(rows, R):
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return ang.cos().float().to(DEV), ang.sin().float().to(DEV)


def qk_ref(x, w, cos, sin, pos, eps, interleaved):
    x = x.double()
    y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double()
    if cos is None:
        return y
    c, s = cos.double()[pos.long()][:, :, None], sin.double()[pos.long()][:, :, None]
    R = 2 * cos.shape[1]
    out = y.clone()
    i = torch.arange(0, R, 2, device=x.device) if interleaved else torch.arange(R // 2,
                                                                               device=x.device)
    j = i + 1 if interleaved else i + R // 2
    out[..., i] = y[..., i] * c - y[..., j] * s
    out[..., j] = y[..., j] * c + y[..., i] * s
    return out


def row_scale(ref):
    return ref.abs().amax(-1, keepdim=True).clamp_min(1e-6)


QK_SHAPES = [  # B, T, HQ, HK, D, R, interleaved, dtype
    (1, 1, 1, 1, 64, 64, False, BF), (2, 7, 4, 2, 128, 128, False, BF),
    (1, 33, 3, 1, 128, 64, False, BF), (2, 5, 6, 2, 256, 64, True, BF),
    (1, 9, 2, 2, 80, 40, False, BF), (1, 9, 5, 1, 96, 48, True, F32),
    (3, 4, 2, 1, 256, 256, False, F32), (1, 6, 2, 1, 33, 32, True, F32),
    (2, 3, 1, 1, 6, 2, False, BF), (1, 300, 12, 12, 128, 128, False, BF),
    (1, 5, 2, 2, 72, 0, False, BF), (2, 40, 16, 4, 64, 32, False, F32),
    (1, 3, 40, 8, 128, 20, False, BF), (70, 1, 16, 4, 128, 128, True, BF),
    (1, 2, 1, 1, 2, 2, False, F32), (1, 2, 1, 1, 1, 0, False, F32),
    # enough tokens for the ring of whole tokens: several tiles a block, ragged ends
    (1, 1301, 3, 1, 128, 128, False, BF), (2, 999, 4, 4, 64, 32, True, BF),
    (3, 1001, 2, 1, 80, 40, False, BF), (1, 701, 5, 2, 96, 96, False, F32),
    (1, 613, 9, 3, 256, 64, False, BF), (2, 2503, 1, 1, 128, 0, False, BF),
    (1, 9001, 1, 1, 64, 64, False, BF), (1, 350, 33, 3, 128, 128, True, F32),
]


def qk_inputs(B, T, HQ, HK, D, R, dt, seed, odd=False):
    gen = gen_of(seed)
    pad = 1 if odd else 0
    n = (HQ + 2 * HK) * D
    qkv = rnd(gen, B, T, n + pad, dtype=dt)[..., pad:]
    q = qkv[..., :HQ * D].unflatten(-1, (HQ, D))
    k = qkv[..., HQ * D:(HQ + HK) * D].unflatten(-1, (HK, D))
    v = qkv[..., (HQ + HK) * D:].unflatten(-1, (HK, D))
    wq, wk = rnd(gen, D) * 0.2 + 1, rnd(gen, D) * 0.2 + 1
    rows = T + 50
    cos, sin = tables(rows, R) if R else (None, None)
    pos = torch.randint(0, rows, (B, T), generator=gen, dtype=torch.int32).to(DEV)
    return q, k, v, wq, wk, cos, sin, pos


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("case", QK_SHAPES)
def test_qk_forward_and_backward(case, odd):
    B, T, HQ, HK, D, R, inter, dt = case
    q, k, _, wq, wk, cos, sin, pos = qk_inputs(B, T, HQ, HK, D, R, dt, 20, odd)
    args = (wq, wk, cos, sin, pos)
    qo, ko = gdr.qk_norm_rope(q, k, *args, eps=1e-5, interleaved=inter)
    gen = gen_of(21)
    dqo, dko = rnd(gen, B, T, HQ, D, dtype=dt), rnd(gen, B, T, HK, D, dtype=dt)
    grads = gdr.qk_norm_rope_bwd(dqo, dko, q, k, *args, eps=1e-5, interleaved=inter)
    for x, w, y, d, dx, dw in ((q, wq, qo, dqo, grads[0], grads[2]),
                               (k, wk, ko, dko, grads[1], grads[3])):
        xr = x.double().detach().requires_grad_(True)
        wr = w.double().requires_grad_(True)
        ref = qk_ref(xr, wr, cos, sin, pos, 1e-5, inter)
        check(y, ref.detach(), 4e-6, row_scale(ref.detach()))
        rx, rw = torch.autograd.grad(ref, (xr, wr), d.double())
        unit = qk_ref(x, None, None, None, None, 1e-5, False)
        inv = (unit / x.double()).abs().nan_to_num(0.0).amax(-1, keepdim=True)
        terms = d.double().abs().amax(-1, keepdim=True) * inv * 2
        check(dx, rx, 4e-6 * max(1, D / 32), terms * unit.abs().amax(-1, keepdim=True).clamp_min(1))
        mags = (d.double().abs().amax(-1, keepdim=True) * 2 * unit.abs()).sum((0, 1, 2))
        check(dw, rw, 4e-6, mags)


def test_qk_many_rows_per_group():
    """Long inputs keep up to 32 heads of a token in one group: 33 + 3 heads, split 17 and 16."""
    q, k, v, wq, wk, cos, sin, pos = qk_inputs(1, 20000, 33, 3, 64, 64, BF, 27)
    qo, ko = gdr.qk_norm_rope(q, k, wq, wk, cos, sin, pos)
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        ref = qk_ref(x, w, cos, sin, pos, 1e-6, False)
        check(y, ref, 4e-6, row_scale(ref))
    table, total = make_pages(torch.tensor([20000]), 64, gen_of(28))
    kc, vc = make_cache(gen_of(29), total, 64, 3, 64, BF)
    at = torch.arange(20000, device=DEV)[None].int()
    order = torch.arange(20000, device=DEV)
    pages = table.to(DEV)[0].long()[order // 64]
    plain = gdr.qk_norm_rope(q, k, wq, wk, cos[:1].expand_as(cos).contiguous(),
                             sin[:1].expand_as(sin).contiguous(), pos)
    same = gdr.qk_norm_rope_append(q, k, v, wq, wk, cos[:1].expand(20000, -1).contiguous(),
                                   sin[:1].expand(20000, -1).contiguous(), at, kc, vc,
                                   table.to(DEV))
    assert torch.equal(same, plain[0])
    assert torch.equal(kc[pages, order % 64], plain[1][0])
    assert torch.equal(vc[pages, order % 64], v[0])


@pytest.mark.parametrize("dt,out", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("D", [128, 30])
def test_qk_output_type(dt, out, D):
    q, k, _, wq, wk, cos, sin, pos = qk_inputs(2, 9, 4, 2, D, D, dt, 22)
    qo, ko = gdr.qk_norm_rope(q, k, wq, wk, cos, sin, pos, out_dtype=out)
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        ref = qk_ref(x, w, cos, sin, pos, 1e-6, False)
        assert y.dtype == out
        check(y, ref, 4e-6, row_scale(ref))
    d = (rnd(gen_of(1), *q.shape, dtype=out), rnd(gen_of(2), *k.shape, dtype=out))
    dq, dk, _, _ = gdr.qk_norm_rope_bwd(*d, q, k, wq, wk, cos, sin, pos)
    assert dq.dtype == dk.dtype == dt


def test_qk_long_positions_and_no_weights():
    q, k, _, _, _, cos, sin, pos = qk_inputs(2, 9, 4, 2, 128, 64, BF, 23)
    a = gdr.qk_norm_rope(q, k, None, None, cos, sin, pos)
    b = gdr.qk_norm_rope(q, k, torch.ones(128, device=DEV), None, cos, sin, pos.long())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    n = gdr.qk_norm_rope(q, k)
    ref = qk_ref(q, None, None, None, None, 1e-6, False)
    check(n[0], ref, 4e-6, row_scale(ref))


@pytest.mark.parametrize("D,T", [(128, 4), (30, 4), (128, 2000)])
def test_qk_zero_rows_and_extremes(D, T):
    """A zero row stays zero (1/sqrt(eps) times 0); a row of infinities gives NaN in it alone."""
    q, k, _, wq, wk, cos, sin, pos = qk_inputs(1, T, 2, 1, D, D, F32, 24)
    q, k = q.clone(), k.clone()
    q[0, 1, 0] = 0
    q[0, 2, 1] = math.inf
    qo, ko = gdr.qk_norm_rope(q, k, wq, wk, cos, sin, pos)
    assert not qo[0, 1, 0].any()
    assert torch.isnan(qo[0, 2, 1]).all()
    keep = torch.ones(T, 2, dtype=torch.bool)
    keep[2, 1] = False
    assert torch.isfinite(qo[0][keep]).all() and torch.isfinite(ko).all()
    dq = gdr.qk_norm_rope_bwd(torch.ones_like(qo[:, :2]), torch.ones_like(ko[:, :2]), q[:, :2],
                              k[:, :2], wq, wk, cos, sin, pos[:, :2].contiguous())[0]
    assert torch.isfinite(dq).all()


@pytest.mark.parametrize("bits", [torch.int32, torch.int64])
@pytest.mark.parametrize("D,T", [(128, 6), (30, 6), (128, 1500)])
def test_qk_positions_out_of_range(D, T, bits):
    q, k, _, wq, wk, cos, sin, pos = qk_inputs(2, T, 4, 2, D, D, BF, 25)
    pos = pos.to(bits)
    good = gdr.qk_norm_rope(q, k, wq, wk, cos, sin, pos)
    bad = pos.clone()
    bad[0, 1], bad[1, 4] = -1, cos.shape[0]
    if bits == torch.int64:
        bad[1, 0] = 1 << 40
    out = gdr.qk_norm_rope(q, k, wq, wk, cos, sin, bad)
    lost = (bad != pos)[:, :, None, None]
    for y, z in zip(out, good):
        assert torch.equal(torch.isnan(y), lost.expand_as(y))
        assert torch.equal(y[~lost.expand_as(y)], z[~lost.expand_as(y)])


def test_qk_runs_are_equal():
    q, k, _, wq, wk, cos, sin, pos = qk_inputs(2, 700, 12, 12, 128, 128, BF, 26)
    d = rnd(gen_of(1), *q.shape, dtype=BF)
    run = lambda: gdr.qk_norm_rope_bwd(d, d, q, k, wq, wk, cos, sin, pos)
    assert all(torch.equal(a, b) for a, b in zip(run(), run()))


def test_qk_no_tokens():
    q = torch.empty(2, 0, 4, 128, device=DEV)
    qo, ko = gdr.qk_norm_rope(q, q)
    assert qo.shape == q.shape
    _, _, dwq, dwk = gdr.qk_norm_rope_bwd(q, q, q, q)
    assert not dwq.any() and not dwk.any()


def test_qk_gradient_against_differences():
    q, k, _, wq, wk, cos, sin, pos = qk_inputs(1, 5, 3, 2, 96, 96, F32, 27)
    gen = gen_of(28)
    dqo, dko = rnd(gen, *q.shape), rnd(gen, *k.shape)
    grads = gdr.qk_norm_rope_bwd(dqo, dko, q, k, wq, wk, cos, sin, pos)

    def loss(q, k, wq, wk):
        qo, ko = gdr.qk_norm_rope(q, k, wq, wk, cos, sin, pos)
        return ((qo.double() * dqo).sum() + (ko.double() * dko).sum()).item()

    base, eps = [q.contiguous(), k.contiguous(), wq, wk], 1e-2
    for i, grad in enumerate(grads):
        v = rnd(gen, *base[i].shape)
        vals = []
        for sign in (1, -1):
            moved = list(base)
            moved[i] = base[i] + sign * eps * v
            vals.append(loss(*moved))
        diff, dot = (vals[0] - vals[1]) / (2 * eps), (grad.double() * v).sum().item()
        # second-order remainder eps^2 and fp32 noise over eps, per unit of |grad| |v|
        assert abs(diff - dot) <= 2e-3 * (grad.double().norm() * v.double().norm()).item()


# ------------------------------------------------------------------ paged caches
def make_pages(lens, page, gen, spare=2):
    need = [-(-int(n) // page) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen)
    most = max(1, max(need))
    table = torch.full((len(need), most), -1, dtype=torch.int32)
    owned = torch.arange(most)[None] < torch.tensor(need)[:, None]
    table[owned] = order[:sum(need)].to(torch.int32)
    return table, total


def make_cache(gen, total, page, HK, D, dt, layout="token"):
    """k and v caches [total, page, HK, D]; "head": heads outside tokens in memory; "odd":
    rows that start at odd elements."""
    out = []
    for _ in range(2):
        if layout == "head":
            out.append(rnd(gen, total, HK, page, D, dtype=dt).transpose(1, 2))
        elif layout == "odd":
            out.append(rnd(gen, total, page, HK, D + 3, dtype=dt)[..., :D])
        else:
            out.append(rnd(gen, total, page, HK, D, dtype=dt))
    return out


@pytest.mark.parametrize("case", [
    # B, T, HQ, HK, D, R, interleaved, dtype, cache dtype, page, layout
    (3, 1, 4, 2, 128, 128, False, BF, BF, 16, "token"), (64, 1, 16, 4, 128, 128, False, BF, BF, 64, "token"),
    (2, 4, 8, 1, 64, 32, True, BF, F32, 17, "token"), (2, 3, 3, 3, 80, 40, False, F32, BF, 1, "token"),
    (2, 2, 6, 2, 96, 48, False, F32, F32, 7, "head"), (1, 1, 1, 1, 33, 32, False, BF, BF, 5, "odd"),
    (2, 40, 4, 2, 256, 256, False, BF, BF, 16, "head"), (2, 2, 4, 2, 128, 0, False, BF, BF, 16, "token"),
])
def test_append(case):
    B, T, HQ, HK, D, R, inter, dt, cdt, page, layout = case
    gen = gen_of(30)
    q, k, v, wq, wk, cos, sin, _ = qk_inputs(B, T, HQ, HK, D, R, dt, 31)
    past = torch.randint(0, 40, (B,), generator=gen)
    table, total = make_pages(past + T, page, gen)
    kc, vc = make_cache(gen, total, page, HK, D, cdt, layout)
    k0, v0 = kc.clone(), vc.clone()
    pos = (past[:, None] + torch.arange(T)).to(torch.int32).to(DEV)
    if R:
        cos, sin = tables(40 + T, R)
    table = table.to(DEV)
    qo = gdr.qk_norm_rope_append(q, k, v, wq, wk, cos, sin, pos, kc, vc, table, interleaved=inter)
    ref = qk_ref(q, wq, cos, sin, pos, 1e-6, inter)
    check(qo, ref, 4e-6, row_scale(ref))
    pg = torch.gather(table.long(), 1, pos.long() // page)
    at = pos.long() % page
    ref = qk_ref(k, wk, cos, sin, pos, 1e-6, inter)
    check(kc[pg, at], ref, 4e-6, row_scale(ref))
    assert torch.equal(vc[pg, at], v.to(cdt))
    k0[pg, at], v0[pg, at] = kc[pg, at], vc[pg, at]      # nothing else was touched
    assert torch.equal(k0, kc) and torch.equal(v0, vc)


def test_append_out_of_range_stores_nothing():
    gen = gen_of(32)
    q, k, v, wq, wk, _, _, _ = qk_inputs(5, 1, 4, 2, 128, 128, BF, 33)
    cos, sin = tables(100, 128)
    table = torch.tensor([[0, 1], [2, 7], [3, -1], [4, 5], [6, 6]], dtype=torch.int32, device=DEV)
    kc, vc = make_cache(gen, 7, 16, 2, 128, BF)
    k0, v0 = kc.clone(), vc.clone()
    pos = torch.tensor([[3], [20], [16], [-1], [32]], dtype=torch.int32, device=DEV)
    qo = gdr.qk_norm_rope_append(q, k, v, wq, wk, cos, sin, pos, kc, vc, table)
    assert torch.isfinite(qo[0]).all() and torch.isnan(qo[1:]).all()
    changed = (kc != k0).any(-1).any(-1)
    assert changed.sum() == 1 and changed[0, 3]
    assert (vc != v0).any(-1).any(-1).sum() == 1


def attn_ref(q, kc, vc, table, lens, scale, window):
    """(o, lse, sum p |v| / sum p) in 64 bits."""
    B, HQ, D = q.shape
    HK, page = kc.shape[2], kc.shape[1]
    o = torch.zeros(B, HQ, D, dtype=torch.float64, device=q.device)
    size = torch.zeros_like(o)
    lse = torch.full((B, HQ), -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(lens.tolist()):
        lo = max(0, n - window) if window else 0
        if n <= lo:
            continue
        j = torch.arange(lo, n, device=q.device)
        pg = table[b].long()[j // page]
        k, v = (c[pg, j % page].double().transpose(0, 1) for c in (kc, vc))
        z = scale * q[b].double().view(HK, HQ // HK, D) @ k.transpose(1, 2)
        p = torch.softmax(z, -1)
        o[b], size[b] = (p @ v).reshape(HQ, D), (p @ v.abs()).reshape(HQ, D)
        lse[b] = torch.logsumexp(z, -1).reshape(HQ)
    return o, lse, size


def attn_check(q, kc, vc, table, lens, window=0, out_dtype=None, scale=None):
    D = q.shape[-1]
    o, lse = gdr.paged_decode_attn(q, kc, vc, table, lens, window=window, out_dtype=out_dtype,
                                   scale=scale)
    ro, rl, size = attn_ref(q, kc, vc, table, lens, scale or 1 / math.sqrt(D), window)
    tol = 4e-5
    if q.dtype == BF and kc.dtype == BF:
        tol += U if o.dtype == BF else U * U
    check(o, ro, tol, size)
    dead = torch.isinf(rl)
    assert torch.equal(lse[dead], rl[dead].float())
    assert not (dead[..., None] & (o != 0)).any()
    err = (lse.double() - rl)[~dead].abs()
    assert not err.numel() or (err <= 4e-5 * (1 + rl[~dead].abs())).all()
    return o, lse


EDGE = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 80, 96, 128, 192, 256, 40, 33, 1])
def test_attn_head_dims(D, dt):
    gen = gen_of(40)
    lens = torch.tensor(EDGE + [300, 1000])
    table, total = make_pages(lens, 16, gen)
    kc, vc = make_cache(gen, total, 16, 2, D, dt)
    q = rnd(gen, len(lens), 6, D, dtype=dt)
    attn_check(q, kc, vc, table.to(DEV), lens.int().to(DEV))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("HQ,HK", [(1, 1), (2, 1), (12, 4), (5, 1), (16, 16), (8, 1), (32, 2),
                                   (20, 1), (33, 1), (48, 1)])
def test_attn_groups(HQ, HK, dt):
    gen = gen_of(41)
    lens = torch.tensor([0, 700, 1, 130, 64])
    table, total = make_pages(lens, 32, gen)
    kc, vc = make_cache(gen, total, 32, HK, 128, dt)
    q = rnd(gen, 5, HQ, 128, dtype=dt)
    attn_check(q, kc, vc, table.to(DEV), lens.int().to(DEV))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("page", [1, 7, 16, 17, 64, 100, 4096])
def test_attn_pages(page, dt):
    gen = gen_of(42)
    lens = torch.tensor(EDGE + [2 * page, 2 * page + 1, 999])
    table, total = make_pages(lens, page, gen)
    kc, vc = make_cache(gen, total, page, 2, 64, dt)
    q = rnd(gen, len(lens), 4, 64, dtype=dt)
    attn_check(q, kc, vc, table.to(DEV), lens.int().to(DEV))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("window", [1, 5, 64, 100, 257, 5000])
def test_attn_window(window, dt):
    gen = gen_of(43)
    lens = torch.tensor(EDGE + [300, 2000])
    table, total = make_pages(lens, 16, gen)
    kc, vc = make_cache(gen, total, 16, 2, 128, dt)
    q = rnd(gen, len(lens), 8, 128, dtype=dt)
    attn_check(q, kc, vc, table.to(DEV), lens.int().to(DEV), window=window)


@pytest.mark.parametrize("lens", [[1], [0], [200], [256], [257], [20011], [1, 40000, 0, 0, 3],
                                  [5000] * 7, [0] * 40 + [3000] + [0] * 40, list(range(0, 700, 7))])
def test_attn_lengths(lens):
    """Short rows (one block each) and long ones cut into parts and joined."""
    gen = gen_of(44)
    lens = torch.tensor(lens)
    table, total = make_pages(lens, 64, gen)
    kc, vc = make_cache(gen, total, 64, 2, 128, BF)
    q = rnd(gen, len(lens), 8, 128, dtype=BF)
    attn_check(q, kc, vc, table.to(DEV), lens.int().to(DEV))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("layout", ["head", "odd"])
def test_attn_layouts(layout, dt):
    gen = gen_of(45)
    lens = torch.tensor([70, 500, 3, 0])
    table, total = make_pages(lens, 16, gen)
    kc, vc = make_cache(gen, total, 16, 2, 128, dt, layout)
    q = rnd(gen, 4, 3 * 8 * 128 + 1, dtype=dt)[:, 1:1 + 8 * 128].unflatten(-1, (8, 128))
    attn_check(q, kc, vc, table.to(DEV), lens.int().to(DEV))


@pytest.mark.parametrize("qd,cd,od", [(F32, BF, BF), (BF, F32, F32), (BF, BF, F32), (F32, F32, BF)])
def test_attn_types(qd, cd, od):
    gen = gen_of(46)
    lens = torch.tensor([70, 500, 3, 0])
    table, total = make_pages(lens, 16, gen)
    kc, vc = make_cache(gen, total, 16, 2, 128, cd)
    attn_check(rnd(gen, 4, 8, 128, dtype=qd), kc, vc, table.to(DEV), lens.int().to(DEV),
               out_dtype=od, scale=0.3)


@pytest.mark.parametrize("dt,D", [(BF, 128), (F32, 64), (BF, 40)])
def test_attn_never_reads_past_a_sequence(dt, D):
    """NaN and infinity in every place that no sequence owns change nothing."""
    gen = gen_of(47)
    lens = torch.tensor([1, 17, 100, 0, 333])
    table, total = make_pages(lens, 16, gen)
    kc, vc = make_cache(gen, total, 16, 2, D, dt)
    q, table, ln = rnd(gen, 5, 4, D, dtype=dt), table.to(DEV), lens.int().to(DEV)
    o, lse = attn_check(q, kc, vc, table, ln)
    live = torch.zeros(total, 16, dtype=torch.bool)
    for b, n in enumerate(lens.tolist()):
        j = torch.arange(n)
        live[table[b].cpu().long()[j // 16], j % 16] = True
    for junk in (math.nan, math.inf, -math.inf):
        k2, v2 = kc.clone(), vc.clone()
        k2[~live.to(DEV)], v2[~live.to(DEV)] = junk, junk
        o2, l2 = gdr.paged_decode_attn(q, k2, v2, table, ln)
        assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dt,D", [(BF, 128), (F32, 64)])
def test_attn_out_of_range(dt, D):
    """A bad length or page gives NaN for its own sequence only."""
    gen = gen_of(48)
    for most in (3, 40):                     # one block per row; rows cut into parts
        lens = torch.full((6,), most * 16)
        table, total = make_pages(lens, 16, gen)
        kc, vc = make_cache(gen, total, 16, 2, D, dt)
        q = rnd(gen, 6, 4, D, dtype=dt)
        good, _ = gdr.paged_decode_attn(q, kc, vc, table.to(DEV), lens.int().to(DEV))
        table[1, 2], table[3, 0] = -1, total
        lens[4], lens[5] = most * 16 + 1, -1
        o, lse = gdr.paged_decode_attn(q, kc, vc, table.to(DEV), lens.int().to(DEV))
        for b in range(6):
            if b in (1, 3, 4, 5):
                assert torch.isnan(o[b]).all() and torch.isnan(lse[b]).all(), b
            else:
                assert torch.isfinite(o[b]).all()
        check(o[0], good[0].double(), 1e-2)
        check(o[2], good[2].double(), 1e-2)


@pytest.mark.parametrize("dt,D", [(BF, 128), (F32, 64)])
def test_attn_extreme_scores(dt, D):
    """Scores far apart and far from zero: the largest one carries the weight."""
    gen = gen_of(49)
    lens = torch.tensor([500, 500])
    table, total = make_pages(lens, 16, gen)
    kc, vc = make_cache(gen, total, 16, 1, D, dt)
    q = rnd(gen, 2, 2, D, dtype=dt)
    kc[table[0, 10].item(), 3] = 200 * q[0, 0]
    kc[table[0, 20].item(), 5] = -200 * q[0, 1]
    o, lse = gdr.paged_decode_attn(q, kc, vc, table.to(DEV), lens.int().to(DEV))
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert torch.equal(o[0, 0], vc[table[0, 10].item(), 3, 0])
    top = (q[0, 0].double() @ kc[table[0, 10].item(), 3, 0].double()) / math.sqrt(D)
    assert abs(lse[0, 0].item() - top.item()) <= 4e-5 * abs(top.item())


def test_attn_offsets_beyond_32_bits():
    """Rows more than 2^31 elements into the caches."""
    gen, page, HK, D = gen_of(50), 64, 2, 128
    total = (1 << 31) // (page * HK * D) + 40
    kc = torch.zeros(total, page, HK, D, dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    last = torch.arange(total - 8, total)
    kc[last], vc[last] = rnd(gen, 8, page, HK, D, dtype=BF), rnd(gen, 8, page, HK, D, dtype=BF)
    table = last.flip(0).int()[None].to(DEV)
    lens = torch.tensor([500], dtype=torch.int32, device=DEV)
    q = rnd(gen, 1, 8, D, dtype=BF)
    attn_check(q, kc, vc, table, lens)
    qn, kn, vn, wq, wk, _, _, _ = qk_inputs(1, 1, 4, HK, D, D, BF, 51)
    cos, sin = tables(600, D)
    pos = torch.tensor([[501]], dtype=torch.int32, device=DEV)
    gdr.qk_norm_rope_append(qn, kn, vn, wq, wk, cos, sin, pos, kc, vc, table)
    assert torch.equal(vc[last[0], 501 % 64], vn[0, 0])


def test_attn_runs_are_equal_and_lse_is_optional():
    gen = gen_of(52)
    lens = torch.tensor([9000, 20, 4000])
    table, total = make_pages(lens, 64, gen)
    kc, vc = make_cache(gen, total, 64, 2, 128, BF)
    q, table, ln = rnd(gen, 3, 16, 128, dtype=BF), table.to(DEV), lens.int().to(DEV)
    a = gdr.paged_decode_attn(q, kc, vc, table, ln)
    ws = torch.full((gdr.paged_decode_attn_workspace_size(q, kc, table),), 255, dtype=torch.uint8,
                    device=DEV)                          # NaN bits: contents do not matter
    b = gdr.paged_decode_attn(q, kc, vc, table, ln, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_another_stream():
    """Calls on a stream that is not torch's current one, buffers allocated inside."""
    gen = gen_of(53)
    x, g, h0, _, _ = scan_inputs(2, 700, 128, BF, F32, 54)
    q, k, _, wq, wk, cos, sin, pos = qk_inputs(2, 50, 4, 2, 128, 128, BF, 55)
    lens = torch.tensor([4000, 30])
    table, total = make_pages(lens, 64, gen)
    kc, vc = make_cache(gen, total, 64, 2, 128, BF)
    qa, table, ln = rnd(gen, 2, 8, 128, dtype=BF), table.to(DEV), lens.int().to(DEV)

    def calls(stream=None):
        return (*gdr.linear_scan_fwd(x, g, h0, stream=stream),
                *gdr.qk_norm_rope(q, k, wq, wk, cos, sin, pos, stream=stream),
                *gdr.qk_norm_rope_bwd(q.contiguous(), k.contiguous(), q, k, wq, wk, cos, sin, pos,
                                      stream=stream),
                *gdr.paged_decode_attn(qa, kc, vc, table, ln, stream=stream))

    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = calls(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_memory_of_results_on_another_stream():
    """Memory that the current stream still reads is not given to a call on another one."""
    x, g, _, _, _ = scan_inputs(1, 4096, 1024, BF, F32, 57)
    want = gdr.linear_scan_fwd(x, g)[0]
    big, old, copy = torch.zeros(1 << 28, device=DEV), torch.full_like(want, 3), want.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        big.mul_(1.0)
    copy.copy_(old)
    del old
    got = gdr.linear_scan_fwd(x, g, stream=side)[0]
    torch.cuda.synchronize()
    assert (copy == 3).all() and torch.equal(got, want)


def test_sizes_past_32_bits_are_refused():
    x = torch.empty(1 << 32, 0, 4, dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="B = 4294967296"):
        gdr.linear_scan_fwd(x, x, output_final_state=False)
    q = torch.empty(1 << 32, 0, 1, 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="B = 4294967296"):
        gdr.qk_norm_rope(q, q)


def test_capture_in_a_graph():
    """The serving calls of one step, captured once and replayed on new inputs."""
    gen = gen_of(56)
    B, HQ, HK, D, page = 3, 8, 2, 128, 16
    past = torch.tensor([5, 700, 0])
    table, total = make_pages(past + 8, page, gen)
    kc, vc = make_cache(gen, total, page, HK, D, BF)
    table = table.to(DEV)
    cos, sin = tables(800, D)
    w = torch.ones(D, device=DEV)
    qkv = rnd(gen, B, 1, HQ + 2 * HK, D, dtype=BF)
    q, k, v = qkv[:, :, :HQ], qkv[:, :, HQ:HQ + HK], qkv[:, :, HQ + HK:]
    pos = past[:, None].int().to(DEV)
    lens = (past + 1).int().to(DEV)
    x, g = rnd(gen, B, 1, 64, dtype=BF), -rnd(gen, B, 1, 64).abs()
    state = rnd(gen, B, 64)

    def step():
        qo = gdr.qk_norm_rope_append(q, k, v, w, w, cos, sin, pos, kc, vc, table)
        o, _ = gdr.paged_decode_attn(qo[:, 0], kc, vc, table, lens)
        h, _ = gdr.linear_scan_fwd(x, g, state, final_state=state)
        return o, h

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    state.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, h = step()
    state.zero_()
    for _ in range(3):
        qkv.copy_(rnd(gen, *qkv.shape, dtype=BF))
        graph.replay()
        torch.cuda.synchronize()
        qo = gdr.qk_norm_rope(q, k, w, w, cos, sin, pos)[0]
        ro, _, size = attn_ref(qo[:, 0], kc, vc, table, lens, 1 / math.sqrt(D), 0)
        check(o, ro, 4e-5 + U, size)
        pos += 1
        lens += 1
    a = g.double().exp()[:, 0]
    want = x[:, 0].double() * (1 + a + a * a)
    check(state, want, 2e-5)


def test_compiled_calls_take_the_ordinary_case(monkeypatch):
    """The compiled calls and the Python ones give the same bits; the ordinary case, results
    passed in or not, never reaches the Python ones."""
    from chunkwise_gated_delta_gdr_gb300 import layers
    gen = gen_of(60)
    x, g, h0, dh, dfinal = scan_inputs(2, 300, 128, BF, F32, 61)
    q, k, v, wq, wk, cos, sin, pos = qk_inputs(3, 1, 4, 2, 128, 64, BF, 62)
    lens = torch.tensor([40, 3000, 7])
    table, total = make_pages(lens + 1, 16, gen)
    kc, vc = make_cache(gen, total, 16, 2, 128, BF)
    table, ln = table.to(DEV), lens.int().to(DEV)
    at = lens[:, None].int().to(DEV)
    cos2, sin2 = tables(4000, 64)
    dq = rnd(gen, *q.shape, dtype=BF), rnd(gen, *k.shape, dtype=BF)
    outs = [torch.empty(2, 300, 128, dtype=BF, device=DEV), torch.empty(2, 128, device=DEV),
            torch.empty(3, 1, 4, 128, dtype=BF, device=DEV)]

    def calls():
        ck = gdr.linear_scan_checkpoints(x)
        r = [*gdr.linear_scan_fwd(x, g, h0, checkpoints=ck),
             *gdr.linear_scan_fwd(x, g, h0, gated_input=True, out=outs[0], final_state=outs[1]),
             *gdr.linear_scan_fwd(x, g, output_final_state=False),
             *gdr.linear_scan_bwd(dh, x, g, ck, dfinal),
             *gdr.qk_norm_rope(q, k, wq, wk, cos, sin, pos), *gdr.qk_norm_rope(q, k),
             *gdr.qk_norm_rope(q, k, wq, None, cos, sin, pos.long(), eps=1e-3, interleaved=True),
             *gdr.qk_norm_rope_bwd(*dq, q, k, wq, wk, cos, sin, pos),
             *gdr.qk_norm_rope_bwd(*dq, q, k, output_weight_grads=False),
             gdr.qk_norm_rope_append(q, k, v, wq, wk, cos2, sin2, at, kc, vc, table, q_out=outs[2]),
             kc, vc, *gdr.paged_decode_attn(q[:, 0], kc, vc, table, ln + 1),
             *gdr.paged_decode_attn(q[:, 0], kc, vc, table, ln + 1, scale=0.2, window=50)]
        return [t if t is None else t.clone() for t in r]

    with monkeypatch.context() as m:
        m.setattr(layers, "_lib", None)                  # the Python calls cannot run
        fast = calls()
    monkeypatch.setattr(layers, "_host", None)
    slow = calls()
    assert len(fast) == len(slow)
    for a, b in zip(fast, slow):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("compiled", [True, False])
def test_refusals_on_the_gpu(compiled, monkeypatch):
    from chunkwise_gated_delta_gdr_gb300 import layers
    if not compiled:
        monkeypatch.setattr(layers, "_host", None)
    x = torch.zeros(2, 8, 16, device=DEV)
    q, k = torch.zeros(2, 3, 4, 64, device=DEV), torch.zeros(2, 3, 2, 64, device=DEV)
    kc = torch.zeros(5, 16, 2, 64, device=DEV)
    table, lens = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.ones(2, device=DEV).int()
    bad = [
        (lambda: gdr.linear_scan_fwd(x, x[:, :4]), ValueError),
        (lambda: gdr.linear_scan_fwd(x, x.cpu()), ValueError),
        (lambda: gdr.linear_scan_fwd(x, x.double()), TypeError),
        (lambda: gdr.linear_scan_fwd(x.transpose(1, 2), x.transpose(1, 2)), ValueError),
        (lambda: gdr.linear_scan_fwd(x, x, torch.zeros(2, 15, device=DEV)), ValueError),
        (lambda: gdr.linear_scan_fwd(x, x, torch.zeros(2, 16, device=DEV).bfloat16()), TypeError),
        (lambda: gdr.linear_scan_fwd(x, x, out=x.bfloat16(), out_dtype=F32), TypeError),
        (lambda: gdr.linear_scan_bwd(x, x, x, None), ValueError),
        (lambda: gdr.linear_scan_bwd(x, x, x, torch.zeros(2, 2, 16, device=DEV)), ValueError),
        (lambda: gdr.qk_norm_rope(q, k[:, :2]), ValueError),
        (lambda: gdr.qk_norm_rope(q, k.bfloat16()), TypeError),
        (lambda: gdr.qk_norm_rope(q, k, eps=0.0), gdr.GdrError),
        (lambda: gdr.qk_norm_rope(q, k, torch.ones(63, device=DEV)), ValueError),
        (lambda: gdr.qk_norm_rope(q, k, None, None, x[0], x[0]), ValueError),
        (lambda: gdr.paged_decode_attn(q[:, 0], kc, kc, table.long(), lens), TypeError),
        (lambda: gdr.paged_decode_attn(q[:, 0], kc, kc, table, lens.long()), TypeError),
        (lambda: gdr.paged_decode_attn(q[:, 0], kc, kc[:, :, :1], table, lens), ValueError),
        (lambda: gdr.paged_decode_attn(q[:, 0, :3], kc, kc, table, lens), gdr.GdrError),
        (lambda: gdr.paged_decode_attn(q[:, 0], kc, kc, table, lens, scale=-1.0), gdr.GdrError),
        (lambda: gdr.paged_decode_attn(q[:, 0], kc, kc, table, lens, window=-1), gdr.GdrError),
        (lambda: gdr.paged_decode_attn(q[:, 0], kc, kc, table, lens,
                                       workspace=torch.zeros(64, dtype=torch.uint8, device=DEV)),
         gdr.GdrError),
    ]
    for i, (call, error) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"refusal {i} did not come")
