"""The layers' operators where values, sizes and arguments are out of the ordinary, against
the 64-bit implementations of test_layers_gpu.py; tolerances as derived there, or beside the
test."""
import ctypes
import math

import pytest
import torch

import chunkwise_gated_delta_gdr_gb300 as gdr
from test_layers_gpu import (BF, DEV, EDGE, F32, attn_ref, check, gen_of, make_cache, make_pages,
                             qk_inputs, qk_ref, rnd, scan_check, scan_inputs, tables)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ weights of the attention
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("D", [64, 80, 96, 128, 192, 256])
def test_attn_weights_keep_two_parts(D, out):
    """bf16 caches, results of either type: a weight loses at most 2^-15 of itself on the tensor
    cores, beside the 4e-5 of every form; whole rows and rows cut into parts and joined."""
    gen = gen_of(70)
    for lens in (torch.tensor(EDGE + [2, 3, 300]), torch.tensor([5, 5000, 0, 700])):
        table, total = make_pages(lens, 16, gen)
        kc, vc = make_cache(gen, total, 16, 2, D, BF)
        q = rnd(gen, len(lens), 6, D, dtype=BF)
        table, lens = table.to(DEV), lens.int().to(DEV)
        o, _ = gdr.paged_decode_attn(q, kc, vc, table, lens, out_dtype=out)
        ref, _, size = attn_ref(q, kc, vc, table, lens, 1 / math.sqrt(D), 0)
        check(o, ref, 4e-5 + 2.0 ** -15, size)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 256), (F32, 64), (BF, 40)])
@pytest.mark.parametrize("n", [90, 3000])
def test_attn_infinite_values(dt, D, out, n):
    """One infinite value makes its channel infinite for the heads that see it, two of opposite
    signs (or a NaN) make it NaN; every other channel keeps its bits."""
    gen = gen_of(71)
    lens = torch.tensor([n, n])
    table, total = make_pages(lens, 16, gen)
    kc, vc = make_cache(gen, total, 16, 2, D, dt)
    kc *= 0.25                               # weights of one size
    q, lens = rnd(gen, 2, 4, D, dtype=dt), lens.int().to(DEV)
    good, lse = gdr.paged_decode_attn(q, kc, vc, table.to(DEV), lens, out_dtype=out)

    def put(j, ch, value):                   # sequence 0, kv head 1: query heads 2 and 3
        vc[table[0, j // 16].item(), j % 16, 1, ch] = value

    put(3, 0, math.inf), put(40, 9, -math.inf), put(n - 1, 2, math.inf)
    put(17, 5, math.inf), put(70, 5, -math.inf), put(20, 7, math.nan)
    o, lse2 = gdr.paged_decode_attn(q, kc, vc, table.to(DEV), lens, out_dtype=out)
    want = good.clone()
    want[0, 2:, [0, 2]], want[0, 2:, 9], want[0, 2:, [5, 7]] = math.inf, -math.inf, math.nan
    assert torch.equal(lse, lse2)
    assert torch.equal(torch.isnan(o), torch.isnan(want))
    assert torch.equal(o.nan_to_num(1.5), want.nan_to_num(1.5))


# ------------------------------------------------------------------ values on their way to the cache
def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF else torch.int32)


@pytest.mark.parametrize("dt,cdt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (64, 0), (256, 256), (80, 40)])
@pytest.mark.parametrize("T", [1, 9])
def test_append_stores_values_unchanged(T, D, R, odd, dt, cdt):
    """Infinities, NaN and -0 in turned and unturned channels of v: bit for bit where the types
    agree (else v.to of the cache's type), by the kernel for aligned rows and the other."""
    B, HQ, HK, page = 3, 4, 2, 16
    q, k, v, wq, wk, cos, sin, _ = qk_inputs(B, T, HQ, HK, D, R, dt, 72, odd)
    cos, sin = tables(60, R) if R else (None, None)
    v = v.clone() if not odd else v          # the rows of `odd` start off every alignment
    for h in range(HK):
        for ch, x in ((0, math.inf), (1, -0.0), (D // 2 - 1, math.nan), (D // 2 + 3, -math.inf),
                      (D - 1, math.nan), (D - 2, math.inf), (D // 4, -0.0)):
            v[:, h % T, h, ch] = x
    table, total = make_pages(torch.full((B,), 40), page, gen_of(73))
    kc, vc = make_cache(gen_of(74), total, page, HK, D, cdt)
    pos = (torch.tensor([[0], [13], [30]]) + torch.arange(T)).int().to(DEV)
    table = table.to(DEV)
    gdr.qk_norm_rope_append(q, k, v, wq, wk, cos, sin, pos, kc, vc, table)
    got = vc[torch.gather(table.long(), 1, pos.long() // page), pos.long() % page]
    want = v.to(cdt)
    if dt == cdt:
        assert torch.equal(bits(got), bits(want))
    else:
        nan = torch.isnan(want)
        assert torch.equal(nan, torch.isnan(got))
        assert torch.equal(bits(got)[~nan], bits(want)[~nan])


# ------------------------------------------------------------------ waits of the scan that give up
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("B,T,D", [(1, 5000, 512), (3, 700, 1024), (1, 3000, 66), (2, 900, 33)])
def test_scan_waits_that_give_up(B, T, D, dt, gated):
    """With few polls allowed, waits for tiles and for other blocks give up: every result is NaN
    or has its right bits, the launch ends by itself, and calls with the usual bound are as ever."""
    x, g, h0, dh, dfinal = scan_inputs(B, T, D, dt, F32, 75)
    ck = gdr.linear_scan_checkpoints(x)

    def calls():
        outs = [torch.full_like(x, 7), torch.full_like(h0, 7), torch.full_like(ck, 7),
                torch.full_like(x, 7), torch.full_like(g, 7), torch.full_like(h0, 7)]
        gdr.linear_scan_fwd(x, g, h0, gated_input=gated, out=outs[0], final_state=outs[1],
                            checkpoints=outs[2])
        gdr.linear_scan_bwd(dh, x, g, ck, dfinal, gated_input=gated, dx=outs[3], dg=outs[4],
                            d_initial_state=outs[5])
        torch.cuda.synchronize()
        return outs

    gdr.linear_scan_fwd(x, g, h0, gated_input=gated, checkpoints=ck)
    want = calls()
    old = gdr.set_flag_wait_limit(-1)
    for polls in (0, 0, 1, 2, 8, 64):
        gdr.set_flag_wait_limit(polls)
        try:
            got = calls()
        finally:
            gdr.set_flag_wait_limit(old)
        for a, b in zip(got, want):
            there = ~torch.isnan(a)
            assert torch.equal(a[there], b[there]), polls
        if polls == 0 and D * x.element_size() % 16 == 0:    # a tile needs a microsecond
            assert torch.isnan(got[0]).any() and torch.isnan(got[3]).any()
    assert all(torch.equal(a, b) for a, b in zip(calls(), want))


# ------------------------------------------------------------------ calls and their statuses
def test_compiled_calls_answer_a_status(monkeypatch):
    """A refusal of the C ABI comes back from the compiled call, and is not asked for twice."""
    from chunkwise_gated_delta_gdr_gb300 import layers
    q, k = torch.zeros(2, 3, 4, 64, device=DEV), torch.zeros(2, 3, 2, 64, device=DEV)
    assert layers._host.qk_norm_rope(q, k, None, None, None, None, None, 0.0, False, None,
                                     None) == gdr.GDR_ERR_INVALID_ARG
    monkeypatch.setattr(layers, "_lib", None)            # the Python call cannot run
    with pytest.raises(gdr.GdrError, match="gdr_qk_norm_rope"):
        gdr.qk_norm_rope(q, k, eps=0.0)


def leave_an_error():
    """A host-side error that the library does not clear: its stream status asked for while the
    stream is being captured, which only ends the capture."""
    paths = {line.split()[-1] for line in open("/proc/self/maps") if "/libcudart.so" in line}
    rt = ctypes.CDLL(paths.pop())
    stream = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    assert rt.cudaStreamBeginCapture(handle, 2) == 0                 # relaxed
    try:
        assert gdr.stream_status(stream) == gdr.GDR_ERR_CUDA
    finally:
        assert rt.cudaStreamEndCapture(handle, ctypes.byref(graph)) != 0
        rt.cudaGetLastError()


@pytest.mark.parametrize("T", [1, 700])
def test_scan_reports_its_own_status(T):
    """An error that an earlier call left behind is not this call's, whose state moves once."""
    x, g, h0, _, _ = scan_inputs(2, T, 64, BF, F32, 76)
    want, state = gdr.linear_scan_fwd(x, g, h0)[1], h0.clone()
    leave_an_error()
    gdr.linear_scan_fwd(x, g, state, final_state=state)
    assert torch.equal(state, want)


@pytest.mark.parametrize("D", [64, 33])
def test_norm_and_attention_report_their_own_status(D):
    q, k, v, wq, wk, cos, sin, _ = qk_inputs(2, 1, 4, 2, D, 32, BF, 77)
    table, total = make_pages(torch.tensor([9, 9]), 16, gen_of(78))
    kc, vc = make_cache(gen_of(79), total, 16, 2, D, BF)
    table, lens = table.to(DEV), torch.tensor([9, 9], dtype=torch.int32, device=DEV)
    pos = (lens - 1)[:, None].contiguous()
    d = torch.ones_like(q, memory_format=torch.contiguous_format)
    for call in (lambda: gdr.qk_norm_rope(q, k, wq, wk, cos, sin, pos),
                 lambda: gdr.qk_norm_rope_bwd(d, d[:, :, :2].contiguous(), q, k, wq, wk, cos, sin,
                                              pos),
                 lambda: gdr.qk_norm_rope_append(q, k, v, wq, wk, cos, sin, pos, kc, vc, table),
                 lambda: gdr.paged_decode_attn(q[:, 0], kc, vc, table, lens)):
        leave_an_error()
        call()


# ------------------------------------------------------------------ slow gates
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("B,T,D", [(2, 1, 64), (1, 20, 66), (1, 300, 64), (3, 260, 33), (40, 31, 514),
                                   (2, 700, 258)])
def test_scan_gated_input_of_slow_gates(B, T, D, dt):
    """Gates of 1e-8 .. 1, of either sign: every state and gradient to its own size. The weight
    -expm1(g) is within 3e-7 of itself; a step rounds exp(g), products and sums, 2.5e-7 of the
    state in all, and x and dh are positive, so that nothing cancels."""
    gen = gen_of(80)
    x = (rnd(gen, B, T, D).abs() + 0.5).to(dt)
    dh = (rnd(gen, B, T, D).abs() + 0.5).to(dt)
    size = 10.0 ** (-8 * torch.rand(D, generator=gen, dtype=torch.float64))
    sign = torch.where(torch.arange(D) % 5 == 4, 1.0, -1.0)
    size[sign > 0] *= 1e-3                               # exp of the sum of these stays near 1
    g = (size * sign).float().to(DEV).expand(B, T, D)
    ck = gdr.linear_scan_checkpoints(x)
    h, s = gdr.linear_scan_fwd(x, g, gated_input=True, out_dtype=F32, checkpoints=ck)
    dx, dg, _ = gdr.linear_scan_bwd(dh, x, g, ck, gated_input=True)
    a, m = g.double().exp(), -torch.expm1(g.double())
    state, past, states = torch.zeros(B, D, dtype=torch.float64, device=DEV), [], []
    for t in range(T):
        past.append(state)
        state = a[:, t] * state + m[:, t] * x[:, t].double()
        states.append(state)
    l, lx, lg = torch.zeros_like(state), [], []
    for t in reversed(range(T)):
        l = l + dh[:, t].double()
        lx.insert(0, l * m[:, t])
        lg.insert(0, l * a[:, t] * (past[t].abs() + x[:, t].double()))   # its terms' sizes
        l = l * a[:, t]
    tol = 5e-7 + 2.5e-7 * T
    for got, ref in ((h, torch.stack(states, 1)), (s, state), (dx, torch.stack(lx, 1))):
        check(got, ref, tol, ref.abs())
    size = torch.stack(lg, 1)
    ref = size / (torch.stack(past, 1).abs() + x.double()) * (torch.stack(past, 1) - x.double())
    check(dg, ref, 2 * tol, size)


def test_checkpoints_on_another_stream():
    """Memory that the current stream still reads is not given to checkpoints that another one
    fills."""
    x, g, _, dh, _ = scan_inputs(1, 65536, 1024, BF, F32, 81)
    ck = gdr.linear_scan_checkpoints(x)
    gdr.linear_scan_fwd(x, g, checkpoints=ck)
    want = gdr.linear_scan_bwd(dh, x, g, ck)
    out = torch.empty_like(x)
    old, copy = torch.full_like(ck, 3), torch.zeros_like(ck)
    big, side = torch.zeros(1 << 28, device=DEV), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        big.mul_(1.0)
    copy.copy_(old)
    del old
    ck = gdr.linear_scan_checkpoints(x, stream=side)
    gdr.linear_scan_fwd(x, g, out=out, checkpoints=ck, stream=side)
    got = gdr.linear_scan_bwd(dh, x, g, ck, stream=side)
    torch.cuda.synchronize()
    assert (copy == 3).all()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ empty caches
@pytest.mark.parametrize("dt,D", [(BF, 128), (F32, 64), (BF, 40)])
@pytest.mark.parametrize("pages,columns", [(0, 0), (3, 0), (0, 2), (0, 100)])
def test_empty_cache(pages, columns, dt, D):
    """No pages, or a table without columns: rows without keys give zeros and -inf, a row that
    says it has keys gives NaN, an append stores nothing and gives NaN."""
    kc = torch.full((pages, 16, 2, D), 3.0, dtype=dt, device=DEV)
    vc = kc.clone()
    table = torch.zeros(3, columns, dtype=torch.int32, device=DEV)
    q = rnd(gen_of(82), 3, 4, D, dtype=dt)
    lens = torch.tensor([0, 5, 0], dtype=torch.int32, device=DEV)
    o, lse = gdr.paged_decode_attn(q, kc, vc, table, lens)
    assert not o[[0, 2]].any() and (lse[[0, 2]] == -math.inf).all()
    assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
    qkv = rnd(gen_of(83), 3, 1, 8, D, dtype=dt)
    pos = torch.tensor([[0], [5], [1 << 30]], dtype=torch.int32, device=DEV)
    qo = gdr.qk_norm_rope_append(qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:], None, None, None,
                                 None, pos, kc, vc, table)
    assert torch.isnan(qo).all()
    assert (kc == 3).all() and (vc == 3).all()


# ------------------------------------------------------------------ branches of the dispatch
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("shape", [(64, 9, 512), (40, 31, 514), (33, 32, 777), (24, 33, 1024)])
def test_scan_wide_and_short(shape, dt, gated):
    """Channels for more blocks than the walk keeps resident, at the number of tokens (32) up to
    which a thread takes its channels by itself, pairs and single channels."""
    scan_check(*scan_inputs(*shape, dt, F32, 84), gated)


@pytest.mark.parametrize("dt,out", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("D,R,inter", [(128, 128, False), (96, 48, True), (30, 30, False), (33, 32, True)])
def test_qk_backward_of_mixed_types(D, R, inter, dt, out):
    """Upstream gradients of another type than q and k: all four gradients."""
    B, T, HQ, HK = 2, 37, 4, 2
    q, k, _, wq, wk, cos, sin, pos = qk_inputs(B, T, HQ, HK, D, R, dt, 85)
    d = rnd(gen_of(86), B, T, HQ, D, dtype=out), rnd(gen_of(87), B, T, HK, D, dtype=out)
    grads = gdr.qk_norm_rope_bwd(*d, q, k, wq, wk, cos, sin, pos, eps=1e-5, interleaved=inter)
    for x, w, dy, dx, dw in ((q, wq, d[0], grads[0], grads[2]), (k, wk, d[1], grads[1], grads[3])):
        xr, wr = x.double().requires_grad_(True), w.double().requires_grad_(True)
        rx, rw = torch.autograd.grad(qk_ref(xr, wr, cos, sin, pos, 1e-5, inter), (xr, wr), dy.double())
        unit = qk_ref(x, None, None, None, None, 1e-5, False)
        inv = (unit / x.double()).abs().nan_to_num(0.0).amax(-1, keepdim=True)
        terms = dy.double().abs().amax(-1, keepdim=True) * inv * 2
        assert dx.dtype == dt and dw.dtype == F32
        check(dx, rx, 4e-6 * max(1, D / 32), terms * unit.abs().amax(-1, keepdim=True).clamp_min(1))
        mags = (dy.double().abs().amax(-1, keepdim=True) * 2 * unit.abs()).sum((0, 1, 2))
        check(dw, rw, 4e-6, mags)
