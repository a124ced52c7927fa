"""GPU numerics of the attention behind a shared prompt, against a plain 64-bit one.

Tolerances. fp32 scores of |s| < 40 are within 40 * 16 * 2^-24 < 4e-5 of themselves, and so is
every weight; on the tensor cores (bf16 q and caches) a weight goes into the product with V as
two bf16, which loses 2^-15 of it at most: (4e-5 [+ 2^-15]) sum p |v| / sum p. A bf16 result has
to be the rounding of a value within that.
"""
import math

import pytest
import torch

import chunkwise_gated_delta_gdr_gb300 as gdr

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"


def rnd(gen, *shape, dtype=F32):
    return torch.randn(*shape, generator=gen, dtype=F32).to(dtype).to(DEV)


def make(B, HQ, HK, D, P, lens, page=16, dtype=BF, qtype=None, seed=0, spare=2, prefix_spare=0,
         layout="pthd"):
    gen = torch.Generator().manual_seed(seed)
    first = -(-P // page) + prefix_spare
    cols = max(1, max(-(-n // page) for n in lens))
    total = first + B * cols + spare
    order = torch.randperm(total, generator=gen).int()
    table = torch.full((B, cols), -1, dtype=torch.int32)
    at = first
    for b, n in enumerate(lens):
        k = -(-n // page)
        table[b, :k] = order[at:at + k]
        at += k
    if layout == "phtd":
        kc, vc = (rnd(gen, total, HK, page, D, dtype=dtype).transpose(1, 2) for _ in range(2))
    elif layout == "wide":          # rows of a wider array, D + 1 apart: no 16-byte pieces
        kc, vc = (rnd(gen, total, page, HK, D + 1, dtype=dtype)[..., :D] for _ in range(2))
    else:
        kc, vc = (rnd(gen, total, page, HK, D, dtype=dtype) for _ in range(2))
    return dict(q=rnd(gen, B, HQ, D, dtype=qtype or dtype), kc=kc, vc=vc,
                prefix=order[:first].to(DEV), P=P, table=table.to(DEV),
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV))


def call(s, **kw):
    return gdr.paged_prefix_attn(s["q"], s["kc"], s["vc"], s["prefix"], s["P"], s["table"],
                                 s["lens"], **kw)


def rows_of(s, table, n):
    page = s["kc"].shape[1]
    at = torch.arange(n, device=DEV)
    pages = table.long()[at // page] if n else at
    return s["kc"][pages, at % page].double(), s["vc"][pages, at % page].double()


def reference(s, scale=None):
    """(o, lse, sum p |v| / sum p)."""
    B, HQ, D = s["q"].shape
    HK = s["kc"].shape[2]
    scale = 1 / math.sqrt(D) if scale is None else scale
    kp, vp = rows_of(s, s["prefix"], s["P"])
    o = torch.zeros(B, HQ, D, dtype=torch.float64, device=DEV)
    size, lse = o.clone(), torch.full((B, HQ), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        k, v = rows_of(s, s["table"][b], n)
        k, v = torch.cat([kp, k]).permute(1, 0, 2), torch.cat([vp, v]).permute(1, 0, 2)
        if k.shape[1] == 0:
            continue
        z = s["q"][b].double().view(HK, HQ // HK, D) @ k.transpose(1, 2) * scale
        p = torch.softmax(z, -1)
        o[b], size[b] = (p @ v).reshape(HQ, D), (p @ v.abs()).reshape(HQ, D)
        lse[b] = torch.logsumexp(z, -1).reshape(HQ)
    return o, lse, size


def check(s, got=None, scale=None, **kw):
    o, lse = call(s, **({} if scale is None else dict(scale=scale)), **kw) if got is None else got
    ref, rlse, size = reference(s, scale)
    tol = 4e-5 + (2.0 ** -15 if s["q"].dtype == s["kc"].dtype == BF else 0)
    lo, hi = ((ref + k * tol * size).to(o.dtype).double() for k in (-1, 1))
    over = torch.maximum(o.double() - hi, lo - o.double())
    assert not torch.isnan(over).any()
    assert over.max().item() <= 0, f"exceeds its bound by {over.max().item():.3e}"
    assert torch.equal(torch.isinf(lse), torch.isinf(rlse))
    live = torch.isfinite(rlse)
    assert ((lse.double() - rlse)[live].abs() <= 4e-5 + 4e-7 * rlse[live].abs()).all()
    return o, lse


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 80, 96, 128, 192, 256, 8, 40, 72, 136, 200, 1, 33])
def test_head_dims(D, dtype):
    check(make(3, 4, 2, D, 333, [0, 17, 40], dtype=dtype, seed=D))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,HQ,HK", [(1, 1, 1), (1, 16, 16), (5, 6, 3), (2, 40, 8), (70, 8, 2),
                                     (33, 16, 1), (129, 2, 1), (300, 3, 3), (64, 32, 4)])
def test_rows(B, HQ, HK, dtype):
    """Rows of a key head from one to several tiles, ragged."""
    check(make(B, HQ, HK, 64, 700, [(7 * b) % 50 for b in range(B)], dtype=dtype, seed=B))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P", [1, 2, 15, 16, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 5003])
def test_prefix_lengths(P, dtype):
    check(make(2, 4, 2, 128, P, [3, 0], dtype=dtype, seed=P))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [1, 7, 16, 17, 48, 64, 100, 128, 1024])
def test_pages(page, dtype):
    check(make(3, 4, 1, 64, 900, [30, 0, 2000], page=page, dtype=dtype, seed=page))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,HQ,HK,P", [(64, 32, 16, 3000), (200, 8, 8, 6000), (40, 16, 2, 20000),
                                       (1, 2, 2, 40000)])
def test_long_prefixes(B, HQ, HK, P, D):
    """Stretches of many tiles, items cut by the blocks' stretches."""
    check(make(B, HQ, HK, D, P, [(11 * b) % 90 for b in range(B)], page=64, seed=P))


def test_more_items_than_blocks():
    """Blocks that take several whole items, and parts of others."""
    check(make(260, 64, 64, 64, 200, [b % 20 for b in range(260)], seed=1))
    check(make(1, 400, 400, 64, 300, [9], seed=2))


@pytest.mark.parametrize("layout", ["pthd", "phtd", "wide"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layouts(layout, dtype):
    check(make(3, 4, 2, 64, 200, [5, 0, 30], dtype=dtype, layout=layout, seed=4))


@pytest.mark.parametrize("D", [64, 128])
def test_queries_as_views(D):
    s = make(3, 4, 2, D, 200, [5, 0, 30], seed=5)
    wide = rnd(torch.Generator().manual_seed(1), 3, 4, 2 * D + 3, dtype=BF)
    for off in (0, 1, 3, D):
        s["q"] = wide[..., off:off + D]
        check(s)
    s["q"] = rnd(torch.Generator().manual_seed(2), 4, 3, D, dtype=BF).transpose(0, 1)
    check(s)
    s["q"] = rnd(torch.Generator().manual_seed(3), 1, 4, D, dtype=BF).expand(3, 4, D)
    check(s)


@pytest.mark.parametrize("qt,ct,ot", [(BF, BF, F32), (F32, BF, F32), (BF, F32, BF), (F32, F32, BF)])
def test_types(qt, ct, ot):
    s = make(5, 4, 2, 128, 500, [5, 0, 30, 64, 1], dtype=ct, qtype=qt, seed=6)
    assert check(s, out_dtype=ot)[0].dtype == ot


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scale_and_growing_scores(dtype):
    """Scores that rise along the keys by hundreds, so that the running maximum moves all the
    way; and a single key that outweighs all others at either end."""
    s = make(4, 4, 2, 128, 1500, [0, 5, 100, 300], dtype=dtype, seed=7)
    check(s, scale=0.02)
    base = s["kc"].clone()
    flat, page = s["prefix"].long(), s["kc"].shape[1]
    ramp = torch.linspace(-1, 1, s["P"], device=DEV)
    at = torch.arange(s["P"], device=DEV)
    s["q"] = s["q"].abs().clamp(0.5, 1.0)
    for sign in (1, -1):
        s["kc"] = base.clone()
        s["kc"][flat[at // page], at % page] += (sign * 3 * ramp)[:, None, None].to(dtype)
        check(s, scale=1.0 / 12)
    for j in (0, 1499):
        s["kc"] = base.clone()
        s["kc"][flat[j // page], j % page] += 3.0
        check(s, scale=1.0 / 12)


@pytest.mark.parametrize("D", [64, 72])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinities_and_nan(dtype, D):
    """-inf in a query's only channel shuts keys out; infinite values come through; what no
    sequence owns is never read."""
    s = make(3, 2, 1, D, 150, [0, 10, 33], dtype=dtype, seed=8, spare=3, prefix_spare=1)
    used = torch.cat([s["prefix"][:-(-150 // 16)].long(), s["table"][s["table"] >= 0].long()])
    free = torch.ones(len(s["kc"]), dtype=torch.bool, device=DEV)
    free[used] = False
    s["kc"][free], s["vc"][free] = float("nan"), float("inf")
    # behind the prompt's end in its last page, too
    s["kc"][s["prefix"][9].long(), 150 - 144:] = float("nan")
    s["vc"][s["prefix"][9].long(), 150 - 144:] = float("inf")
    o, lse = check(s)
    # An infinite value of a key with a weight that is not 0.
    s["vc"][s["prefix"][3].long(), 5, 0, 2] = float("inf")
    got, _ = call(s)
    assert (got[:, :, 2] == float("inf")).all()
    keep = [i for i in range(D) if i != 2]
    assert torch.equal(got[..., keep], o[..., keep])
    # A NaN key: every sequence's row.
    s["kc"][s["prefix"][3].long(), 5, 0, 0] = float("nan")
    assert torch.isnan(call(s)[0]).all()


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64), (BF, 40)])
def test_keys_shut_out(dtype, D):
    """Keys whose score is -inf: in part of the prompt, in all of it, and everywhere."""
    s = make(3, 2, 1, D, 300, [0, 10, 33], dtype=dtype, seed=9)
    s["q"][..., 0] = 1.0
    full = s["kc"].clone()
    page, at = s["kc"].shape[1], torch.arange(300, device=DEV)
    rows = s["prefix"].long()[at // page]
    for part in (at < 200, at >= 70, at >= 0):
        s["kc"] = full.clone()
        s["kc"][rows[part], (at % page)[part], :, 0] = -math.inf
        o, lse = call(s)
        ref, rlse, size = reference(s)
        none = torch.isinf(rlse)                 # no key left
        assert torch.equal(torch.isinf(lse), none) and (o[none] == 0).all()
        tol = (4e-5 + 2.0 ** -15) * size[~none] + (2.0 ** -8 * ref[~none].abs() if dtype == BF else 0)
        assert ((o.double() - ref)[~none].abs() <= tol).all()


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64), (BF, 40)])
def test_out_of_range(dtype, D):
    s = make(4, 4, 2, D, 200, [5, 0, 30, 7], dtype=dtype, seed=10)
    want, wlse = call(s)
    own = dict(s, table=s["table"].clone(), lens=s["lens"].clone())
    own["table"][0, 0] = len(s["kc"])
    own["lens"][2] = own["table"].shape[1] * 16 + 1
    o, lse = call(own)
    for b in (0, 2):
        assert torch.isnan(o[b]).all() and torch.isnan(lse[b]).all()
    for b in (1, 3):
        assert torch.equal(o[b], want[b]) and torch.equal(lse[b], wlse[b])
    for page in (-1, len(s["kc"])):
        bad = dict(s, prefix=s["prefix"].clone())
        bad["prefix"][7] = page
        o, lse = call(bad)
        assert torch.isnan(o).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_without_shared_or_own_keys(dtype):
    s = make(4, 4, 2, 128, 0, [5, 0, 30, 7], dtype=dtype, seed=11)
    o, lse = check(s)
    want = gdr.paged_decode_attn(s["q"], s["kc"], s["vc"], s["table"], s["lens"])
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    check(make(4, 4, 2, 128, 300, [0, 0, 0, 0], dtype=dtype, seed=12))
    s = make(2, 4, 2, 128, 300, [0, 0], dtype=dtype, seed=12)
    s["table"] = s["table"][:, :0].contiguous()
    check(s)
    s["q"], s["table"], s["lens"] = s["q"][:0], s["table"][:0], s["lens"][:0]
    assert call(s)[0].shape == (0, 4, 128)


def test_equals_one_table_per_sequence():
    """Against paged_decode_attn with the prompt's pages at the front of every table: the same
    keys, so the same result up to both calls' tolerances."""
    s = make(20, 8, 2, 128, 640, [(7 * b) % 50 for b in range(20)], seed=13)
    whole = torch.cat([s["prefix"][:40].repeat(20, 1), s["table"]], 1).contiguous()
    o, lse = call(s, out_dtype=F32)
    o2, lse2 = gdr.paged_decode_attn(s["q"], s["kc"], s["vc"], whole, s["lens"] + 640,
                                     out_dtype=F32)
    _, _, size = reference(s)
    assert ((o - o2).abs() <= 2 * (4e-5 + 2.0 ** -15) * size).all()
    assert (lse - lse2).abs().max() <= 1e-4


def test_offsets_beyond_32_bits():
    """Pages whose elements lie past 2^31 (a page stride of 2^26 elements)."""
    stride, pages, page, HK, D = 1 << 26, 40, 16, 2, 64
    pool = torch.empty(pages * stride, dtype=BF, device=DEV)
    kc = pool.as_strided((pages, page, HK, D), (stride, HK * D, D, 1))
    vc = pool[1 << 20:].as_strided((pages, page, HK, D), (stride, HK * D, D, 1))
    s = make(3, 4, HK, D, 300, [5, 0, 100], page=page, seed=14, spare=pages - 19 - 21)
    assert len(s["kc"]) == pages
    kc.copy_(s["kc"])
    vc.copy_(s["vc"])
    want = call(s)
    s["kc"], s["vc"] = kc, vc
    for a, b in zip(want, call(s)):
        assert torch.equal(a, b)


def test_runs_are_equal_and_outputs_are_used():
    s = make(30, 8, 2, 128, 3000, [(7 * b) % 50 for b in range(30)], seed=15)
    out, lse = torch.empty_like(s["q"]), torch.empty(30, 8, device=DEV)
    ws = torch.empty(gdr.paged_prefix_attn_workspace_size(s["q"], s["kc"], s["prefix"], s["P"],
                                                          s["table"]), dtype=torch.uint8, device=DEV)
    a = call(s)
    ws.fill_(255)
    b = call(s, out=out, lse=lse, workspace=ws)
    assert b[0] is out and b[1] is lse
    assert torch.equal(a[0], out) and torch.equal(a[1], lse)


def test_another_stream_and_capture():
    s = make(30, 8, 2, 128, 3000, [(7 * b) % 50 for b in range(30)], seed=16)
    want = call(s)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = call(s, stream=stream)
    stream.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call(s)
    gen = torch.Generator().manual_seed(3)
    for _ in range(2):
        s["q"].copy_(rnd(gen, *s["q"].shape))
        s["lens"].copy_(torch.randint(0, 40, (30,), generator=gen))
        s["table"].clamp_(min=0)
        graph.replay()
        for a, b in zip(held, call(s)):
            assert torch.equal(a, b)


def test_compiled_and_python_calls_agree(monkeypatch):
    from chunkwise_gated_delta_gdr_gb300 import layers
    s = make(5, 8, 2, 128, 300, [5, 0, 30, 7, 1], seed=17)
    want = call(s)
    monkeypatch.setattr(layers, "_host", None)
    for a, b in zip(want, call(s)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("compiled", [True, False])
def test_refusals_on_the_gpu(compiled, monkeypatch):
    from chunkwise_gated_delta_gdr_gb300 import layers
    if not compiled:
        monkeypatch.setattr(layers, "_host", None)
    s = make(3, 4, 2, 64, 100, [5, 0, 30], seed=18)
    for error, kw in [(ValueError, dict(prefix=s["prefix"][None])),
                      (TypeError, dict(prefix=s["prefix"].long())),
                      (ValueError, dict(prefix=s["prefix"].cpu())),
                      (ValueError, dict(prefix=s["prefix"].repeat(2)[::2])),
                      (ValueError, dict(P=-1)), (ValueError, dict(P=1 << 31)),
                      (ValueError, dict(P=5.0)),
                      (gdr.GdrError, dict(P=16 * len(s["prefix"]) + 1)),
                      (ValueError, dict(lens=s["lens"][:2])),
                      (ValueError, dict(table=s["table"][:2])),
                      (ValueError, dict(q=s["q"][..., :32])),
                      (gdr.GdrError, dict(q=s["q"][:, :3]))]:
        with pytest.raises(error):
            call({**s, **kw})
    with pytest.raises(gdr.GdrError):
        call(s, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        call(s, out=torch.empty_like(s["q"]), out_dtype=F32)
    check(s)


@pytest.mark.parametrize("D,B,HQ,HK,P,page", [(128, 64, 16, 4, 5000, 64), (128, 3, 4, 2, 5000, 64),
                                              (64, 200, 2, 2, 900, 17), (256, 40, 8, 2, 3001, 128)])
def test_waits_that_give_up(D, B, HQ, HK, P, page):
    """With few polls allowed the kernel's waits give up: every result is NaN or has its right
    bits, the launch ends by itself, and calls with the usual bound are as ever."""
    s = make(B, HQ, HK, D, P, [(7 * b) % 40 for b in range(B)], page=page, seed=19)
    want = call(s)
    old = gdr.set_flag_wait_limit(-1)
    for polls in (0, 0, 16, 32, 128, 1024):      # a sixteenth of them per wait
        gdr.set_flag_wait_limit(polls)
        try:
            got = call(s, out=torch.full_like(s["q"], 7),
                       lse=torch.full((B, HQ), 7.0, device=DEV))
            torch.cuda.synchronize()
        finally:
            gdr.set_flag_wait_limit(old)
        for a, b in zip(got, want):
            there = ~torch.isnan(a)
            assert torch.equal(a[there], b[there]), polls
        if polls == 0:                           # a tile needs a microsecond
            assert torch.isnan(got[0]).any() and torch.isnan(got[1]).any()
    for a, b in zip(call(s), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64), (BF, 40)])
def test_prompt_in_an_empty_cache(dtype, D):
    """A cache without pages has no page that a prompt could name: NaN, and nothing is read."""
    s = make(3, 4, 2, D, 40, [0, 0, 0], dtype=dtype, seed=20)
    s["kc"], s["vc"] = s["kc"][:0], s["vc"][:0]
    o, lse = call(s)
    assert torch.isnan(o).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("page", [16, 64])
def test_broadcast_heads(page):
    """Key heads that are one head (a stride of 0 between them)."""
    s = make(9, 8, 1, 128, 300, [5, 0, 30, 64, 1, 2, 3, 4, 5], page=page, seed=21)
    want = call(s)
    s["kc"], s["vc"] = (t.expand(-1, -1, 4, -1) for t in (s["kc"], s["vc"]))
    ref, _, size = reference(s)
    o, _ = check(s)
    assert ((o.double() - want[0].double()).abs() <= 2 * (2.0 ** -8 * ref.abs() + 1e-4 * size)).all()


def test_two_calls_at_once():
    """Calls on two streams that run side by side, each with its own inputs and scratch."""
    cases = [make(64, 16, 4, 128, 4000, [(7 * b) % 90 for b in range(64)], page=64, seed=22),
             make(9, 8, 2, 128, 6000, [(5 * b) % 40 for b in range(9)], page=17, seed=23)]
    want = [call(s) for s in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for s, stream in zip(cases, streams):
            with torch.cuda.stream(stream):
                x = s["q"].unsqueeze(1)
                y = gdr.gated_norm(x, x)
                got.append((call(s), y, gdr.residual_norm(y.flatten(2), x.flatten(2))[0]))
        torch.cuda.synchronize()
        for s, w, (g, y, r) in zip(cases, want, got):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
            x = s["q"].unsqueeze(1)
            again = gdr.gated_norm(x, x)
            assert torch.equal(y, again)
            assert torch.equal(r, gdr.residual_norm(again.flatten(2), x.flatten(2))[0])


@pytest.mark.parametrize("dtype,D,page,P", [(BF, 128, 64, 3000), (BF, 64, 17, 700), (F32, 64, 16, 900),
                                            (BF, 40, 16, 300), (BF, 128, 16, 0)])
def test_inputs_written_just_before(dtype, D, page, P):
    """Queries, keys, tables and lengths that the kernels right before write, one of which lets
    the next one begin at once, in a queue that the device is behind with: the bits of the same
    calls waited for one by one. With own keys of several blocks, whose parts are joined, too."""
    B, HQ, HK, n = 20, 8, 2, 6
    s = make(B, HQ, HK, D, P, [(131 * b) % 2000 for b in range(B)], page=page, dtype=dtype, seed=24)
    gen = torch.Generator().manual_seed(25)
    q = rnd(gen, n, B, 1, HQ, D, dtype=dtype)
    z = rnd(gen, n, B, 1, HQ, D, dtype=dtype)
    k, v = (rnd(gen, n, B, 1, HK, D, dtype=dtype) for _ in range(2))
    lens = torch.stack([torch.randperm(B, generator=gen).to(DEV) for _ in range(n)])
    lens, tables = s["lens"].clone()[lens], s["table"][lens]
    kc, vc = s["kc"].clone(), s["vc"].clone()
    # The table of the sequence that a length came from; each sequence's last key is new.
    held = [dict(s, kc=kc.clone(), vc=vc.clone(), table=s["table"].clone(), lens=s["lens"].clone())
            for _ in range(n)]
    busy = rnd(gen, 1, 1 << 14, 8, 128)

    def step(i, wait):
        h = held[i]
        h["kc"].copy_(kc), h["vc"].copy_(vc)
        h["table"].copy_(tables[i]), h["lens"].copy_(lens[i])
        pos = (h["lens"] - 1)[:, None].contiguous()
        gdr.qk_norm_rope_append(q[i], k[i], v[i], None, None, None, None, pos, h["kc"], h["vc"],
                                h["table"])
        h["q"] = gdr.gated_norm(q[i], z[i])[:, 0]
        if wait:
            torch.cuda.synchronize()
        out = [call(h), gdr.paged_decode_attn(h["q"], h["kc"], h["vc"], h["table"], h["lens"])]
        if wait:
            torch.cuda.synchronize()
        return [t for pair in out for t in pair]

    want = [[t.clone() for t in step(i, True)] for i in range(n)]
    for _ in range(3):
        for h in held:                           # nothing of the last round is left to be found
            h["kc"].zero_(), h["vc"].zero_(), h["lens"].zero_(), h["table"].fill_(-1)
        torch.cuda.synchronize()
        gdr.gated_norm(busy, busy)
        got = [step(i, False) for i in range(n)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_capture_behind_copies_and_another_stream():
    """Calls captured behind a copy, a fill and another stream's kernel, as a program's first
    kernels are; the replays take what those leave."""
    s = make(9, 8, 2, 128, 1000, [(131 * b) % 900 for b in range(9)], page=64, seed=26)
    source, x = s["q"].clone(), torch.zeros(9, 1, 8, 128, dtype=BF, device=DEV)
    side = torch.cuda.Stream()
    state = torch.zeros(9, 1024, dtype=F32, device=DEV)

    def run():
        main = torch.cuda.current_stream()
        x.zero_()
        y = gdr.gated_norm(x, x, activation="sigmoid")               # behind a fill
        s["q"].copy_(source)
        a = call(s)                                                  # behind a copy
        side.wait_stream(main)
        with torch.cuda.stream(side):
            g = a[0].unsqueeze(1) * 2
        state.add_(1)
        main.wait_stream(side)
        z = gdr.gated_norm(g, g)                                     # behind both streams
        side.wait_stream(main)
        with torch.cuda.stream(side):
            w = gdr.residual_norm(state.view(9, 1, 1024), z.flatten(2))
        main.wait_stream(side)
        b = gdr.paged_decode_attn(z[:, 0], s["kc"], s["vc"], s["table"], s["lens"])
        return [y, *a, z, *w, *b]

    run()
    state.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    gen = torch.Generator().manual_seed(27)
    for _ in range(3):
        source.copy_(rnd(gen, *source.shape))
        before = state.clone()
        graph.replay()
        got = [t.clone() for t in held]
        state.copy_(before)
        for a, b in zip(got, run()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 256), (F32, 64), (BF, 40)])
def test_keys_shut_out_to_the_rounding(dtype, D, ot):
    """Keys whose score is -inf in part of the prompt, in all of it and everywhere: rows with a key
    left are the rounding of a value within the bound, as everywhere, and so is their lse."""
    s = make(3, 2, 1, D, 300, [0, 10, 33], dtype=dtype, seed=28)
    s["q"][..., 0] = 1.0
    full = s["kc"].clone()
    page, at = s["kc"].shape[1], torch.arange(300, device=DEV)
    rows = s["prefix"].long()[at // page]
    for part in (at < 200, at >= 70, at % 3 != 1, at >= 0):
        s["kc"] = full.clone()
        s["kc"][rows[part], (at % page)[part], :, 0] = -math.inf
        o, lse = call(s, out_dtype=ot)
        ref, rlse, size = reference(s)
        live = torch.isfinite(rlse)
        assert (o[~live] == 0).all() and (lse[~live] == -math.inf).all()
        tol = 4e-5 + (2.0 ** -15 if dtype == BF and D != 40 else 0)
        lo, hi = ((ref + k * tol * size).to(ot).double()[live] for k in (-1, 1))
        assert ((o.double()[live] <= hi) & (o.double()[live] >= lo)).all()
        assert ((lse.double() - rlse)[live].abs() <= 4e-5 + 4e-7 * rlse[live].abs()).all()
