"""Cases that time the operators a hybrid decoder runs beside the gated delta rule.

Three operators, each called the way a program calls it:

  linear_scan     h_t = exp(g_t) h_{t-1} + u_t per channel, u_t = x_t or (1 - exp(g_t)) x_t:
                  forward, training step (forward and backward), one token
  qk_norm_rope    RMS norm of every query and key head, then the position rotation:
                  forward, training step, and the serving form that writes the new keys
                  and values into a paged cache
  paged attention one new token per sequence against that cache

``own`` picks the side: the framework's entry points, or the same formulas in plain torch
operations in 32 bits. ``exact`` restates every formula in 64 bits, written separately.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SPARE_PAGES = 3      # pages of a cache that no sequence owns


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # The decode step of a recurrent layer: 64 sequences, 16 x 128 channels, one token
        # each. The call is a few microseconds: launch and host cost decide it.
        dict(name="scan_step_b64_d2048", op="scan_fwd", B=64, T=1, D=2048, dtype="bf16",
             gate="f32", gated=False, fused=False, state=True),
        # Prefill of one prompt at the headline width (12 x 128 channels), gates that also
        # scale the input; 24 column blocks alone do not fill the card, so T is split.
        dict(name="scan_prefill_t4096_d1536", op="scan_fwd", B=1, T=4096, D=1536, dtype="bf16",
             gate="f32", gated=True, fused=False, state=False),
        # One long document with a carried state, ragged against every tile: 2.1 GB through HBM.
        dict(name="scan_long_t65000_d4096", op="scan_fwd", B=1, T=65000, D=4096, dtype="bf16",
             gate="f32", gated=False, fused=False, state=True),
        # A training step of the same layer, 2 x 8192 tokens: forward, then all gradients.
        dict(name="scan_train_b2_t8192_d4096", op="scan_train", B=2, T=8192, D=4096, dtype="bf16",
             gate="f32", gated=True, fused=False, state=False),
        # A small 32-bit training step with sizes off every tile (3 x 1021 x 777).
        dict(name="scan_train_f32_odd", op="scan_train", B=3, T=1021, D=777, dtype="f32",
             gate="f32", gated=False, fused=False, state=True),
        # The attention layer's decode step before its attention: 64 new tokens, q, k and v as
        # views of one projection, keys and values written into their pages.
        dict(name="qk_append_b64_h16", op="qk_append", B=64, T=1, HQ=16, HK=4, D=128, R=128,
             dtype="bf16", interleaved=False, page=64, past=300),
        # Prefill, 2 x 8192 tokens, 32 query and 4 key heads, half of each head rotated.
        dict(name="qk_prefill_b2_t8192", op="qk_fwd", B=2, T=8192, HQ=32, HK=4, D=128, R=64,
             dtype="bf16", interleaved=False),
        # A training step at the headline shape: 4096 tokens, 12 heads, whole heads rotated.
        dict(name="qk_train_t4096_h12", op="qk_train", B=1, T=4096, HQ=12, HK=12, D=128, R=128,
             dtype="bf16", interleaved=False),
        # Serving a full batch: 64 sequences of mixed lengths up to 8192, 8 queries per key head.
        dict(name="attn_b64_ragged8192", op="attn", B=64, L=8192, HQ=32, HK=4, D=128, page=64,
             dtype="bf16", window=0),
        # One long document: a single row has to fill the card, split over its 65000 keys.
        dict(name="attn_b1_t65000", op="attn", B=1, L=65000, HQ=32, HK=16, D=128, page=64,
             dtype="bf16", window=0),
        # The start of a few chats: short caches, one query per key head, small pages.
        dict(name="attn_b4_short", op="attn", B=4, L=200, HQ=16, HK=16, D=128, page=16,
             dtype="bf16", window=0),
        # 32-bit caches with a sliding window, odd pages and grouped heads.
        dict(name="attn_f32_window", op="attn", B=5, L=2999, HQ=6, HK=3, D=64, page=48,
             dtype="f32", window=300),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_train", "qk_fwd", "qk_train", "qk_append", "attn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("scan"):
        B = _log(rng, 1, 64)
        D = _log(rng, 16, 4096)
        D = rng.choice([D, max(64, D // 64 * 64)])
        most = 65000 if op == "scan_fwd" else 16384
        T = _log(rng, 1, min(most, max(1, (1 << 26) // (B * D))))
        gate = rng.choice(["f32", "f32", "bf16"])
        return dict(op=op, B=B, T=T, D=D, dtype=dtype, gate=gate,
                    gated=rng.random() < 0.5, fused=rng.random() < 0.3,
                    state=rng.random() < 0.5)
    D = rng.choice([64, 128, 256, 80, 96])
    HK = rng.choice([1, 2, 3, 4, 8, 16])
    if op.startswith("qk"):
        HQ = HK * rng.choice([1, 2, 4, 8])
        R = rng.choice([D, D // 2])
        if op == "qk_append":
            return dict(op=op, B=_log(rng, 1, 128), T=rng.choice([1, 1, 1, 4]), HQ=HQ, HK=HK, D=D,
                        R=R, dtype=dtype, interleaved=rng.random() < 0.3,
                        page=rng.choice([16, 32, 64, 17]), past=_log(rng, 1, 1024))
        B = _log(rng, 1, 8)
        T = _log(rng, 1, max(1, min(16384, (1 << 26) // (B * (HQ + HK) * D))))
        return dict(op=op, B=B, T=T, HQ=HQ, HK=HK, D=D, R=R, dtype=dtype,
                    interleaved=rng.random() < 0.3)
    B = _log(rng, 1, 128)
    L = _log(rng, 1, max(64, min(65000, (1 << 27) // (B * HK * D))))
    return dict(op=op, B=B, L=L, HQ=HK * rng.choice([1, 2, 4, 5, 8, 16]), HK=HK, D=D,
                page=rng.choice([16, 32, 64, 128, 17]), dtype=dtype,
                window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))


# ------------------------------------------------------------------ inputs
def _lens(case, seed):
    """Cache lengths on the host: spread over 0..L, one of each end when there is room."""
    gen = torch.Generator().manual_seed(seed + 17)
    B, L = case["B"], case["L"]
    lens = torch.randint(0, L + 1, (B,), generator=gen)
    lens[0] = L
    if B > 2:
        lens[1] = 0
    return lens


def _pages(lens, page, most, gen):
    """(page table [B, pages of `most` tokens] with -1 where no page is owned, pages in the
    cache): a pool that holds every sequence at its longest, pages handed out in any order."""
    need = [(int(n) + page - 1) // page for n in lens]
    most = max(1, (most + page - 1) // page)
    total = len(need) * most + SPARE_PAGES
    order = torch.randperm(total, generator=gen)
    owned = torch.arange(most)[None, :] < torch.tensor(need)[:, None]
    table = torch.full((len(need), most), -1, dtype=torch.int32)
    table[owned] = order[: sum(need)].to(torch.int32)
    return table, total


def _rope_table(rows, R, dev):
    """cos and sin [rows, R / 2] of the usual geometric frequencies."""
    freq = 10000.0 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)
    angle = torch.arange(rows, device=dev, dtype=torch.float64)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed + 5)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    s = dict(case)
    if case["op"].startswith("scan"):
        B, T, D = case["B"], case["T"], case["D"]
        if case["fused"]:                      # x is a view of a wider projection
            s["x"] = randn(B, T, 2 * D, dtype=dt)[..., :D]
        else:
            s["x"] = randn(B, T, D, dtype=dt)
        # Log-decays of a recurrent layer: most channels forget over tens of tokens.
        g = torch.nn.functional.logsigmoid(randn(B, T, D).add_(3.0))
        s["g"] = g.to(DTYPES[case["gate"]])
        s["h0"] = randn(B, D) if case["state"] else None
        if case["op"] == "scan_train":
            s["dh"] = randn(B, T, D, dtype=dt)
            s["dfinal"] = randn(B, D) if case["state"] else None
        elif T == 1:                           # a decoder's fixed buffers
            s["out"] = torch.empty(B, T, D, dtype=dt, device=dev)
            s["final"] = torch.empty(B, D, device=dev)
        return s
    D = case["D"]
    if case["op"] == "attn":
        lens = _lens(case, seed)
        table, total = _pages(lens, case["page"], case["L"], cpu)
        s["lens"] = lens.to(torch.int32).to(dev)
        s["table"] = table.to(dev)
        s["k_cache"] = randn(total, case["page"], case["HK"], D, dtype=dt)
        s["v_cache"] = randn(total, case["page"], case["HK"], D, dtype=dt)
        s["q"] = randn(case["B"], case["HQ"], D, dtype=dt)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["B"], case["HQ"], device=dev)
        return s
    B, T, HQ, HK = case["B"], case["T"], case["HQ"], case["HK"]
    # q, k and v are views of one projection's output, as the layer has them.
    qkv = randn(B, T, (HQ + 2 * HK) * D, dtype=dt)
    s["q"] = qkv[..., : HQ * D].unflatten(-1, (HQ, D))
    s["k"] = qkv[..., HQ * D: (HQ + HK) * D].unflatten(-1, (HK, D))
    s["v"] = qkv[..., (HQ + HK) * D:].unflatten(-1, (HK, D))
    s["wq"] = randn(D).mul_(0.2).add_(1.0)
    s["wk"] = randn(D).mul_(0.2).add_(1.0)
    if case["op"] == "qk_append":
        past = torch.randint(0, case["past"] + 1, (B,), generator=cpu)
        table, total = _pages(past + T, case["page"], case["past"] + T, cpu)
        s["table"] = table.to(dev)
        s["k_cache"] = randn(total, case["page"], HK, D, dtype=dt)
        s["v_cache"] = randn(total, case["page"], HK, D, dtype=dt)
        s["pos"] = (past[:, None] + torch.arange(T)).to(torch.int32).to(dev)
        s["cos"], s["sin"] = _rope_table(case["past"] + T, case["R"], dev)
        s["q_out"] = torch.empty(B, T, HQ, D, dtype=dt, device=dev)
    else:
        s["pos"] = torch.arange(T, device=dev, dtype=torch.int32).expand(B, T).contiguous()
        s["cos"], s["sin"] = _rope_table(T, case["R"], dev)
        if case["op"] == "qk_train":
            s["dq"] = randn(B, T, HQ, D, dtype=dt)
            s["dk"] = randn(B, T, HK, D, dtype=dt)
    return s


# ------------------------------------------------------------------ one pass
EPS = 1e-6


def run(s):
    return _OWN[s["op"]](s) if own else _PLAIN[s["op"]](s)


def _own_scan_fwd(s):
    import chunkwise_gated_delta_gdr_gb300 as gdr
    return gdr.linear_scan_fwd(s["x"], s["g"], s["h0"], gated_input=s["gated"],
                               out=s.get("out"), final_state=s.get("final"))


def _own_scan_train(s):
    import chunkwise_gated_delta_gdr_gb300 as gdr
    ck = gdr.linear_scan_checkpoints(s["x"])
    h, final = gdr.linear_scan_fwd(s["x"], s["g"], s["h0"], gated_input=s["gated"], checkpoints=ck)
    dx, dg, dh0 = gdr.linear_scan_bwd(s["dh"], s["x"], s["g"], ck, s["dfinal"],
                                      gated_input=s["gated"])
    return h, final, dx, dg, dh0


def _own_qk_fwd(s):
    import chunkwise_gated_delta_gdr_gb300 as gdr
    return gdr.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"],
                            eps=EPS, interleaved=s["interleaved"])


def _own_qk_train(s):
    import chunkwise_gated_delta_gdr_gb300 as gdr
    fwd = gdr.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"],
                           eps=EPS, interleaved=s["interleaved"])
    bwd = gdr.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["cos"],
                               s["sin"], s["pos"], eps=EPS, interleaved=s["interleaved"])
    return tuple(fwd) + tuple(bwd)


def _own_qk_append(s):
    import chunkwise_gated_delta_gdr_gb300 as gdr
    q = gdr.qk_norm_rope_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"],
                                s["pos"], s["k_cache"], s["v_cache"], s["table"], eps=EPS,
                                interleaved=s["interleaved"], q_out=s["q_out"])
    return q, s["k_cache"], s["v_cache"]


def _own_attn(s):
    import chunkwise_gated_delta_gdr_gb300 as gdr
    if "ws" not in s:          # the scratch a decoder allocates once for its batch
        s["ws"] = torch.empty(gdr.paged_decode_attn_workspace_size(
            s["q"], s["k_cache"], s["table"]), dtype=torch.uint8, device=s["q"].device)
    return gdr.paged_decode_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                 window=s["window"], out=s["out"], lse=s["lse"],
                                 workspace=s["ws"])


# The plain forms.
def _scan(a, u):
    """Inclusive scan of h <- a h + u along dim 1 by doubling (log2 T elementwise steps)."""
    T, step = u.shape[1], 1
    while step < T:
        u[:, step:] += a[:, step:] * u[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    return u


def _scan_inputs(s):
    a = s["g"].float().exp()
    x = s["x"].float()
    u = (1 - a) * x if s["gated"] else x.clone()
    if s["h0"] is not None:
        u[:, 0] += a[:, 0] * s["h0"]
    return a, x, u


def _plain_scan_fwd(s):
    a, _, u = _scan_inputs(s)
    h = _scan(a, u)
    return h.to(s["x"].dtype), h[:, -1].clone()


def _plain_scan_train(s):
    a, x, u = _scan_inputs(s)
    h = _scan(a.clone(), u)
    # lam_t = dh_t + a_{t+1} lam_{t+1}: the same scan from the other end.
    lam = s["dh"].float().flip(1)
    if s["dfinal"] is not None:
        lam[:, 0] += s["dfinal"]
    later = torch.cat([torch.ones_like(a[:, :1]), a[:, 1:].flip(1)], 1)
    lam = _scan(later, lam).flip(1)
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]
    before = torch.cat([first, h[:, :-1]], 1)
    if s["gated"]:
        dx, dg = lam * (1 - a), lam * a * (before - x)
    else:
        dx, dg = lam, lam * a * before
    return (h.to(s["x"].dtype), h[:, -1].clone(), dx.to(s["x"].dtype), dg.to(s["g"].dtype),
            lam[:, 0] * a[:, 0])


def _rotate(y, s, back=False):
    """Rotate the first R channels of y [B, T, H, D] by each token's angle."""
    R = 2 * s["cos"].shape[1]
    c, n = s["cos"][s["pos"].long()][:, :, None], s["sin"][s["pos"].long()][:, :, None]
    n = -n if back else n
    if s["interleaved"]:
        p, q = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack([p * c - q * n, q * c + p * n], -1).flatten(-2)
    else:
        p, q = y[..., : R // 2], y[..., R // 2: R]
        turned = torch.cat([p * c - q * n, q * c + p * n], -1)
    return torch.cat([turned, y[..., R:]], -1)


def _norm(x):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _plain_qk_fwd(s):
    return tuple(_rotate(_norm(s[n])[0] * s["w" + n], s).to(s[n].dtype) for n in ("q", "k"))


def _plain_qk_train(s):
    outs, grads, weights = [], [], []
    for n in ("q", "k"):
        unit, r = _norm(s[n])
        outs.append(_rotate(unit * s["w" + n], s).to(s[n].dtype))
        d = _rotate(s["d" + n].float(), s, back=True)
        weights.append((d * unit).sum((0, 1, 2)))
        d = d * s["w" + n]
        grads.append((r * (d - unit * (d * unit).mean(-1, keepdim=True))).to(s[n].dtype))
    return tuple(outs + grads + weights)


def _plain_qk_append(s):
    q, k = _plain_qk_fwd(s)
    pos = s["pos"].long()
    page = torch.gather(s["table"].long(), 1, pos // s["page"])
    s["k_cache"][page, pos % s["page"]] = k
    s["v_cache"][page, pos % s["page"]] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _plain_attn(s):
    B, HQ, D = s["q"].shape
    page, HK = s["page"], s["HK"]
    table = s["table"].long().clamp_min(0)
    keys = torch.arange(table.shape[1] * page, device=table.device)
    lens = s["lens"].long()[:, None]
    live = keys < lens
    if s["window"]:
        live &= keys >= lens - s["window"]
    k = s["k_cache"][table].flatten(1, 2).float()
    v = s["v_cache"][table].flatten(1, 2).float()
    v = torch.where(live[:, :, None, None], v, torch.zeros((), device=v.device))
    q = s["q"].float().view(B, HK, HQ // HK, D) * (1.0 / math.sqrt(D))
    score = torch.einsum("bhgd,bnhd->bhgn", q, k)
    score = torch.where(live[:, None, None], score, score.new_tensor(-math.inf))
    top = score.max(-1, keepdim=True).values
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgn,bnhd->bhgd", p, v)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))
    return o.view(B, HQ, D).to(s["q"].dtype), lse.view(B, HQ)


_OWN = dict(scan_fwd=_own_scan_fwd, scan_train=_own_scan_train, qk_fwd=_own_qk_fwd,
            qk_train=_own_qk_train, qk_append=_own_qk_append, attn=_own_attn)
_PLAIN = dict(scan_fwd=_plain_scan_fwd, scan_train=_plain_scan_train, qk_fwd=_plain_qk_fwd,
              qk_train=_plain_qk_train, qk_append=_plain_qk_append, attn=_plain_attn)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("scan"):
        n = case["B"] * case["T"] * case["D"]
        ge = 2 if case["gate"] == "bf16" else 4
        ends = case["B"] * case["D"] * 4 * (2 if case["state"] else 1)
        if case["op"] == "scan_fwd":
            return {"bytes": n * (2 * e + ge) + ends, "flops": 4 * n}
        # forward: x, g in, h out; backward: dh, x, g in, dx, dg out; states and their gradients
        return {"bytes": n * (2 * e + ge) + n * (3 * e + 2 * ge) + 2 * ends, "flops": 14 * n}
    D = case["D"]
    if case["op"] == "attn":
        # Lengths differ by seed: their mean over 0..L, one of them L and one 0.
        B, L = case["B"], case["L"]
        keys = [L] + ([0] if B > 2 else []) + [L / 2] * (B - (2 if B > 2 else 1))
        W = case["window"]
        if W:
            keys = [min(n, W) if n in (0, L) else _mean_windowed(L, W) for n in keys]
        total = sum(keys)
        return {"bytes": 2 * total * case["HK"] * D * e + 2 * B * case["HQ"] * D * e
                + 4 * B * case["HQ"], "flops": 4 * total * case["HQ"] * D}
    tok, heads = case["B"] * case["T"], case["HQ"] + case["HK"]
    table = min(tok, case["T"] if case["op"] != "qk_append" else tok) * case["R"] * 4
    io = tok * heads * D * e
    if case["op"] == "qk_fwd":
        return {"bytes": 2 * io + table, "flops": 8 * tok * heads * D}
    if case["op"] == "qk_append":
        return {"bytes": 2 * io + 2 * tok * case["HK"] * D * e + table,
                "flops": 8 * tok * heads * D}
    return {"bytes": 2 * io + 3 * io + 2 * table, "flops": 24 * tok * heads * D}


def _mean_windowed(L, W):
    """Mean of min(n, W) over n = 0..L."""
    W = min(W, L)
    return (W * (W + 1) / 2 + (L - W) * W) / (L + 1)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"scan_fwd": _exact_scan, "scan_train": _exact_scan, "qk_fwd": _exact_qk,
            "qk_train": _exact_qk, "qk_append": _exact_qk, "attn": _exact_attn}[case["op"]](s)


def _exact_scan(s):
    """The recurrence token by token, and its adjoint token by token from the last."""
    x, g = s["x"].double(), s["g"].double()
    B, T, D = x.shape
    a = torch.exp(g)
    m = -torch.expm1(g) if s["gated"] else torch.ones_like(g)
    state = torch.zeros(B, D, dtype=torch.float64, device=x.device)
    if s["h0"] is not None:
        state = s["h0"].double()
    start, h = state, torch.empty_like(x)
    for t in range(T):
        state = torch.addcmul(m[:, t] * x[:, t], a[:, t], state)
        h[:, t] = state
    if s["op"] == "scan_fwd":
        return h, state
    dx, dg = torch.empty_like(x), torch.empty_like(x)
    lam = torch.zeros_like(state) if s["dfinal"] is None else s["dfinal"].double()
    for t in reversed(range(T)):
        lam = lam + s["dh"][:, t].double()
        past = h[:, t - 1] if t else start
        dx[:, t] = lam * m[:, t]
        dm = -a[:, t] * x[:, t] if s["gated"] else 0.0
        dg[:, t] = lam * (a[:, t] * past + dm)
        lam = lam * a[:, t]
    return h, state, dx, dg, lam


def _exact_qk(s):
    """The rotation as a product of complex numbers; gradients by differentiating it."""
    R = 2 * s["cos"].shape[1]
    rows = s["pos"].long()
    turn = torch.complex(s["cos"].double(), s["sin"].double())[rows][:, :, None]

    def forward(x, w):
        y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w
        head, tail = y[..., :R], y[..., R:]
        if s["interleaved"]:
            pair = head.unflatten(-1, (R // 2, 2))
            z = torch.complex(pair[..., 0], pair[..., 1]) * turn
            head = torch.view_as_real(z).flatten(-2)
        else:
            pair = head.unflatten(-1, (2, R // 2))
            z = torch.complex(pair[..., 0, :], pair[..., 1, :]) * turn
            head = torch.cat([z.real, z.imag], -1)
        return torch.cat([head, tail], -1)

    outs, grads, weights = [], [], []
    for n in ("q", "k"):
        x, w = s[n].double().requires_grad_(True), s["w" + n].double().requires_grad_(True)
        y = forward(x, w)
        outs.append(y.detach())
        if s["op"] == "qk_train":
            dx, dw = torch.autograd.grad(y, (x, w), s["d" + n].double())
            grads.append(dx)
            weights.append(dw)
    if s["op"] != "qk_append":
        return tuple(outs + grads + weights)
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    table, where = s["table"].tolist(), s["pos"].tolist()
    for b in range(s["B"]):
        for t in range(s["T"]):
            slot, at = table[b][where[b][t] // s["page"]], where[b][t] % s["page"]
            k_cache[slot, at] = outs[1][b, t]
            v_cache[slot, at] = s["v"][b, t].double()
    return outs[0], k_cache, v_cache


def _exact_attn(s):
    """Sequence by sequence: its own keys gathered, one softmax over all of them."""
    B, HQ, D = s["q"].shape
    G = HQ // s["HK"]
    o = torch.zeros(B, HQ, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, HQ), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - s["window"]) if s["window"] else 0
        if n <= lo:
            continue
        at = torch.arange(lo, n, device=s["q"].device)
        page, row = s["table"][b].long()[at // s["page"]], at % s["page"]
        k = s["k_cache"][page, row].double().permute(1, 0, 2)            # [HK, n, D]
        v = s["v_cache"][page, row].double().permute(1, 0, 2)
        q = s["q"][b].double().view(s["HK"], G, D)
        z = q @ k.transpose(1, 2) / math.sqrt(D)
        o[b] = (torch.softmax(z, -1) @ v).reshape(HQ, D)
        lse[b] = torch.logsumexp(z, -1).reshape(HQ)
    return o, lse
