"""Cases that time the norms around a decoder's layers and the attention of a batch with a
shared prompt.

Three operators, each called the way a program calls it:

  gated_norm         the RMS norm of a recurrent layer's output heads with its output gate:
                     norm(x) w act(z), or norm(x act(z)) w: forward, training step
  residual_norm      r' = r + s act(z) p(y), p the block's output or its RMS norm, then the
                     next block's RMS norm of r': forward, training step
  paged_prefix_attn  one new token per sequence against a prompt that the batch shares and
                     against its own paged cache

``own`` picks the side: the framework's entry points, or the same formulas in plain torch
operations in 32 bits. ``exact`` restates every formula in 64 bits, written separately.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SPARE_PAGES = 3      # pages of a cache that no sequence owns
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # A decode step of 64 sequences: the 16 x 128 output channels of a delta-rule layer
        # before its output projection. A few microseconds: launch and host cost decide it.
        dict(name="gated_step_b64_h16", op="gated_fwd", B=64, T=1, H=16, D=128, dtype="bf16",
             act="silu", first=False, per_head=False, fused=True),
        # Prefill, 2 x 8192 tokens of 32 value heads, the gate a slice of a projection.
        dict(name="gated_prefill_b2_t8192_h32", op="gated_fwd", B=2, T=8192, H=32, D=128,
             dtype="bf16", act="sigmoid", first=False, per_head=False, fused=True),
        # A training step at the headline shape: 4096 tokens, 12 heads of 128.
        dict(name="gated_train_t4096_h12", op="gated_train", B=1, T=4096, H=12, D=128,
             dtype="bf16", act="silu", first=False, per_head=False, fused=False),
        # The same step of a layer that gates first and norms groups of 512 channels, each
        # with its own weights.
        dict(name="gated_train_groups_d512", op="gated_train", B=2, T=4096, H=4, D=512,
             dtype="bf16", act="silu", first=True, per_head=True, fused=True),
        # Between two layers of a decode step: 64 tokens, 2048 channels, a 32-bit residual.
        dict(name="residual_step_b64_d2048", op="res_fwd", B=64, T=1, D=2048, dtype="bf16",
             rdtype="f32", gate="", post=False, scale="one"),
        # A training step between two layers, 2 x 8192 tokens, 4096 channels: add and norm.
        dict(name="residual_train_b2_t8192_d4096", op="res_train", B=2, T=8192, D=4096,
             dtype="bf16", rdtype="bf16", gate="", post=False, scale="one"),
        # Everything a block can ask for: its output normed, gated and scaled per channel.
        dict(name="residual_train_gated_t4096_d1536", op="res_train", B=1, T=4096, D=1536,
             dtype="bf16", rdtype="f32", gate="sigmoid", post=True, scale="vector"),
        # A small 32-bit training step with sizes off every tile (3 x 1021 x 777).
        dict(name="residual_train_f32_odd", op="res_train", B=3, T=1021, D=777, dtype="f32",
             rdtype="f32", gate="", post=True, scale="one"),
        # 64 chats behind one system prompt of 8192 tokens, up to 512 tokens of their own.
        dict(name="prefix_b64_p8192", op="prefix", B=64, P=8192, L=512, HQ=32, HK=4, D=128,
             page=64, dtype="bf16"),
        # 128 questions about one long document: 65000 shared keys, 16 key heads.
        dict(name="prefix_b128_p65000", op="prefix", B=128, P=65000, L=1024, HQ=32, HK=16, D=128,
             page=64, dtype="bf16"),
        # A few chats behind a short prompt, small pages: latency.
        dict(name="prefix_b4_short", op="prefix", B=4, P=200, L=60, HQ=16, HK=16, D=128, page=16,
             dtype="bf16"),
        # 32-bit caches, odd pages, grouped heads.
        dict(name="prefix_f32_odd", op="prefix", B=5, P=2999, L=300, HQ=6, HK=3, D=64, page=48,
             dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["gated_fwd", "gated_train", "res_fwd", "res_train", "prefix", "prefix"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("gated"):
        D = rng.choice([64, 128, 128, 256, 80, 96, _log(rng, 16, 4096)])
        H = rng.choice([1, 2, 3, 4, 8, 12, 16, 32])
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, min(16384, (1 << 26) // (B * H * D))))
        return dict(op=op, B=B, T=T, H=H, D=D, dtype=dtype,
                    act=rng.choice(["silu", "silu", "sigmoid"]), first=rng.random() < 0.4,
                    per_head=rng.random() < 0.4, fused=rng.random() < 0.5)
    if op.startswith("res"):
        D = _log(rng, 16, 8192)
        D = rng.choice([D, max(64, D // 64 * 64), max(64, D // 64 * 64)])
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, min(16384, (1 << 25) // (B * D))))
        return dict(op=op, B=B, T=T, D=D, dtype=dtype,
                    rdtype="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                    gate=rng.choice(["", "", "sigmoid", "silu"]), post=rng.random() < 0.4,
                    scale=rng.choice(["one", "number", "vector"]))
    D = rng.choice([64, 128, 128, 256, 80, 96])
    HK = rng.choice([1, 2, 3, 4, 8, 16])
    G = rng.choice([1, 2, 4, 5, 8, 16])
    B = _log(rng, 1, 256)
    # Keys x rows x channels of the largest listed case at most; a 16th of it in 32 bits.
    most = (1 << 35) // (1 if dtype == "bf16" else 16)
    P = _log(rng, 1, max(64, min(65000, most // (B * HK * G * D), (1 << 27) // (HK * D))))
    L = _log(rng, 1, max(64, min(4096, (1 << 26) // (B * HK * D))))
    return dict(op="prefix", B=B, P=P, L=L, HQ=HK * G, HK=HK, D=D,
                page=rng.choice([16, 32, 64, 128, 17]), dtype=dtype)


# ------------------------------------------------------------------ inputs
def _lens(case, seed):
    """Keys of each sequence behind the shared ones, on the host: spread over 0..L, one of
    each end when there is room."""
    gen = torch.Generator().manual_seed(seed + 17)
    B, L = case["B"], case["L"]
    lens = torch.randint(0, L + 1, (B,), generator=gen)
    lens[0] = L
    if B > 2:
        lens[1] = 0
    return lens


def _pages(lens, shared, page, most, gen):
    """(shared pages [n], page table [B, pages of `most` tokens] with -1 where no page is
    owned, pages in the cache), pages handed out in any order."""
    need = [(int(n) + page - 1) // page for n in lens]
    first, most = (shared + page - 1) // page, max(1, (most + page - 1) // page)
    total = first + len(need) * most + SPARE_PAGES
    order = torch.randperm(total, generator=gen).to(torch.int32)
    owned = torch.arange(most)[None, :] < torch.tensor(need)[:, None]
    table = torch.full((len(need), most), -1, dtype=torch.int32)
    table[owned] = order[first: first + sum(need)]
    return order[:first].clone(), table, total


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed + 5)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def weight(*shape):
        return randn(*shape).mul_(0.2).add_(1.0)

    s = dict(case)
    D, B = case["D"], case["B"]
    if case["op"] == "prefix":
        lens = _lens(case, seed)
        prefix, table, total = _pages(lens, case["P"], case["page"], case["L"], cpu)
        s["prefix"], s["table"] = prefix.to(dev), table.to(dev)
        s["lens"] = lens.to(torch.int32).to(dev)
        s["k_cache"] = randn(total, case["page"], case["HK"], D, dtype=dt)
        s["v_cache"] = randn(total, case["page"], case["HK"], D, dtype=dt)
        s["q"] = randn(B, case["HQ"], D, dtype=dt)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, case["HQ"], device=dev)
        return s
    T = case["T"]
    if case["op"].startswith("gated"):
        H = case["H"]
        s["x"] = randn(B, T, H, D, dtype=dt)
        if case["fused"]:                      # the gate is a slice of a wider projection
            s["z"] = randn(B, T, 2 * H * D, dtype=dt)[..., H * D:].unflatten(-1, (H, D))
        else:
            s["z"] = randn(B, T, H, D, dtype=dt)
        s["w"] = weight(H, D) if case["per_head"] else weight(D)
        if case["op"] == "gated_train":
            s["dout"] = randn(B, T, H, D, dtype=dt)
        elif T == 1:                           # a decoder's fixed buffers
            s["out"] = torch.empty(B, T, H, D, dtype=dt, device=dev)
        return s
    rt = DTYPES[case["rdtype"]]
    s["r"] = randn(B, T, D).mul_(3.0).to(rt)   # the sum of some layers' outputs
    s["y"] = randn(B, T, D, dtype=dt)
    s["z"] = randn(B, T, D, dtype=dt) if case["gate"] else None
    s["w"] = weight(D)
    s["wp"] = weight(D) if case["post"] else None
    s["s"] = {"one": 1.0, "number": 0.25, "vector": None}[case["scale"]]
    if s["s"] is None:
        s["s"] = randn(D).mul_(0.1).add_(0.5)
    if case["op"] == "res_train":
        s["dout"] = randn(B, T, D, dtype=dt)
        s["dres"] = randn(B, T, D, dtype=rt)
    elif T == 1:
        s["out"] = torch.empty(B, T, D, dtype=dt, device=dev)
        s["r_out"] = torch.empty(B, T, D, dtype=rt, device=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _OWN[s["op"]](s) if own else _PLAIN[s["op"]](s)


def _own_gated_fwd(s):
    import chunkwise_gated_delta_gdr_gb300 as gdr
    return gdr.gated_norm(s["x"], s["z"], s["w"], activation=s["act"], gate_first=s["first"],
                          eps=EPS, out=s.get("out"))


def _own_gated_train(s):
    import chunkwise_gated_delta_gdr_gb300 as gdr
    kw = dict(activation=s["act"], gate_first=s["first"], eps=EPS)
    out = gdr.gated_norm(s["x"], s["z"], s["w"], **kw)
    return (out, *gdr.gated_norm_bwd(s["dout"], s["x"], s["z"], s["w"], **kw))


def _res_kw(s):
    return dict(gate=s["z"], activation=s["gate"] or "sigmoid", post_norm=s["post"],
                post_weight=s["wp"], scale=s["s"], eps=EPS)


def _own_res_fwd(s):
    import chunkwise_gated_delta_gdr_gb300 as gdr
    return gdr.residual_norm(s["r"], s["y"], s["w"], **_res_kw(s), out=s.get("out"),
                             residual_out=s.get("r_out"))


def _own_res_train(s):
    import chunkwise_gated_delta_gdr_gb300 as gdr
    kw = _res_kw(s)
    out, r = gdr.residual_norm(s["r"], s["y"], s["w"], **kw)
    grads = gdr.residual_norm_bwd(s["dout"], s["dres"], r, s["y"], s["w"], **kw)
    return (out, r, *[g for g in grads if g is not None])


def _own_prefix(s):
    import chunkwise_gated_delta_gdr_gb300 as gdr
    if "ws" not in s:          # the scratch a decoder allocates once for its batch
        s["ws"] = torch.empty(gdr.paged_prefix_attn_workspace_size(
            s["q"], s["k_cache"], s["prefix"], s["P"], s["table"]), dtype=torch.uint8,
            device=s["q"].device)
    return gdr.paged_prefix_attn(s["q"], s["k_cache"], s["v_cache"], s["prefix"], s["P"],
                                 s["table"], s["lens"], out=s["out"], lse=s["lse"],
                                 workspace=s["ws"])


# The plain forms.
def _unit(x):
    """x over its root mean square, and one over that."""
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _unit_back(d, u, r):
    return r * (d - u * (d * u).mean(-1, keepdim=True))


def _act(z, kind):
    """act(z) and its derivative."""
    g = 1.0 / (1.0 + torch.exp(-z))
    if kind == "sigmoid":
        return g, g * (1 - g)
    return z * g, g * (1 + z * (1 - g))


def _plain_gated_fwd(s):
    a, _ = _act(s["z"].float(), s["act"])
    x = s["x"].float()
    if s["first"]:
        y = _unit(x * a)[0] * s["w"]
    else:
        y = _unit(x)[0] * s["w"] * a
    return y.to(s["x"].dtype)


def _plain_gated_train(s):
    dt, w = s["x"].dtype, s["w"]
    x, d = s["x"].float(), s["dout"].float()
    a, da = _act(s["z"].float(), s["act"])
    over = (0, 1) if w.dim() == 2 else (0, 1, 2)
    if s["first"]:
        u, r = _unit(x * a)
        out, dw = u * w, (d * u).sum(over)
        dv = _unit_back(d * w, u, r)
        dx, dz = dv * a, dv * x * da
    else:
        u, r = _unit(x)
        out, dw = u * w * a, (d * a * u).sum(over)
        dx, dz = _unit_back(d * a * w, u, r), d * u * w * da
    return out.to(dt), dx.to(dt), dz.to(dt), dw


def _branch(s):
    """The block's output as it goes into the residual, but for the scale: (unit of y and one
    over its root mean square, or nothing), p, act(z), its derivative."""
    y = s["y"].float()
    u = r = None
    p = y
    if s["post"]:
        u, r = _unit(y)
        p = u * s["wp"]
    a, da = (None, None) if s["z"] is None else _act(s["z"].float(), s["gate"])
    return u, r, p, a, da


def _plain_res_fwd(s):
    _, _, p, a, _ = _branch(s)
    r = s["r"].float() + s["s"] * (p if a is None else p * a)
    return (_unit(r)[0] * s["w"]).to(s["y"].dtype), r.to(s["r"].dtype)


def _plain_res_train(s):
    dt, rt = s["y"].dtype, s["r"].dtype
    out, res = _plain_res_fwd(s)
    uy, ry, p, a, da = _branch(s)
    u, r = _unit(res.float())
    d = s["dout"].float()
    grads = [(d * u).sum((0, 1))]
    g = s["dres"].float() + _unit_back(d * s["w"], u, r)
    dt_ = g * s["s"]
    dp = dt_ if a is None else dt_ * a
    dz = None if a is None else (dt_ * p * da).to(dt)
    dy = dp
    if s["post"]:
        grads.append((dp * uy).sum((0, 1)))
        dy = _unit_back(dp * s["wp"], uy, ry)
    if isinstance(s["s"], torch.Tensor):
        grads.append((g * (p if a is None else p * a)).sum((0, 1)))
    first = [g.to(rt), dy.to(dt)] + ([] if dz is None else [dz])
    return (out, res, *first, *grads)


def _plain_prefix(s):
    B, HQ, D = s["q"].shape
    page, HK, P = s["page"], s["HK"], s["P"]
    table = s["table"].long().clamp_min(0)
    live = torch.arange(table.shape[1] * page, device=table.device) < s["lens"].long()[:, None]
    shared = s["prefix"].long()
    kp = s["k_cache"][shared].flatten(0, 1)[:P].float()
    vp = s["v_cache"][shared].flatten(0, 1)[:P].float()
    k = s["k_cache"][table].flatten(1, 2).float()
    v = s["v_cache"][table].flatten(1, 2).float()
    v = torch.where(live[:, :, None, None], v, torch.zeros((), device=v.device))
    q = s["q"].float().view(B, HK, HQ // HK, D) * (1.0 / math.sqrt(D))
    own_score = torch.einsum("bhgd,bnhd->bhgn", q, k)
    own_score = torch.where(live[:, None, None], own_score, own_score.new_tensor(-math.inf))
    score = torch.cat([torch.einsum("bhgd,nhd->bhgn", q, kp), own_score], -1)
    top = score.max(-1, keepdim=True).values
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgn,nhd->bhgd", p[..., :P], vp)
    o = o + torch.einsum("bhgn,bnhd->bhgd", p[..., P:], v)
    return (o / total).reshape(B, HQ, D).to(s["q"].dtype), (top + torch.log(total)).view(B, HQ)


_OWN = dict(gated_fwd=_own_gated_fwd, gated_train=_own_gated_train, res_fwd=_own_res_fwd,
            res_train=_own_res_train, prefix=_own_prefix)
_PLAIN = dict(gated_fwd=_plain_gated_fwd, gated_train=_plain_gated_train, res_fwd=_plain_res_fwd,
              res_train=_plain_res_train, prefix=_plain_prefix)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, D = case["B"], case["D"]
    if case["op"] == "prefix":
        # Lengths differ by seed: their mean over 0..L, one of them L and one 0.
        P, L, HQ, HK = case["P"], case["L"], case["HQ"], case["HK"]
        keys = L + (B - (2 if B > 2 else 1)) * L / 2
        return {"bytes": 2 * (P + keys) * HK * D * e + 2 * B * HQ * D * e + 4 * B * HQ,
                "flops": 4 * (B * P + keys) * HQ * D}
    if case["op"].startswith("gated"):
        n = B * case["T"] * case["H"] * D
        w = 4 * D * (case["H"] if case["per_head"] else 1)
        # forward: x, z in, out out; backward: d, x, z in, dx, dz out
        if case["op"] == "gated_fwd":
            return {"bytes": 3 * n * e + w, "flops": 9 * n}
        return {"bytes": 8 * n * e + 3 * w, "flops": 32 * n}
    re = 2 if case["rdtype"] == "bf16" else 4
    n, z = B * case["T"] * D, 1 if case["gate"] else 0
    vectors = 4 * D * (1 + case["post"] + (case["scale"] == "vector"))
    fwd = n * (2 * re + (2 + z) * e)             # r, y, z in, r', out out
    if case["op"] == "res_fwd":
        return {"bytes": fwd + vectors, "flops": 12 * n}
    # backward: d_out, d_r', r', y (if normed, gated or scaled by a vector), z in, dr, dy, dz out
    reads_y = case["post"] or z or case["scale"] == "vector"
    bwd = n * (3 * re + (2 + bool(reads_y) + 2 * z) * e)
    return {"bytes": fwd + bwd + 3 * vectors, "flops": 40 * n}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefix":
        return _exact_prefix(s)
    return _exact_gated(s) if case["op"].startswith("gated") else _exact_residual(s)


def _exact_norm(x, w):
    return x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w


def _exact_act(z, kind):
    return torch.sigmoid(z) if kind == "sigmoid" else z * torch.sigmoid(z)


def _exact_gated(s):
    """Gradients by differentiating the definition."""
    x, z, w = (s[n].double().requires_grad_(True) for n in ("x", "z", "w"))
    a = _exact_act(z, s["act"])
    y = _exact_norm(x * a, w) if s["first"] else _exact_norm(x, w) * a
    if s["op"] == "gated_fwd":
        return y.detach()
    return (y.detach(), *torch.autograd.grad(y, (x, z, w), s["dout"].double()))


def _exact_residual(s):
    """The branch and the norm behind it, each differentiated by itself: the backward pass has
    the residual as it is stored."""
    leaf = lambda t: t.double().requires_grad_(True)  # noqa: E731
    y, w = leaf(s["y"]), leaf(s["w"])
    z = None if s["z"] is None else leaf(s["z"])
    wp = leaf(s["wp"]) if s["post"] else None
    scale = leaf(s["s"]) if isinstance(s["s"], torch.Tensor) else s["s"]
    t = _exact_norm(y, wp) if s["post"] else y
    if z is not None:
        t = t * _exact_act(z, s["gate"])
    t = t * scale
    res = s["r"].double() + t.detach()
    out = _exact_norm(res, w.detach())
    if s["op"] == "res_fwd":
        return out, res
    stored = leaf(res.to(s["r"].dtype))
    g, dw = torch.autograd.grad(_exact_norm(stored, w), (stored, w), s["dout"].double())
    g = g + s["dres"].double()
    want = [n for n in (y, z, wp, scale) if isinstance(n, torch.Tensor)]
    got = dict(zip(map(id, want), torch.autograd.grad(t, want, g)))
    grads = [g, got[id(y)]] + ([got[id(z)]] if z is not None else []) + [dw]
    grads += [got[id(n)] for n in (wp, scale) if isinstance(n, torch.Tensor)]
    return (out, res, *grads)


def _exact_prefix(s):
    """Sequence by sequence: shared and own keys gathered, one softmax over all of them."""
    B, HQ, D = s["q"].shape
    HK, P, page = s["HK"], s["P"], s["page"]
    G = HQ // HK
    dev = s["q"].device
    at = torch.arange(P, device=dev)
    rows = s["prefix"].long()[at // page] * page + at % page
    flat_k, flat_v = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    kp, vp = flat_k[rows].double().permute(1, 2, 0), flat_v[rows].double().permute(1, 0, 2)
    o = torch.empty(B, HQ, D, dtype=torch.float64, device=dev)
    lse = torch.empty(B, HQ, dtype=torch.float64, device=dev)
    for b, n in enumerate(s["lens"].tolist()):
        at = torch.arange(n, device=dev)
        rows = s["table"][b].long()[at // page] * page + at % page
        q = s["q"][b].double().view(HK, G, D)
        k, v = flat_k[rows].double().permute(1, 2, 0), flat_v[rows].double().permute(1, 0, 2)
        z = torch.cat([q @ kp, q @ k], -1) / math.sqrt(D)
        w = torch.softmax(z, -1)
        o[b] = (w[..., :P] @ vp + w[..., P:] @ v).reshape(HQ, D)
        lse[b] = torch.logsumexp(z, -1).reshape(HQ)
    return o, lse
