"""A small hybrid decoder on the library's layers: gated delta rule, gated linear recurrence,
attention over a paged cache.

    python examples/hybrid_decoder.py            # generates a few tokens, then trains a little

Random weights, three layers, every sequence operation a kernel of the library; the dense
projections are torch matrix products. Shows how the entry points fit together:

  prefill   chunk_fwd, linear_scan_fwd, qk_norm_rope_append, paged_decode_attn (one row per
            prompt token, its own length), states and pages left for decoding
  decode    recurrent_fwd, linear_scan_fwd on one token with the state in place,
            qk_norm_rope_append, paged_decode_attn
  training  linear_scan_fwd / _bwd and qk_norm_rope / _bwd as autograd functions

NormedDecoder is the same stack with an output gate behind the delta rule (gated_norm) and its
adds and norms in one call between two layers (residual_norm); generate_shared() decodes a batch
behind one prompt, whose states are computed and whose keys are stored and read once
(paged_prefix_attn). GatedNorm and ResidualNorm are their autograd functions.
"""
from __future__ import annotations

import math
import os
import sys

import torch
import torch.nn.functional as nnf

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunkwise_gated_delta_gdr_gb300 as gdr  # noqa: E402

WIDTH, VOCAB, PAGE = 256, 512, 16
DELTA_HEADS, DELTA_DIM = 2, 128                  # q, k, v heads of the delta rule
HQ, HK, DIM = 4, 2, 64                           # attention heads


def rope_table(rows, dim, device):
    freq = 10000.0 ** (-torch.arange(0, dim, 2, device=device, dtype=torch.float64) / dim)
    angle = torch.arange(rows, device=device, dtype=torch.float64)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def unit(x):
    return x * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6).to(x.dtype)


class Cache:
    """What decoding carries: a state per recurrent layer, pages for the attention layer."""

    def __init__(self, batch, longest, device):
        self.delta = torch.zeros(batch, DELTA_HEADS, DELTA_DIM, DELTA_DIM, device=device)
        self.scan = torch.zeros(batch, WIDTH, device=device)
        pages = -(-longest // PAGE)
        self.table = torch.randperm(batch * pages, device=device).view(batch, pages).int()
        shape = (batch * pages, PAGE, HK, DIM)
        self.k = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        self.v = torch.zeros_like(self.k)
        self.length = 0


class HybridDecoder:
    def __init__(self, device, seed=0, longest=512):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(n, m):
            w = torch.randn(n, m, generator=gen, device=device) / math.sqrt(n)
            return w.to(torch.bfloat16)

        qkv = DELTA_HEADS * DELTA_DIM
        self.embed = weight(VOCAB, WIDTH) * math.sqrt(VOCAB)
        self.delta_in, self.delta_gate = weight(WIDTH, 3 * qkv), weight(WIDTH, 2 * DELTA_HEADS)
        self.delta_out = weight(qkv, WIDTH)
        self.scan_in, self.scan_out = weight(WIDTH, 2 * WIDTH), weight(WIDTH, WIDTH)
        self.attn_in = weight(WIDTH, (HQ + 2 * HK) * DIM)
        self.attn_out = weight(HQ * DIM, WIDTH)
        self.q_weight = torch.ones(DIM, device=device)
        self.k_weight = torch.ones(DIM, device=device)
        self.cos, self.sin = rope_table(longest, DIM, device)
        self.head = weight(WIDTH, VOCAB)
        self.device = device

    def delta(self, x, cache):
        B, T, _ = x.shape
        q, k, v = (x @ self.delta_in).view(B, T, 3, DELTA_HEADS, DELTA_DIM).unbind(2)
        gates = (x @ self.delta_gate).float().view(B, T, 2, DELTA_HEADS)
        g = nnf.logsigmoid(gates[:, :, 0] + 2.0).contiguous()
        beta = torch.sigmoid(gates[:, :, 1]).contiguous()
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        if T == 1:
            o = gdr.recurrent_fwd(q, k, v, g, beta, cache.delta)
        else:
            o, _ = gdr.chunk_fwd(q, k, v, g, beta, cache.delta, final_state=cache.delta)
        return o.view(B, T, -1) @ self.delta_out

    def scan(self, x, cache):
        value, gate = (x @ self.scan_in).chunk(2, -1)          # views of one projection
        h, _ = gdr.linear_scan_fwd(value, nnf.logsigmoid(gate.float() + 3.0), cache.scan,
                                   gated_input=True, final_state=cache.scan)
        return h @ self.scan_out

    def attention(self, x, cache):
        B, T, _ = x.shape
        qkv = (x @ self.attn_in).view(B, T, HQ + 2 * HK, DIM)
        pos = (cache.length + torch.arange(T, device=x.device, dtype=torch.int32)).repeat(B, 1)
        q = gdr.qk_norm_rope_append(qkv[:, :, :HQ], qkv[:, :, HQ:HQ + HK], qkv[:, :, HQ + HK:],
                                    self.q_weight, self.k_weight, self.cos, self.sin, pos,
                                    cache.k, cache.v, cache.table)
        # Each token attends to the cache up to itself: its own row, table and length.
        table = cache.table.repeat_interleave(T, 0) if T > 1 else cache.table
        o, _ = gdr.paged_decode_attn(q.view(B * T, HQ, DIM), cache.k, cache.v, table,
                                     (pos + 1).view(-1))
        return o.view(B, T, -1) @ self.attn_out

    def forward(self, tokens, cache):
        """tokens [B, T]: logits [B, T, VOCAB]; `cache` moves on by T tokens."""
        x = self.embed[tokens]
        for layer in (self.delta, self.scan, self.attention):
            x = x + layer(unit(x), cache)
        cache.length += tokens.shape[1]
        return unit(x) @ self.head

    def generate(self, prompt, steps):
        """Greedy: (tokens [B, steps], logits of every step [B, steps, VOCAB])."""
        cache = Cache(prompt.shape[0], prompt.shape[1] + steps, self.device)
        logits = self.forward(prompt, cache)[:, -1:]
        tokens, seen = [], []
        for i in range(steps):
            seen.append(logits)
            tokens.append(logits.argmax(-1))
            if i + 1 < steps:
                logits = self.forward(tokens[-1], cache)
        return torch.cat(tokens, 1), torch.cat(seen, 1)


# ------------------------------------------------------------------ gate, norms, shared prompt
class SharedCache:
    """What decoding behind a shared prompt carries: the prompt's whole pages once (`shared` tokens),
    and for every sequence its states and pages for `longest` tokens of its own in the same arrays."""

    def __init__(self, shared, batch, longest, device):
        self.shared = shared
        first, own = shared // PAGE, -(-longest // PAGE)
        order = torch.randperm(first + batch * own, device=device).int()
        self.prefix, self.table = order[:first].clone(), order[first:].view(batch, own)
        # New keys are stored by their position in the sequence: prompt's pages, then its own.
        self.whole = torch.cat([self.prefix.repeat(batch, 1), self.table], 1).contiguous()
        shape = (first + batch * own, PAGE, HK, DIM)
        self.k = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        self.v = torch.zeros_like(self.k)
        self.delta = torch.zeros(batch, DELTA_HEADS, DELTA_DIM, DELTA_DIM, device=device)
        self.scan = torch.zeros(batch, WIDTH, device=device)
        self.length = self.shared

    def prompt(self):
        """A cache of one sequence that fills the prompt's pages."""
        one = Cache.__new__(Cache)
        one.delta, one.scan = torch.zeros_like(self.delta[:1]), torch.zeros_like(self.scan[:1])
        one.table, one.k, one.v, one.length = self.prefix[None], self.k, self.v, 0
        return one


class NormedDecoder(HybridDecoder):
    def __init__(self, device, seed=0, longest=512):
        super().__init__(device, seed, longest)
        gen = torch.Generator(device=device).manual_seed(seed + 1)
        heads = DELTA_HEADS * DELTA_DIM
        self.gate_in = (torch.randn(WIDTH, heads, generator=gen, device=device)
                        / math.sqrt(WIDTH)).to(torch.bfloat16)
        self.gate_weight = torch.ones(DELTA_DIM, device=device)
        self.norms = [torch.ones(WIDTH, device=device) for _ in range(4)]

    def delta(self, x, cache):
        B, T, _ = x.shape
        q, k, v = (x @ self.delta_in).view(B, T, 3, DELTA_HEADS, DELTA_DIM).unbind(2)
        gates = (x @ self.delta_gate).float().view(B, T, 2, DELTA_HEADS)
        g = nnf.logsigmoid(gates[:, :, 0] + 2.0).contiguous()
        beta = torch.sigmoid(gates[:, :, 1]).contiguous()
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        if T == 1:
            o = gdr.recurrent_fwd(q, k, v, g, beta, cache.delta)
        else:
            o, _ = gdr.chunk_fwd(q, k, v, g, beta, cache.delta, final_state=cache.delta)
        z = (x @ self.gate_in).view(B, T, DELTA_HEADS, DELTA_DIM)
        o = gdr.gated_norm(o.view(z.shape), z, self.gate_weight)
        return o.view(B, T, -1) @ self.delta_out

    def attention(self, x, cache):
        if not isinstance(cache, SharedCache):
            return super().attention(x, cache)
        B, T, _ = x.shape
        qkv = (x @ self.attn_in).view(B, T, HQ + 2 * HK, DIM)
        pos = (cache.length + torch.arange(T, device=x.device, dtype=torch.int32)).repeat(B, 1)
        q = gdr.qk_norm_rope_append(qkv[:, :, :HQ], qkv[:, :, HQ:HQ + HK], qkv[:, :, HQ + HK:],
                                    self.q_weight, self.k_weight, self.cos, self.sin, pos,
                                    cache.k, cache.v, cache.whole)
        table = cache.table.repeat_interleave(T, 0) if T > 1 else cache.table
        o, _ = gdr.paged_prefix_attn(q.view(B * T, HQ, DIM), cache.k, cache.v, cache.prefix,
                                     cache.shared, table, (pos + 1 - cache.shared).view(-1))
        return o.view(B, T, -1) @ self.attn_out

    def forward(self, tokens, cache):
        residual = self.embed[tokens].float()        # kept in 32 bits
        x, _ = gdr.residual_norm(residual, None, self.norms[0], out_dtype=torch.bfloat16)
        for layer, weight in zip((self.delta, self.scan, self.attention), self.norms[1:]):
            x, residual = gdr.residual_norm(residual, layer(x, cache), weight,
                                            residual_out=residual)
        cache.length += tokens.shape[1]
        return x @ self.head

    def generate_shared(self, prompt, tails, steps):
        """Greedy, for a batch behind one prompt: prompt [P], tails [B, n] the rest of each
        sequence; (tokens [B, steps], logits of every step [B, steps, VOCAB])."""
        B, n = tails.shape
        if len(prompt) + n == 0:
            raise ValueError("prompt and tails are empty: there is nothing to continue")
        # Whole pages. Without tails the prompt's last token is each sequence's own: the first new
        # token needs its logits.
        shared = (len(prompt) - (n == 0)) // PAGE * PAGE
        cache = SharedCache(shared, B, len(prompt) - shared + n + steps, self.device)
        if cache.shared:
            once = cache.prompt()
            self.forward(prompt[None, :cache.shared], once)
            cache.delta.copy_(once.delta.expand_as(cache.delta))
            cache.scan.copy_(once.scan.expand_as(cache.scan))
        rest = torch.cat([prompt[cache.shared:].expand(B, -1), tails], 1)
        logits = self.forward(rest, cache)[:, -1:]
        tokens, seen = [], []
        for i in range(steps):
            seen.append(logits)
            tokens.append(logits.argmax(-1))
            if i + 1 < steps:
                logits = self.forward(tokens[-1], cache)
        return torch.cat(tokens, 1), torch.cat(seen, 1)


# ------------------------------------------------------------------ training
class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, weight):
        ctx.save_for_backward(x, gate, weight)
        return gdr.gated_norm(x, gate, weight)

    @staticmethod
    def backward(ctx, d):
        return gdr.gated_norm_bwd(d.contiguous(), *ctx.saved_tensors)


class ResidualNorm(torch.autograd.Function):
    """(out, residual + scale y) with a scale per channel."""

    @staticmethod
    def forward(ctx, residual, y, weight, scale):
        out, residual = gdr.residual_norm(residual, y, weight, scale=scale)
        ctx.save_for_backward(residual, y, weight, scale)
        return out, residual

    @staticmethod
    def backward(ctx, d, d_residual):
        residual, y, weight, scale = ctx.saved_tensors
        dr, dy, _, dw, _, ds = gdr.residual_norm_bwd(d.contiguous(), d_residual.contiguous(),
                                                     residual, y, weight, scale=scale)
        return dr, dy, dw, ds


class LinearScan(torch.autograd.Function):
    """h = linear_scan(x, g) with the input gated, from a zero state."""

    @staticmethod
    def forward(ctx, x, g):
        ck = gdr.linear_scan_checkpoints(x)
        h, _ = gdr.linear_scan_fwd(x, g, gated_input=True, output_final_state=False,
                                   checkpoints=ck)
        ctx.save_for_backward(x, g, ck)
        return h

    @staticmethod
    def backward(ctx, dh):
        x, g, ck = ctx.saved_tensors
        dx, dg, _ = gdr.linear_scan_bwd(dh, x, g, ck, gated_input=True,
                                        output_initial_state_grad=False)
        return dx, dg


class QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions):
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        return gdr.qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions)

    @staticmethod
    def backward(ctx, dq, dk):
        return (*gdr.qk_norm_rope_bwd(dq.contiguous(), dk.contiguous(), *ctx.saved_tensors),
                None, None, None)


def train(device, steps=30, seed=0):
    """Fits a recurrent layer followed by normed, rotated queries and keys to a target;
    returns the losses."""
    torch.manual_seed(seed)
    B, T = 2, 200
    x = torch.randn(B, T, WIDTH, device=device)
    target = torch.randn(B, T, HQ, DIM, device=device) * 0.5
    cos, sin = rope_table(T, DIM, device)
    pos = torch.arange(T, device=device, dtype=torch.int32).repeat(B, 1)
    w_in = torch.randn(WIDTH, 2 * WIDTH, device=device) / math.sqrt(WIDTH)
    w_qk = torch.randn(WIDTH, (HQ + HK) * DIM, device=device) / math.sqrt(WIDTH)
    params = [w_in, w_qk, torch.ones(DIM, device=device), torch.ones(DIM, device=device)]
    for p in params:
        p.requires_grad_(True)
    opt = torch.optim.Adam(params, lr=3e-3)
    losses = []
    for _ in range(steps):
        value, gate = (x @ params[0]).chunk(2, -1)
        h = LinearScan.apply(value, nnf.logsigmoid(gate + 3.0))
        qk = (h @ params[1]).view(B, T, HQ + HK, DIM)
        q, k = QkNormRope.apply(qk[:, :, :HQ], qk[:, :, HQ:], params[2], params[3], cos, sin, pos)
        loss = nnf.mse_loss(q, target) + nnf.mse_loss(k, target[:, :, :HK])
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


if __name__ == "__main__":
    dev = torch.device("cuda:0")
    model = HybridDecoder(dev)
    prompt = torch.randint(0, VOCAB, (3, 100), generator=torch.Generator().manual_seed(1)).to(dev)
    out, _ = model.generate(prompt, 16)
    print("generated:", out.tolist())
    out, _ = NormedDecoder(dev).generate_shared(prompt[0], prompt[:, :7], 16)
    print("behind one prompt:", out.tolist())
    losses = train(dev)
    print(f"training loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
