"""A small language model of selective-scan blocks, trained and then asked for tokens.

    python examples/train_lm.py [--steps 60] [--dim 256] [--layers 2] [--dtype bf16]
                                [--mixer scan|lru] [--mlp 512] [--loss library|own]

Every operator of the library that such a model needs is used where it would be used:

    embedding (msel_embed_fwd)             ids -> residual stream, fp32
    per block
        norm (msel_norm_fwd)               adds the last block's output to the residual stream
        input projection                   one GEMM per batch row, to [batch, channels, seqlen]
        conv + SiLU (msel_conv1d_fwd)
        projections to delta, B, C
        scan (msel_scan_fwd)               without its own gate
        gated norm (msel_gated_norm_fwd)   turned to [batch, seqlen, channels]
        output projection
    last norm, head tied to the embedding's table, cross entropy
    backward; the embedding's gradient is added into the head's (msel_embed_bwd with base)
    clipping over all gradients (msel_grad_clip), AdamW

With --mixer lru the scan gives way to the gated linear recurrence (msel_lru_fwd), whose gates are
projections of the convolution's output; with --mlp a gated feed-forward block of that hidden width
(msel_gated_mlp_fwd) follows every mixer; with --loss own the loss is the mean log probability of
msel_logprob_fwd, and the continued tokens come with their log probability and entropy.

The projections are plain library products; autograd carries the gradients between the
operators.  Generation keeps a convolution and a scan state per block and takes one token per
call.  The data are synthetic: sequences that repeat a random pattern, so that a model that
carries state predicts all but the first period.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_26_amd as msel  # noqa: E402


class Norm(torch.autograd.Function):
    """(out, s) of msel_norm_fwd: s = residual + x, out = norm(s) * weight."""

    @staticmethod
    def forward(ctx, x, weight, residual):
        out, s = msel.msel_norm_fwd(x, weight, residual)
        ctx.save_for_backward(s, weight)
        return out, s

    @staticmethod
    def backward(ctx, dout, ds):
        s, weight = ctx.saved_tensors
        g = msel.msel_norm_bwd(s, weight, dout.contiguous(),
                               None if ds is None else ds.contiguous())
        return g["dx"], g["dweight"], g["dresidual"]


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return msel.msel_conv1d_fwd(x, weight, bias)[0]

    @staticmethod
    def backward(ctx, dout):
        x, weight, bias = ctx.saved_tensors
        g = msel.msel_conv1d_bwd(x, weight, dout.contiguous(), bias)
        return g["dx"], g["dweight"], g["dbias"]


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, bias):
        out, _, cs = msel.msel_scan_fwd(u, delta, A, B, C, D, None, bias, True,
                                        return_final_state=False, return_chunk_states=True)
        ctx.save_for_backward(u, delta, A, B, C, D, bias, cs)
        return out

    @staticmethod
    def backward(ctx, dout):
        u, delta, A, B, C, D, bias, cs = ctx.saved_tensors
        g = msel.msel_scan_bwd(u, delta, A, B, C, dout.contiguous(), D, None, bias, True,
                               chunk_states=cs)
        return (g["du"], g["ddelta"], g["dA"], g["dB"].to(B.dtype), g["dC"].to(C.dtype), g["dD"],
                g["ddelta_bias"])


class GatedNorm(torch.autograd.Function):
    """norm(x * silu(z)) * weight over the channels of [batch, dim, seqlen], to
    [batch, seqlen, dim]."""

    @staticmethod
    def forward(ctx, x, z, weight):
        ctx.save_for_backward(x, z, weight)
        return msel.msel_gated_norm_fwd(x, z, weight, out_layout="bld")

    @staticmethod
    def backward(ctx, dout):
        x, z, weight = ctx.saved_tensors
        g = msel.msel_gated_norm_bwd(x, z, weight, dout.contiguous(), out_layout="bld")
        return g["dx"], g["dz"], g["dweight"]


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate_a, gate_x, lam):
        out, _, cs = msel.msel_lru_fwd(x, gate_a, gate_x, lam, return_final_state=False,
                                       return_chunk_states=True)
        ctx.save_for_backward(x, gate_a, gate_x, lam, cs)
        return out

    @staticmethod
    def backward(ctx, dout):
        x, gate_a, gate_x, lam, cs = ctx.saved_tensors
        g = msel.msel_lru_bwd(x, gate_a, gate_x, lam, dout.contiguous(), chunk_states=cs)
        return g["dx"], g["dgate_a"], g["dgate_x"], g["dlam"]


class GatedMlp(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up):
        ctx.save_for_backward(x, w_gate, w_up)
        return msel.msel_gated_mlp_fwd(x, w_gate, w_up)

    @staticmethod
    def backward(ctx, dout):
        g = msel.msel_gated_mlp_bwd(*ctx.saved_tensors, dout.contiguous())
        return g["dx"], g["dw_gate"], g["dw_up"]


class LogProb(torch.autograd.Function):
    """The log probability of each row's token."""

    @staticmethod
    def forward(ctx, logits, ids):
        r = msel.msel_logprob_fwd(logits, ids)
        ctx.save_for_backward(logits, ids, r["lse"])
        return r["logprob"]

    @staticmethod
    def backward(ctx, dlogprob):
        logits, ids, lse = ctx.saved_tensors
        return msel.msel_logprob_bwd(logits, ids, lse, dlogprob.contiguous()), None


def project(weight, rows):
    """weight [n, k] times each matrix [k, seqlen] of the list `rows`, to [batch, n, seqlen]."""
    return torch.stack([weight @ m for m in rows])


class Block(torch.nn.Module):
    def __init__(self, dim, dstate=16, width=4):
        super().__init__()
        E, R = 2 * dim, max(1, dim // 16)
        self.E, self.R, self.N = E, R, dstate

        def weight(n, k):
            return torch.nn.Parameter(torch.randn(n, k) / math.sqrt(k))

        self.norm = torch.nn.Parameter(torch.ones(dim))
        self.w_in = weight(2 * E, dim)
        self.conv_w = torch.nn.Parameter(torch.randn(E, width) / math.sqrt(width))
        self.conv_b = torch.nn.Parameter(torch.zeros(E))
        self.w_x = weight(R + 2 * dstate, E)
        self.w_dt = weight(E, R)
        # steps of 0.001 to 0.1 after the softplus
        dt = torch.exp(torch.rand(E) * math.log(100.0) + math.log(0.001))
        self.dt_bias = torch.nn.Parameter(dt + torch.log(-torch.expm1(-dt)))
        self.A_log = torch.nn.Parameter(torch.arange(1.0, dstate + 1).log().repeat(E, 1))
        self.D = torch.nn.Parameter(torch.ones(E))
        self.gate_norm = torch.nn.Parameter(torch.ones(E))
        self.w_out = weight(dim, E)

    def inputs(self, h):
        """x and z, [batch, E, seqlen], of h [batch, seqlen, dim]."""
        w = self.w_in.to(h.dtype)
        rows = [m.T for m in h]
        return project(w[:self.E], rows), project(w[self.E:], rows)

    def steps(self, u):
        """delta, B and C of u [batch, E, seqlen]."""
        low = project(self.w_x.to(u.dtype), list(u))
        B = low[:, self.R:self.R + self.N].contiguous()
        C = low[:, self.R + self.N:].contiguous()
        return project(self.w_dt.to(u.dtype), [m[:self.R] for m in low]), B, C

    def output(self, y):
        return (y.reshape(-1, self.E) @ self.w_out.to(y.dtype).T).view(*y.shape[:2], -1)

    def forward(self, x, residual):
        """The block's output (added to the stream by the next norm) and the residual stream."""
        h, residual = Norm.apply(x, self.norm, residual)
        u, z = self.inputs(h)
        u = Conv.apply(u, self.conv_w, self.conv_b)
        delta, B, C = self.steps(u)
        y = Scan.apply(u, delta, -torch.exp(self.A_log), B, C, self.D, self.dt_bias)
        return self.output(GatedNorm.apply(y, z, self.gate_norm)), residual

    @torch.no_grad()
    def step(self, x, residual, state):
        """One token: x [batch, 1, dim]; state {"conv", "scan"} and residual, in place."""
        h, _ = msel.msel_norm_fwd(x, self.norm, residual, residual_out=residual)
        u, z = self.inputs(h)
        u, _ = msel.msel_conv1d_fwd(u, self.conv_w, self.conv_b, state["conv"],
                                    state_out=state["conv"])
        delta, B, C = self.steps(u)
        y, state["scan"], _ = msel.msel_scan_fwd(u, delta, -torch.exp(self.A_log), B, C, self.D,
                                                 None, self.dt_bias, True, state["scan"])
        return self.output(msel.msel_gated_norm_fwd(y, z, self.gate_norm, out_layout="bld"))

    def new_state(self, batch, dev, dtype):
        return {"conv": torch.zeros(batch, self.E, self.conv_w.shape[1] - 1, device=dev,
                                    dtype=dtype),
                "scan": torch.zeros(batch, self.E, self.N, device=dev)}


class LruBlock(torch.nn.Module):
    """Block with the gated linear recurrence in the scan's place."""

    def __init__(self, dim, width=4):
        super().__init__()
        self.E = E = 2 * dim

        def weight(n, k):
            return torch.nn.Parameter(torch.randn(n, k) / math.sqrt(k))

        self.norm = torch.nn.Parameter(torch.ones(dim))
        self.w_in = weight(2 * E, dim)
        self.conv_w = torch.nn.Parameter(torch.randn(E, width) / math.sqrt(width))
        self.conv_b = torch.nn.Parameter(torch.zeros(E))
        self.w_gates = weight(2 * E, E)
        # at an open gate a^8 between 0.9 and 0.999
        a8 = torch.rand(E) * 0.099 + 0.9
        self.rate = torch.nn.Parameter(torch.log(torch.expm1(-torch.log(a8) / 8.0)))
        self.gate_norm = torch.nn.Parameter(torch.ones(E))
        self.w_out = weight(dim, E)

    inputs, output = Block.inputs, Block.output

    def gates(self, u):
        w = self.w_gates.to(u.dtype)
        return project(w[:self.E], list(u)), project(w[self.E:], list(u))

    def lam(self):
        return -8.0 * F.softplus(self.rate)

    def forward(self, x, residual):
        h, residual = Norm.apply(x, self.norm, residual)
        u, z = self.inputs(h)
        u = Conv.apply(u, self.conv_w, self.conv_b)
        y = Recurrence.apply(u, *self.gates(u), self.lam())
        return self.output(GatedNorm.apply(y, z, self.gate_norm)), residual

    @torch.no_grad()
    def step(self, x, residual, state):
        h, _ = msel.msel_norm_fwd(x, self.norm, residual, residual_out=residual)
        u, z = self.inputs(h)
        u, _ = msel.msel_conv1d_fwd(u, self.conv_w, self.conv_b, state["conv"],
                                    state_out=state["conv"])
        y, _, _ = msel.msel_lru_fwd(u, *self.gates(u), self.lam(), state["lru"],
                                    final_state=state["lru"])
        return self.output(msel.msel_gated_norm_fwd(y, z, self.gate_norm, out_layout="bld"))

    def new_state(self, batch, dev, dtype):
        return {"conv": torch.zeros(batch, self.E, self.conv_w.shape[1] - 1, device=dev,
                                    dtype=dtype),
                "lru": torch.zeros(batch, self.E, device=dev)}


class MlpBlock(torch.nn.Module):
    """The gated feed-forward block behind a mixer, with its norm and its way back."""

    def __init__(self, dim, hidden):
        super().__init__()

        def weight(n, k):
            return torch.nn.Parameter(torch.randn(n, k) / math.sqrt(k))

        self.norm = torch.nn.Parameter(torch.ones(dim))
        self.w_gate, self.w_up = weight(hidden, dim), weight(hidden, dim)
        self.w_down = weight(dim, hidden)

    def forward(self, x, residual):
        h, residual = Norm.apply(x, self.norm, residual)
        y = GatedMlp.apply(h, self.w_gate.to(h.dtype), self.w_up.to(h.dtype))
        return y @ self.w_down.to(y.dtype).T, residual

    @torch.no_grad()
    def step(self, x, residual, state):
        h, _ = msel.msel_norm_fwd(x, self.norm, residual, residual_out=residual)
        y = msel.msel_gated_mlp_fwd(h, self.w_gate.to(h.dtype), self.w_up.to(h.dtype))
        return y @ self.w_down.to(y.dtype).T

    def new_state(self, batch, dev, dtype):
        return {}


class Model(torch.nn.Module):
    """mixer: "scan" or "lru"; mlp: the hidden width of a feed-forward block behind every mixer, 0
    for none; own_loss: log probabilities from the library's kernels, not PyTorch's."""

    def __init__(self, vocab, dim, layers, dtype=torch.bfloat16, mixer="scan", mlp=0,
                 own_loss=False):
        super().__init__()
        self.vocab, self.dim, self.dtype, self.own_loss = vocab, dim, dtype, own_loss
        self.table = torch.nn.Parameter(torch.randn(vocab, dim) / math.sqrt(dim))
        self.scale = math.sqrt(dim)  # of the embedding: its rows then have unit variance
        blocks = []
        for _ in range(layers):
            blocks.append(Block(dim) if mixer == "scan" else LruBlock(dim))
            if mlp:
                blocks.append(MlpBlock(dim, mlp))
        self.blocks = torch.nn.ModuleList(blocks)
        self.norm = torch.nn.Parameter(torch.ones(dim))

    def logits(self, h):
        return h.reshape(-1, self.dim) @ self.table.to(h.dtype).T

    def head(self, h):
        return self.logits(h).float()

    def loss(self, ids, targets):
        """Cross entropy, and the embedding's output as the leaf that its gradient stops at."""
        emb = msel.msel_embed_fwd(ids, self.table.detach(), self.scale).requires_grad_()
        x, residual = torch.zeros_like(emb, dtype=self.dtype), emb
        for b in self.blocks:
            x, residual = b(x, residual)
        h, _ = Norm.apply(x, self.norm, residual)
        if self.own_loss:
            return -LogProb.apply(self.logits(h), targets.reshape(-1)).mean(), emb
        return F.cross_entropy(self.head(h), targets.reshape(-1)), emb

    def backward(self, loss, emb, ids):
        loss.backward()
        # the table is the head's weight too: the embedding's gradient is added to that one
        g = self.table.grad
        msel.msel_embed_bwd(ids, emb.grad, self.vocab, self.scale, base=g, dweight=g)

    @torch.no_grad()
    def new_state(self, batch):
        return [b.new_state(batch, self.table.device, self.dtype) for b in self.blocks]

    @torch.no_grad()
    def step(self, ids, state):
        """Logits [batch, vocab] of one token per sequence."""
        residual = msel.msel_embed_fwd(ids.contiguous()[:, None], self.table.detach(), self.scale)
        x = torch.zeros_like(residual, dtype=self.dtype)
        for b, s in zip(self.blocks, state):
            x = b.step(x, residual, s)
        h, _ = msel.msel_norm_fwd(x, self.norm, residual)
        return self.head(h)


def batches(vocab, batch, seqlen, period, seed, device):
    """Sequences that repeat a random pattern of `period` tokens."""
    g = torch.Generator().manual_seed(seed)
    while True:
        pattern = torch.randint(vocab, (batch, period), generator=g)
        ids = pattern.repeat(1, seqlen // period + 2)[:, :seqlen + 1].to(device)
        yield ids[:, :-1].contiguous(), ids[:, 1:].contiguous()


def train(model, data, steps, lr=2e-3, max_norm=1.0, report=None):
    """Returns the losses."""
    opt = torch.optim.AdamW(model.parameters(), lr=lr, betas=(0.9, 0.95), weight_decay=0.0)
    grads, losses = None, []
    for k in range(steps):
        ids, targets = next(data)
        opt.zero_grad(set_to_none=False)
        loss, emb = model.loss(ids, targets)
        model.backward(loss, emb, ids)
        if grads is None:  # the gradients stay the same tensors from here on
            grads = msel.GradList(p.grad for p in model.parameters())
        norm = msel.msel_grad_clip(grads, max_norm)
        opt.step()
        losses.append(loss.item())
        if report and (k % report == 0 or k == steps - 1):
            print(f"step {k:4d}  loss {losses[-1]:.4f}  gradient norm {float(norm):.3f}", flush=True)
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--vocab", type=int, default=61)
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--seqlen", type=int, default=96)
    ap.add_argument("--period", type=int, default=3)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    ap.add_argument("--mixer", choices=("scan", "lru"), default="scan")
    ap.add_argument("--mlp", type=int, default=0)
    ap.add_argument("--loss", choices=("library", "own"), default="library")
    a = ap.parse_args()
    torch.manual_seed(0)
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    model = Model(a.vocab, a.dim, a.layers, dtype, a.mixer, a.mlp, a.loss == "own").cuda()
    data = batches(a.vocab, a.batch, a.seqlen, a.period, 1, "cuda")
    train(model, data, a.steps, report=10)
    # continue a pattern token by token
    ids, _ = next(data)
    state = model.new_state(a.batch)
    for t in range(2 * a.period):
        logits = model.step(ids[:, t], state)
    right, scores = 0, []
    for t in range(2 * a.period, 4 * a.period):
        if a.loss == "own":
            r = msel.msel_logprob_fwd(logits, top=1, want_entropy=True)
            token = r["top_ids"][:, 0]
            scores.append(torch.stack([r["top_logprobs"][:, 0], r["entropy"]]))
        else:
            token = logits.argmax(-1)
        right += int((token == ids[:, t]).sum())
        logits = model.step(token, state)
    print(f"continued tokens that follow the pattern: {right} of {2 * a.period * a.batch}")
    if scores:
        logprob, entropy = torch.stack(scores).mean((0, 2)).tolist()
        print(f"their mean log probability {logprob:.4f}, the mean entropy {entropy:.4f}")


if __name__ == "__main__":
    main()
