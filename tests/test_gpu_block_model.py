"""A language model of the gated recurrence, the gated feed-forward block and the library's log
probabilities (examples/train_lm.py with those options) on the GPU: its loss and all its gradients
against the same model written out plainly in fp64 on the CPU, its steps for single tokens against
the whole sequence, and that it runs in bf16."""
import math
import os
import sys

import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import train_lm  # noqa: E402


def plain_loss(p, ids, targets, blocks, scale, eps=1e-5):
    """The model on fp64 parameters p, one operation at a time; blocks: "lru" or "mlp" each."""
    def norm(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w

    def silu(v):
        return v * torch.sigmoid(v)

    s = p["table"][ids] * scale
    for i, kind in enumerate(blocks):
        q = {k.split(".", 2)[2]: v for k, v in p.items() if k.startswith(f"blocks.{i}.")}
        h = norm(s, q["norm"])
        if kind == "mlp":
            s = s + (silu(h @ q["w_gate"].T) * (h @ q["w_up"].T)) @ q["w_down"].T
            continue
        x, z = (h @ q["w_in"].T).chunk(2, -1)
        W = q["conv_w"].shape[1]
        pad = torch.nn.functional.pad(x, (0, 0, W - 1, 0))
        u = silu(sum(pad[:, j:j + x.shape[1]] * q["conv_w"][:, j] for j in range(W)) + q["conv_b"])
        ga, gx = (u @ q["w_gates"].T).chunk(2, -1)
        lam = -8.0 * torch.nn.functional.softplus(q["rate"])
        state, ys = 0.0, []
        for t in range(x.shape[1]):
            a = torch.exp(lam * torch.sigmoid(ga[:, t]))
            state = a * state + torch.sqrt(1 - a * a) * torch.sigmoid(gx[:, t]) * u[:, t]
            ys.append(state)
        s = s + norm(torch.stack(ys, 1) * silu(z), q["gate_norm"]) @ q["w_out"].T
    logits = norm(s, p["norm"]) @ p["table"].T
    return torch.nn.functional.cross_entropy(logits.reshape(-1, logits.shape[-1]),
                                             targets.reshape(-1))


def _model(dim=24, layers=2, vocab=31, dtype=torch.float32, mlp=40):
    torch.manual_seed(3)
    m = train_lm.Model(vocab, dim, layers, dtype, "lru", mlp, True)
    with torch.no_grad():  # norms and biases away from their neutral values
        for n, q in m.named_parameters():
            if "norm" in n or n.endswith("conv_b"):
                q.add_(torch.randn_like(q) * 0.1)
    return m.cuda()


def test_loss_and_gradients_against_the_plain_model():
    # fp32 throughout: some 40 operations deep, each with relative errors of at most a few hundred
    # roundings of 2^-24 (sums of 24 to 74 terms, the recurrence over 37 steps) that the norms keep
    # from growing: 2^-24 * 40 * 300 = 7e-4 of a gradient's largest element
    log("block model gradients")
    m = _model()
    ids, targets = next(train_lm.batches(31, 3, 37, 5, 7, "cuda"))
    loss, emb = m.loss(ids, targets)
    m.backward(loss, emb, ids)
    p = {n: q.detach().double().cpu().requires_grad_() for n, q in m.named_parameters()}
    ref = plain_loss(p, ids.cpu(), targets.cpu(), ["lru", "mlp"] * 2, m.scale)
    ref.backward()
    assert abs(loss.item() - ref.item()) <= 1e-5 * ref.item()
    for n, q in m.named_parameters():
        err = float((q.grad.double().cpu() - p[n].grad).abs().max() / p[n].grad.abs().max())
        assert err <= 7e-4, (n, err)


def test_single_tokens_give_the_sequence():
    log("block model steps")
    m = _model()
    ids, _ = next(train_lm.batches(31, 3, 9, 4, 7, "cuda"))
    state = m.new_state(3)
    steps = torch.stack([m.step(ids[:, t], state) for t in range(ids.shape[1])], 1)
    with torch.no_grad():
        emb = train_lm.msel.msel_embed_fwd(ids, m.table.detach(), m.scale)
        x, residual = torch.zeros_like(emb), emb
        for b in m.blocks:
            x, residual = b(x, residual)
        whole = m.head(train_lm.Norm.apply(x, m.norm, residual)[0]).view_as(steps)
    assert float((steps - whole).abs().max()) <= 7e-4 * float(whole.abs().max())


@pytest.mark.parametrize("mixer", ["scan", "lru"])
def test_it_runs_in_bf16(mixer):
    log(f"block model training {mixer}")
    torch.manual_seed(0)
    m = train_lm.Model(31, 64, 2, torch.bfloat16, mixer, 96, True).cuda()
    losses = train_lm.train(m, train_lm.batches(31, 8, 64, 2, 1, "cuda"), 4)
    assert all(math.isfinite(v) for v in losses)
    for n, q in m.named_parameters():
        assert torch.isfinite(q.grad).all() and bool((q.grad != 0).any()), n


def test_a_captured_backward_beside_a_living_graph():
    """A backward pass of these operators captured while an eager autograd graph of the same leaves
    lives: both give the eager gradients."""
    log("captured backward")
    x = torch.randn(64, 48, device="cuda").bfloat16().requires_grad_()
    w = [torch.randn(80, 48, device="cuda").bfloat16().mul_(0.1).requires_grad_() for _ in range(2)]
    ids = torch.arange(64, device="cuda") % 80
    leaves = [x, *w]

    def grads():
        h = train_lm.GatedMlp.apply(x, *w)
        loss = -train_lm.LogProb.apply(h, ids).mean()
        return torch.autograd.grad(loss, leaves)
    ref = [g.clone() for g in grads()]
    alive = -train_lm.LogProb.apply(train_lm.GatedMlp.apply(x, *w), ids).mean()
    # the capture has leaves of its own: it shares their memory, and no autograd node with `alive`
    x2, w2 = x.detach().requires_grad_(), [v.detach().requires_grad_() for v in w]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())

    def captured():
        loss = -train_lm.LogProb.apply(train_lm.GatedMlp.apply(x2, *w2), ids).mean()
        return torch.autograd.grad(loss, [x2, *w2])
    with torch.cuda.stream(side):
        for _ in range(2):
            captured()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            cap = captured()
    torch.cuda.synchronize()
    for _ in range(3):
        for c in cap:
            c.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for c, r in zip(cap, ref):
            assert torch.equal(c, r)
    for g, r in zip(torch.autograd.grad(alive, leaves), ref):
        assert torch.equal(g, r)
