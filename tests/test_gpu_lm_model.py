"""The language model of examples/train_lm.py on the GPU: its loss and all its gradients against
the same model written out plainly in fp64 on the CPU (token by token, with autograd), its steps
for single tokens against the whole sequence, and that it learns."""
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


def plain_loss(p, ids, targets, layers, scale, eps=1e-5):
    """The model on fp64 parameters p, one operation at a time."""
    def norm(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w

    s = p["table"][ids] * scale
    for i in range(layers):
        q = {k.split(".", 2)[2]: v for k, v in p.items() if k.startswith(f"blocks.{i}.")}
        h = norm(s, q["norm"])
        x, z = (h @ q["w_in"].T).chunk(2, -1)              # [batch, seqlen, E]
        W = q["conv_w"].shape[1]
        pad = torch.nn.functional.pad(x, (0, 0, W - 1, 0))
        u = sum(pad[:, j:j + x.shape[1]] * q["conv_w"][:, j] for j in range(W)) + q["conv_b"]
        u = u * torch.sigmoid(u)
        N, R = q["A_log"].shape[1], q["w_dt"].shape[1]
        low = u @ q["w_x"].T
        B, C = low[..., R:R + N], low[..., R + N:]
        delta = torch.nn.functional.softplus(low[..., :R] @ q["w_dt"].T + q["dt_bias"])
        A = -torch.exp(q["A_log"])
        state, ys = 0.0, []
        for t in range(x.shape[1]):
            d = delta[:, t, :, None]
            state = torch.exp(d * A) * state + d * B[:, t, None] * u[:, t, :, None]
            ys.append((state * C[:, t, None]).sum(-1) + q["D"] * u[:, t])
        y = torch.stack(ys, 1)
        s = s + norm(y * (z * torch.sigmoid(z)), q["gate_norm"]) @ q["w_out"].T
    logits = norm(s, p["norm"]) @ p["table"].T
    return torch.nn.functional.cross_entropy(logits.reshape(-1, logits.shape[-1]),
                                             targets.reshape(-1))


def _model(dim=24, layers=2, vocab=31, dtype=torch.float32):
    torch.manual_seed(3)
    m = train_lm.Model(vocab, dim, layers, dtype)
    with torch.no_grad():  # norms and biases away from their neutral values
        for n, q in m.named_parameters():
            if "norm" in n or n.endswith(("conv_b", ".D")):
                q.add_(torch.randn_like(q) * 0.1)
    return m.cuda()


def test_loss_and_gradients_against_the_plain_model():
    # fp32 throughout: the model is about 30 operations deep, each with relative errors of at most
    # a few hundred roundings of 2^-24 (sums of 24 to 74 terms, the scan over 37 steps) that the
    # norms keep from growing: 2^-24 * 30 * 300 = 5e-4 of a gradient's largest element
    log("model gradients")
    m = _model()
    ids, targets = next(train_lm.batches(31, 3, 37, 5, 7, "cuda"))
    loss, emb = m.loss(ids, targets)
    m.backward(loss, emb, ids)
    p = {n: q.detach().double().cpu().requires_grad_() for n, q in m.named_parameters()}
    ref = plain_loss(p, ids.cpu(), targets.cpu(), 2, m.scale)
    ref.backward()
    assert abs(loss.item() - ref.item()) <= 1e-5 * ref.item()
    for n, q in m.named_parameters():
        err = float((q.grad.double().cpu() - p[n].grad).abs().max() / p[n].grad.abs().max())
        assert err <= 5e-4, (n, err)


def test_single_tokens_give_the_sequence():
    log("model steps")
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
    assert float((steps - whole).abs().max()) <= 5e-4 * float(whole.abs().max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_it_learns(dtype):
    """A pattern of period 2: the loss falls from about log(vocab) to less than half of it."""
    log(f"model training {dtype}")
    torch.manual_seed(0)
    m = train_lm.Model(31, 64, 2, dtype).cuda()
    losses = train_lm.train(m, train_lm.batches(31, 16, 64, 2, 1, "cuda"), 40)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.5 * losses[0], (losses[0], losses[-1])
