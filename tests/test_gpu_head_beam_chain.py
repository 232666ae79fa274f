"""The operators run together, as a program would: beam search from hidden states to reordered caches, and a training
step from hidden states through the head and the distillation loss back to their gradient."""
import numpy as np
import pytest
import torch

from vocab_wide_draft_amd import binding as B

import beam_oracle as O
from head_oracle import wide, worth

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")


def _head(V, D, kind, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn((V, D), generator=g) * D ** -0.5 * 4
    q = B.quantize_blocks(wide(w, dev), 128, kind)
    return {"weight": q, "transposed": B.transpose_blocks(q, D)}


def _search(kind, END):
    """Twelve steps of three requests with four beams: hidden states from a cache of token vectors, logits from the 8-bit
    head, shaped by penalties, a mask and a temperature, selected, and the caches reordered.  Each step against the plain
    form of the operators on the step's own inputs."""
    R, Bm, V, D, T, steps = 3, 4, 1200, 96, 12, 12
    head = _head(V, D, kind, 1)
    W = worth(head["weight"], 128)[:, :D]
    g = torch.Generator().manual_seed(2)
    embed = torch.randn((V, D), generator=g).to(dev)
    embed[7] *= 3
    mask = torch.randint(-2**31, 2**31, (1, -(-V // 32)), generator=g, dtype=torch.int64).to(torch.int32).to(dev)
    cache = torch.zeros((R, Bm, T + 1, D), device=dev)
    cache[:, :, 0] = embed[torch.tensor([11, 12, 13])].view(R, 1, D)
    history = torch.zeros((R, Bm, T + 1), dtype=torch.int32, device=dev)
    scores = torch.full((R, Bm), -float("inf"), device=dev)
    scores[:, 0] = 0.0
    finished = torch.zeros((R, Bm), dtype=torch.int32, device=dev)
    presence, temp = torch.full((R * Bm,), 0.4, device=dev), torch.full((R * Bm,), 0.8, device=dev)
    ended, tokens = 0, []
    for step in range(steps):
        n = step + 1
        hidden = (cache[:, :, :n].sum(2) / n ** 0.5).view(R * Bm, D)
        logits = B.head_logits(hidden, head)
        xq = worth(B.quantize_blocks(hidden, 1, kind), 1)[:, :D]
        size = xq.abs() @ W.abs().t()
        assert ((logits.cpu().double() - xq @ W.t()).abs() <= size * (D + 8) * 2.0 ** -24).all()
        shaped = B.shape_logits(logits, 1, history=history.view(R * Bm, T + 1), history_len=torch.full((R * Bm,), step, dtype=torch.int32, device=dev),
                                presence=presence, temperature=temp, mask=mask, mask_row=torch.where(torch.arange(R * Bm, device=dev) % 3 == 1, 0, -1).to(torch.int32))
        assert not shaped["status"].any()
        out = B.beam_select(shaped["logits"], scores, Bm, finished=finished, end_token=END)
        want = O.select(shaped["logits"].cpu().numpy(), scores.cpu().numpy(), Bm, finished.cpu().numpy(), END)
        for name, w in zip(("parent", "token"), want):
            np.testing.assert_array_equal(out[name].cpu().numpy(), w)
        np.testing.assert_array_equal(out["finished"].cpu().numpy(), want[3])
        assert (out["len"] == Bm).all() and not out["status"].any()
        before = [cache.cpu().clone(), history.cpu().clone()]
        length = torch.full((R,), n, dtype=torch.int32, device=dev)
        assert not B.beam_reorder([cache, history], out["parent"], length)["status"].any()
        for now, old in zip((cache, history), before):
            w = old.clone()
            for r in range(R):
                for b in range(Bm):
                    w[r, b, :n] = old[r, int(want[0][r, b]), :n]
            assert torch.equal(now.cpu(), w)
        scores, finished = out["score"], out["finished"]
        history[:, :, step] = out["token"]
        if n < T:
            cache[:, :, n] = embed[out["token"].long()]
        ended += int(finished.sum())
        tokens += out["token"].flatten().tolist()
    assert (scores[:, :-1] >= scores[:, 1:]).all() and torch.isfinite(scores).all()
    return ended, tokens


@pytest.mark.parametrize("kind", [torch.float32, torch.float8_e8m0fnu])
def test_beam_search(kind):
    _, tokens = _search(kind, 7)
    # once more, ended by a token that the search selects
    ended, _ = _search(kind, max(set(tokens), key=tokens.count))
    assert ended > 0


def _teacher(n, V, k, seed):
    g = torch.Generator().manual_seed(seed)
    return B.top_logits(wide(torch.randn((n, V), generator=g) * 3, dev), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V,D", [(7, 900, 200), (70, 4000, 512)])
def test_training_step(n, V, D, dtype):
    """The gradient of the mean distillation loss with respect to the hidden states is the logits' gradient through the
    transposed head, whatever hands it over."""
    head = _head(V, D, torch.float8_e8m0fnu, 3)
    teacher = _teacher(n, V, 32, 4)
    x = wide(torch.randn((n, D), generator=torch.Generator().manual_seed(5)).to(dtype), dev).requires_grad_()
    logits = B.head_logits(x, head)
    B.distill_loss(logits, teacher).mean().backward()
    at = logits.detach().requires_grad_()
    B.distill_loss(at, teacher).mean().backward()
    assert torch.equal(x.grad, B.block_linear(wide(at.grad.cpu(), dev), head["transposed"], dtype))


def test_training_step_in_a_graph():
    """Forward and backward captured together and replayed with other hidden states."""
    n, V, D = 40, 3000, 256
    head, teacher = _head(V, D, torch.float32, 3), _teacher(n, V, 16, 4)
    inputs = [torch.randn((n, D), generator=torch.Generator().manual_seed(k)).to(torch.bfloat16).to(dev) for k in (1, 2)]

    def run(x):
        loss = B.distill_loss(B.head_logits(x, head, torch.float32), teacher)
        return loss, torch.autograd.grad(loss.sum(), x)[0]

    want = [[t.detach().clone() for t in run(x.clone().requires_grad_())] for x in inputs]
    x = inputs[0].clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss, grad = run(x)
    for k in (1, 0, 1):
        with torch.no_grad():
            x.copy_(inputs[k])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[k][0]) and torch.equal(grad, want[k][1])
        run(inputs[0].clone().requires_grad_())


def test_saved_tensor_hooks_are_heard():
    """Checkpointing or host offload: the backward pass uses what the hooks give back."""
    head = _head(600, 128, torch.float32, 3)
    x = torch.randn((5, 128), device=dev).requires_grad_()
    up = torch.randn((5, 600), device=dev)
    (want,) = torch.autograd.grad(B.head_logits(x, head), x, up)
    with torch.autograd.graph.save_on_cpu():
        y = B.head_logits(x, head)
    (got,) = torch.autograd.grad(y, x, up)
    assert torch.equal(got, want)
    y = torch.utils.checkpoint.checkpoint(lambda t: B.head_logits(t, head), x, use_reentrant=False)
    (got,) = torch.autograd.grad(y, x, up)
    assert torch.equal(got, want)
