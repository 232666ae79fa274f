"""Derivatives that head_logits does not have are refused before any device work; so none is lost in silence."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from vocab_wide_draft_amd import binding as B


def _head(width=128, V=16):
    w = {"values": torch.zeros(V, width).to(torch.float8_e4m3fn), "scales": torch.ones(1, -(-width // 128))}
    return {"weight": w, "transposed": B.transpose_blocks(w, width)}


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("out", [None, torch.float32])
def test_forward_mode_tangents_are_refused(out, grad):
    x, t = torch.ones(2, 128), torch.ones(2, 128)
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        with pytest.raises(NotImplementedError, match="forward-mode"):
            B.head_logits(forward_ad.make_dual(x, t), _head(), out)
        with pytest.raises(ValueError, match="on the GPU"):  # without a tangent the call goes on to its other checks
            B.head_logits(x, _head(), out)


def test_forward_mode_through_functions_of_functions():
    x = torch.ones(2, 128)
    for derivative in (lambda f: torch.func.jvp(f, (x,), (x,)), lambda f: torch.func.jacfwd(f)(x)):
        with pytest.raises(NotImplementedError, match="forward-mode"):
            derivative(lambda t: B.head_logits(t, _head()))


@pytest.mark.parametrize("part", ["weight", "transposed"])
def test_the_head_is_constant_whatever_x_needs(part):
    """A head that a derivative is asked of is refused, also where x itself needs none; without derivatives it is taken."""
    x, head = torch.ones(2, 128), _head()
    head[part]["scales"].requires_grad_()
    for t in (x, x.clone().requires_grad_()):
        with pytest.raises(ValueError, match="constant"):
            B.head_logits(t, head)
    with torch.no_grad(), pytest.raises(ValueError, match="on the GPU"):
        B.head_logits(x, head)
    head[part]["scales"].requires_grad_(False)
    with forward_ad.dual_level():
        head[part] = {"values": head[part]["values"], "scales": forward_ad.make_dual(head[part]["scales"], torch.ones_like(head[part]["scales"]))}
        with pytest.raises(ValueError, match="constant"):
            B.head_logits(x, head)
