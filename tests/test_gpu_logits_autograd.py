"""The differentiable forms of the logit operators as a training loop uses them."""

import pytest

from tests._helpers import announce, require_gpu

pytestmark = pytest.mark.gpu


def both(torch):
    """name -> (function of the logits that gives the form's outputs)"""
    import bit_block_scaled_bf16_amd as nv
    from bit_block_scaled_bf16_amd.logits import DistillFunction, TokenLogprobsFunction

    rows, vocab = 5, 700
    torch.manual_seed(1)
    z = torch.randn(rows, vocab, device="cuda") * 2
    tok = torch.arange(rows, device="cuda")
    t = nv.token_logprobs(z + 0.3 * torch.randn_like(z), top_k=7)
    return z, {"token_logprobs": lambda x: TokenLogprobsFunction.apply(x, tok, 1.0),
               "distill": lambda x: DistillFunction.apply(x, t.top_ids, t.top_logp, tok, True, 1.0)}


@pytest.mark.parametrize("name", ["token_logprobs", "distill"])
def test_outputs_may_be_changed_in_place(name):
    """loss.mul_(weights), logp.masked_fill_(...): each output is a tensor of its
    own, and the gradient is that of the same product out of place."""
    torch = require_gpu()
    announce(f"in place {name}")
    z, forms = both(torch)
    mask = torch.arange(z.shape[0], device="cuda") == 2
    w = torch.rand(z.shape[0], device="cuda")
    grads = []
    for in_place in (False, True):
        for which in (0, 1) if name == "distill" else (0,):  # (the entropy is kept for the gradient)
            x = z.clone().requires_grad_(True)
            y = forms[name](x)
            other = y[1 - which].detach().clone()
            v = y[which]
            if in_place:
                v.mul_(w)
                v.masked_fill_(mask, 0.0)
            else:
                v = (v * w).masked_fill(mask, 0.0)
            assert torch.equal(y[1 - which], other)
            v.sum().backward()
            grads.append(x.grad)
    half = len(grads) // 2
    for a, b in zip(grads[:half], grads[half:]):
        assert torch.equal(a, b)


def test_outputs_share_no_storage():
    torch = require_gpu()
    announce("storage")
    z, forms = both(torch)
    for name, form in forms.items():
        y = form(z.clone().requires_grad_(True))
        assert y[0].untyped_storage().data_ptr() != y[1].untyped_storage().data_ptr(), name
        assert not y[0]._is_view() and not y[1]._is_view(), name


@pytest.mark.parametrize("name", ["token_logprobs", "distill"])
def test_second_derivatives_are_refused(name):
    """They are not computed: asking for one raises instead of dropping it."""
    torch = require_gpu()
    announce(f"second derivative {name}")
    z, forms = both(torch)
    x = z.clone().requires_grad_(True)
    g, = torch.autograd.grad(sum(t.sum() for t in forms[name](x)), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.square().sum().backward()
