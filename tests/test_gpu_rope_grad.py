"""Gradients through kvc.rope: the transposed rotation, never dropped silently."""
import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
from oracle import paged as og
import paged_utils as u
from q8_utils import dev_bf16, random_rows

pytestmark = pytest.mark.gpu


def _freq(r):
    return 10000.0 ** (-2.0 * np.arange(r // 2) / r)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("n,H,d,r,inter,m", [(5, 3, 64, 64, False, 1.0), (7, 2, 128, 26, True, 1.2), (1, 1, 128, 2, False, -0.5), (0, 2, 64, 64, False, 1.0)])
def test_gradient_is_the_transposed_rotation(n, H, d, r, inter, m, back):
    plan = kvc.Rope(u.dev(_freq(r)), interleaved=inter, mscale=m)
    at = torch.arange(n, dtype=torch.int32, device="cuda") * 977
    x = dev_bf16(random_rows(1, n, H, d)).requires_grad_()
    g = dev_bf16(random_rows(2, n, H, d))
    y = kvc.rope(plan, x, at, backward=back)
    assert y.requires_grad and torch.equal(y.detach().view(torch.int16), kvc.rope(plan, x.detach(), at, backward=back).view(torch.int16))
    y.backward(g)
    ref, size = og.rope(og.widen(u.bits(g)), at.cpu().numpy(), _freq(r), m, inter, not back)
    u.check_rope(u.bits(x.grad), ref, size, m)
    # in a longer program: the slice of a projection, used twice, an expanded gradient
    w = dev_bf16(random_rows(3, n, H + 2, d)).requires_grad_()
    z = kvc.rope(plan, w[:, 1: 1 + H], at, backward=back)
    (z.sum() + (z * g).sum()).backward()
    ones = torch.ones_like(g)
    want = kvc.rope(plan, (ones + g).contiguous(), at, backward=not back)
    assert torch.equal(w.grad[:, 1: 1 + H], want) and not bool(w.grad[:, 0].any()) and not bool(w.grad[:, H + 1:].any())


def test_gradient_by_differences():
    """The map is linear: f(x + e) - f(x - e) for steps that bf16 holds, against <gradient, e>."""
    n, H, d, r = 3, 2, 64, 40
    plan = kvc.Rope(u.dev(_freq(r)), mscale=1.3)
    at = torch.tensor([0, 5, 100000], dtype=torch.int32, device="cuda")
    g = dev_bf16(random_rows(4, n, H, d))
    x = torch.zeros((n, H, d), dtype=torch.bfloat16, device="cuda").requires_grad_()
    kvc.rope(plan, x, at).backward(g)
    for where in ((0, 0, 0), (1, 1, 19), (2, 0, 25), (2, 1, 39), (1, 0, 50)):
        e = torch.zeros_like(g)
        e[where] = 1.0
        with torch.no_grad():
            diff = ((kvc.rope(plan, e, at).double() - kvc.rope(plan, -e, at).double()) * g.double()).sum() / 2
        # each rotated value and the gradient are rounded to bf16 once
        room = 2.0 ** -8 * 4 * 1.3 * float(g[where[0], where[1]].double().abs().max())
        assert abs(float(diff - x.grad[where].double())) <= room


def test_second_gradients_streams_and_refusals():
    plan = kvc.Rope(u.dev(_freq(64)))
    at = torch.arange(4, dtype=torch.int32, device="cuda")
    x = dev_bf16(random_rows(5, 4, 2, 64)).requires_grad_()
    g = dev_bf16(random_rows(6, 4, 2, 64)).requires_grad_()
    (gx,) = torch.autograd.grad(kvc.rope(plan, x, at), x, g, create_graph=True)
    (gg,) = torch.autograd.grad(gx, g, dev_bf16(random_rows(7, 4, 2, 64)))
    assert torch.equal(gg.view(torch.int16), kvc.rope(plan, dev_bf16(random_rows(7, 4, 2, 64)), at).view(torch.int16))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = kvc.rope(plan, x, at, stream=s)
    s.synchronize()
    assert torch.equal(y.detach().view(torch.int16), kvc.rope(plan, x.detach(), at).view(torch.int16))
    out = torch.empty_like(x.detach())
    for a, b in ((x, out), (x, x), (x.detach(), out.clone().requires_grad_())):
        with pytest.raises(ValueError):
            kvc.rope(plan, a, at, y=b)
    with torch.no_grad():
        assert kvc.rope(plan, x, at, y=out) is out and not kvc.rope(plan, x, at).requires_grad
        kvc.rope(plan, x, at, y=x)
    assert torch.equal(x.detach().view(torch.int16), out.view(torch.int16))
