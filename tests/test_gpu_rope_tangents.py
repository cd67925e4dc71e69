"""Forward-mode derivatives of ops.rope (torch.autograd.forward_ad): a linear map's tangent is
the map of the tangent, in forward passes, through ops.attention, and in backward passes."""
import pytest
import torch
import torch.autograd.forward_ad as fwd_ad

from block_sparse_gqa_topk_gb300 import ops

pytestmark = pytest.mark.gpu


def randn(shape, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("given", [False, True])
def test_tangents_are_turned(given):
    r = ops.new_rope(16, interleaved=True)
    q, k, dq = randn((2, 5, 3, 24), 1), randn((2, 5, 24), 2), randn((2, 5, 3, 24), 3)
    pos = torch.arange(10, device="cuda").view(2, 5) * 7 if given else None
    want, turned = ops.msa_rope((q, k), r, pos), ops.msa_rope(dq, r, pos)[0]
    with fwd_ad.dual_level():
        y, z = ops.rope((fwd_ad.make_dual(q, dq), k), r, pos)
        py, pz = fwd_ad.unpack_dual(y), fwd_ad.unpack_dual(z)
        assert torch.equal(py.primal, want[0]) and torch.equal(pz.primal, want[1])
        assert torch.equal(py.tangent, turned)
        assert pz.tangent is None or not pz.tangent.any()
        # without tangents, and with an input that wants a gradient beside one with a tangent
        assert fwd_ad.unpack_dual(ops.rope(q, r, pos)[0]).tangent is None
        k2 = k.clone().requires_grad_()
        y, z = ops.rope((fwd_ad.make_dual(q, dq), k2), r, pos)
        assert torch.equal(fwd_ad.unpack_dual(y).tangent, turned)
        dz = randn(z.shape, 4)
        (g,) = torch.autograd.grad(z, k2, dz)
        assert torch.equal(fwd_ad.unpack_dual(g).primal, ops.msa_rope(dz, r, pos, inverse=True)[0])


def test_tangents_of_gradients():
    """A backward pass within a dual level: the gradient's own tangent."""
    r = ops.new_rope(16)
    x, dy, t = randn((4, 2, 16), 5).requires_grad_(), randn((4, 2, 16), 6), randn((4, 2, 16), 7)
    pos = torch.arange(4, device="cuda")
    with fwd_ad.dual_level():
        (y,) = ops.rope(x, r, pos)
        (g,) = torch.autograd.grad(y, x, fwd_ad.make_dual(dy, t))
        g = fwd_ad.unpack_dual(g)
        assert torch.equal(g.primal, ops.msa_rope(dy, r, pos, inverse=True)[0])
        assert torch.equal(g.tangent, ops.msa_rope(t, r, pos, inverse=True)[0])


def test_attention_and_in_place_calls_do_not_drop_them():
    """The attention has no forward-mode derivative and says so, with a rope as without one; a
    tensor with a tangent is not turned in place."""
    bf = torch.bfloat16
    q, k, v = randn((1, 130, 2, 64), 8, bf), randn((1, 130, 1, 64), 9, bf), randn((1, 130, 1, 64), 10, bf)
    qi, ki = randn((1, 130, 1, 32), 11, bf), randn((1, 130, 32), 12, bf)
    r = ops.new_rope(32)
    with fwd_ad.dual_level():
        dual = fwd_ad.make_dual(q, torch.ones_like(q))
        for kw in (dict(), dict(rope=r)):
            with pytest.raises((RuntimeError, NotImplementedError)):
                ops.attention(dual, k, v, qi, ki, 1, **kw)
        before = q.clone()
        with pytest.raises(ValueError):
            ops.msa_rope(dual, r, inplace=True)
        assert torch.equal(q, before)
        ops.msa_rope(ki, r, inplace=True)  # without a tangent it is
    assert ops.device_status() == 0
