"""Rotary positions (ops.msa_rope, ops.rope) against their formula in 64 bits.

Tolerance, by arithmetic: the angle's fraction of a turn is rounded once to float32 (at most
pi * 2^-24 radians), the sine and cosine are within 2 ulp (2^-23 each) and the two products
and their sum round at most twice (2^-23 of each product): below 1e-6 m (|x1| + |x2|)
together.  The result is then rounded once to its type: half a step, eps / 2 of the value
(plus half the smallest step for a subnormal float16)."""
import fractions
import math

import numpy as np
import pytest
import torch

from block_sparse_gqa_topk_gb300 import ops
from parity import f64, to_dev  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SCALINGS = {"none": None, "linear": {"type": "linear", "factor": 2.5},
            "ntk": {"type": "ntk", "factor": 4.0},
            "yarn": {"type": "yarn", "factor": 8.0, "original_len": 4096}}


def frequencies(rot, scaling, base=10000.0):
    """The documented formulas, written apart from the library's."""
    out, m = [], 1.0
    for i in range(rot // 2):
        f = math.exp(-2 * i / rot * math.log(base))
        if scaling and scaling["type"] == "linear":
            f /= scaling["factor"]
        if scaling and scaling["type"] == "ntk":
            f = math.exp(-2 * i / rot * math.log(base * scaling["factor"] ** (rot / (rot - 2))))
        if scaling and scaling["type"] == "yarn":
            r = scaling["original_len"] * f / (2 * math.pi)
            g = 1.0 if r >= 32 else 0.0 if r <= 1 else (r - 1) / 31
            f = f * (g + (1 - g) / scaling["factor"])
            m = 0.1 * math.log(scaling["factor"]) + 1
        out.append(f)
    return np.array(out), m


def reference(x, pos, freq, m, rot, inter, back=False):
    """x float64 [.., H, d], pos [..]: (y, the tolerance's |x1| + |x2| per value)."""
    a = pos[..., None, None] * freq
    c, s = np.cos(a) * m, np.sin(a) * m * (-1 if back else 1)
    y, size = x.copy(), np.zeros_like(x)
    i = np.arange(rot // 2)
    p1, p2 = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    x1, x2 = x[..., p1], x[..., p2]
    y[..., p1], y[..., p2] = x1 * c - x2 * s, x2 * c + x1 * s
    size[..., p1] = size[..., p2] = m * (np.abs(x1) + np.abs(x2))
    return y, size


def check(got, want, size, dtype):
    step = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    tol = step * (np.abs(want) + 1e-6 * size) + 1e-6 * size + tiny
    off = np.abs(f64(got.detach()) - want)
    assert (off <= tol).all(), (off - tol).max()


def randn(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("scaling", sorted(SCALINGS))
def test_matches_formula(dtype, inter, scaling):
    """Four tensors of one layer, part of the head, every type, layout and scaling; the
    positions given and implied."""
    dt, rot, B, N = TYPES[dtype], 32, 2, 37
    xs = [randn(s, dt, i) for i, s in enumerate([(B, N, 4, 128), (B, N, 2, 128), (B, N, 2, 32), (B, N, 32)])]
    r = ops.new_rope(rot, interleaved=inter, scaling=SCALINGS[scaling])
    freq, m = frequencies(rot, SCALINGS[scaling])
    pos = torch.randint(0, 1 << 20, (B, N), generator=torch.Generator().manual_seed(9))
    for p in (None, pos.to(torch.int32).cuda(), pos.cuda()):
        for back in (False, True):
            ys = ops.msa_rope(xs, r, p, inverse=back)
            at = pos.numpy() if p is not None else np.tile(np.arange(N), (B, 1))
            for x, y in zip(xs, ys):
                h = f64(x) if x.dim() == 4 else f64(x)[:, :, None]
                want, size = reference(h, at.astype(np.float64), freq, m, rot, inter, back)
                assert y.is_contiguous() and y.dtype == dt
                check(y, want.reshape(x.shape), size.reshape(x.shape), dt)
    assert ops.device_status() == 0


@pytest.mark.parametrize("rot,d", [(2, 2), (2, 64), (6, 7), (10, 33), (64, 64), (96, 128), (128, 200),
                                   (512, 512)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T", [1, 13])
def test_odd_head_sizes(rot, d, inter, T):
    """Heads whose pairs, tails and rows do not fill 16-byte vectors, and those that do."""
    x = randn((T, 3, d), torch.bfloat16, rot + d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 97
    (y,) = ops.msa_rope(x, ops.new_rope(rot, interleaved=inter), pos)
    freq, m = frequencies(rot, None)
    want, size = reference(f64(x), pos.cpu().numpy().astype(np.float64), freq, m, rot, inter)
    check(y, want, size, torch.bfloat16)
    assert torch.equal(y[..., rot:], x[..., rot:])


def test_far_positions_are_as_exact_as_near_ones():
    """Angles up to position 2^31 - 1 (and negative ones) against exact rational arithmetic."""
    rot = 8
    two_pi = fractions.Fraction(2 * 31415926535897932384626433832795028841971693993751, 10 ** 49)
    f = [1.0, 0.1, 0.7390851332151607, 6.5]  # one above a turn a position
    at = [0, 1, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 31 - 1, -1, -(2 ** 31)]
    x = torch.zeros(len(at), 1, rot, device="cuda")
    x[..., :4] = 1.0
    (y,) = ops.msa_rope(x, ops.new_rope(rot, inv_freq=f), torch.tensor(at, dtype=torch.int32, device="cuda"))
    y = f64(y)[:, 0]
    for n, p in enumerate(at):
        for i, w in enumerate(f):
            turn = float((fractions.Fraction(p) * fractions.Fraction(w) / two_pi) % 1)
            assert abs(y[n, i] - math.cos(2 * math.pi * turn)) <= 1e-6
            assert abs(y[n, i + 4] - math.sin(2 * math.pi * turn)) <= 1e-6
    # int64 positions past 32 bits: the same fraction of a turn, still exact
    far = 2 ** 40 + 12345
    (y,) = ops.msa_rope(x[:1], ops.new_rope(rot, inv_freq=f), torch.tensor([far], device="cuda"))
    for i, w in enumerate(f):
        # turns are rounded to 2^-64, so 2^40 positions move the angle by at most 2^-24 turns
        turn = float((fractions.Fraction(far) * fractions.Fraction(w) / two_pi) % 1)
        assert abs(f64(y)[0, 0, i] - math.cos(2 * math.pi * turn)) <= 1e-6 + 2 * math.pi * 2.0 ** -24


@pytest.mark.parametrize("inter", [False, True])
def test_strided_views_and_in_place(inter):
    """Views of one fused projection (token and head strides, an odd offset too), an expanded
    tensor, a transposed head axis; in place changes the views' values and nothing else."""
    N, H, d, rot = 21, 3, 64, 32
    r = ops.new_rope(rot, interleaved=inter)
    freq, m = frequencies(rot, None)
    pos = torch.randperm(N, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    at = pos.cpu().numpy().astype(np.float64)
    for pad in (0, 8, 3):
        flat = randn((N, H * d + d + pad), torch.bfloat16, 3)
        q, k = flat[:, pad:pad + H * d].unflatten(-1, (H, d)), flat[:, pad + H * d:]
        want = [reference(f64(q), at, freq, m, rot, inter), reference(f64(k)[:, None], at, freq, m, rot, inter)]
        for y, w in zip(ops.msa_rope((q, k), r, pos), want):
            check(y, w[0].reshape(y.shape), w[1].reshape(y.shape), torch.bfloat16)
        before = flat.clone()
        out = ops.msa_rope((q, k), r, pos, inplace=True)
        assert out[0] is q and out[1] is k
        for y, w in zip(out, want):
            check(y, w[0].reshape(y.shape), w[1].reshape(y.shape), torch.bfloat16)
        assert torch.equal(flat[:, :pad], before[:, :pad])
    wide = randn((N, 1, d), torch.bfloat16, 4).expand(N, H, d)
    swapped = randn((H, N, d), torch.bfloat16, 5).transpose(0, 1)
    cols = randn((N, d, H), torch.bfloat16, 6).transpose(1, 2)  # last axis strided: copied
    for x in (wide, swapped, cols):
        (y,) = ops.msa_rope(x, r, pos)
        w = reference(f64(x), at, freq, m, rot, inter)
        check(y, w[0], w[1], torch.bfloat16)
    with pytest.raises(ValueError):
        ops.msa_rope(wide, r, pos, inplace=True)
    with pytest.raises(ValueError):
        ops.msa_rope(cols, r, pos, inplace=True)


def test_gradients():
    """Gradients of ops.rope: the formula's, against differences, of broadcast inputs, of
    outputs that are not used, and twice."""
    B, N, rot, d = 2, 5, 16, 24
    r = ops.new_rope(rot, interleaved=True, scaling=SCALINGS["yarn"])
    freq, m = frequencies(rot, SCALINGS["yarn"])
    pos = torch.randint(0, 5000, (B, N), generator=torch.Generator().manual_seed(2)).cuda()
    at = pos.cpu().numpy().astype(np.float64)
    q, k = (randn((B, N, h, d), torch.float32, 7 + h).requires_grad_() for h in (3, 1))
    dq, dk = randn(q.shape, torch.float32, 20), randn(k.shape, torch.float32, 21)
    yq, yk = ops.rope((q, k), r, pos)
    gq, gk = torch.autograd.grad((yq, yk), (q, k), (dq, dk), retain_graph=True)
    for g, dy in ((gq, dq), (gk, dk)):
        want, size = reference(f64(dy), at, freq, m, rot, True, back=True)
        check(g, want, size, torch.float32)
    # differences: the operator is linear, so a step of 1 has no error of its own
    for b, n, h, e in ((0, 0, 0, 0), (1, 4, 2, 15), (0, 3, 1, 20)):
        q1, q0 = q.detach().clone(), q.detach().clone()
        q1[b, n, h, e] += 0.5
        q0[b, n, h, e] -= 0.5
        y1, y0 = ops.msa_rope(q1, r, pos)[0], ops.msa_rope(q0, r, pos)[0]
        diff = float(((y1 - y0).double() * dq.double()).sum())
        # each of the two y's is off by at most 1e-6 (|x1| + |x2|) and half a step: < 1e-5 a value
        assert abs(diff - float(gq[b, n, h, e])) <= 2 * 2 * 1e-5 * float(dq[b, n, h].abs().max())
    # implied positions, and an input that needs no gradient
    yq, yk = ops.rope((q, k.detach()), r)
    (g,) = torch.autograd.grad(yq, q, dq)
    want, size = reference(f64(dq), np.tile(np.arange(N, dtype=np.float64), (B, 1)), freq, m, rot, True, back=True)
    check(g, want, size, torch.float32)
    assert not yk.requires_grad or torch.autograd.grad(ops.rope((q, k.detach()), r)[1].sum(), q,
                                                       allow_unused=True) == (None,)
    yq, yk = ops.rope((q, k), r, pos)
    # only one output used; the gradient of a sum arrives as a broadcast scalar
    (only,) = torch.autograd.grad(yq.sum(), q, retain_graph=True)
    want, size = reference(np.ones(q.shape), at, freq, m, rot, True, back=True)
    check(only, want, size, torch.float32)
    assert torch.autograd.grad(yq.sum(), k, retain_graph=True, allow_unused=True) == (None,)
    # an input shared by all heads: its gradient sums over them
    one = randn((B, N, 1, d), torch.float32, 30).requires_grad_()
    (y,) = ops.rope(one.expand(B, N, 4, d), r, pos)
    dy = randn(y.shape, torch.float32, 31)
    (g,) = torch.autograd.grad(y, one, dy)
    want, size = reference(f64(dy), at, freq, m, rot, True, back=True)
    assert np.abs(f64(g) - want.sum(2, keepdims=True)).max() <= 4 * (1e-6 + 2.0 ** -23) * size.max() * 2
    # the gradient is itself differentiable: turning there and back scales by m^2
    (y,) = ops.rope(q, r, pos)
    v = dq.clone().requires_grad_()
    (g,) = torch.autograd.grad(y, q, v, create_graph=True)
    (gg,) = torch.autograd.grad(g, v, dq)
    want, size = reference(f64(dq), at, freq, m, rot, True)
    check(gg, want, size, torch.float32)


def test_attention_takes_the_rope():
    """ops.attention with a rope is the attention of the rotated operands, gradients included."""
    B, N, H_q, H_kv, d, di = 1, 300, 4, 2, 64, 32
    make = lambda: [randn(s, torch.bfloat16, 40 + i).requires_grad_()  # noqa: E731
                    for i, s in enumerate([(B, N, H_q, d), (B, N, H_kv, d), (B, N, H_kv, d),
                                           (B, N, H_kv, di), (B, N, di)])]
    r = ops.new_rope(32)
    pos = (torch.arange(N, device="cuda") + 1000)[None]
    a, b = make(), make()
    o1 = ops.attention(*a, topk=2, rope=r, positions=pos)
    q, k, qi, ki = ops.rope((b[0], b[1], b[3], b[4]), r, pos)
    o2 = ops.attention(q, k, b[2], qi, ki, topk=2)
    assert torch.equal(o1, o2)
    dO = randn(o1.shape, torch.bfloat16, 50)
    o1.backward(dO)
    o2.backward(dO)
    for x, y in zip(a, b):
        # the attention's backward may order its sums differently from run to run
        assert (x.grad.float() - y.grad.float()).abs().max() <= 1e-2 * y.grad.float().abs().max()
    with pytest.raises(ValueError):
        ops.attention(*a, topk=2, positions=pos)


def test_streams_graphs_and_empty_calls():
    """A side stream, a captured forward and backward replayed on new values, and calls without
    tokens.  (PyTorch itself refuses to capture a backward while an eager graph of the same
    leaf lives, whatever the operator: the leaf's accumulation belongs to the eager stream.)"""
    x = randn((64, 4, 64), torch.bfloat16, 60).requires_grad_()
    pos = torch.arange(64, device="cuda")
    r = ops.new_rope(64)
    dy = randn(x.shape, torch.bfloat16, 61)
    (alive,) = ops.rope(x, r, pos)
    (want,) = torch.autograd.grad(alive, x, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        (y,) = ops.rope(x, r, pos)
        (g,) = torch.autograd.grad(y, x, dy)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, alive) and torch.equal(g, want)
    del alive, y  # and with them the eager graphs of x
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (y,) = ops.rope(x, r, pos)
        (g,) = torch.autograd.grad(y, x, dy)
    with torch.no_grad():
        pos += 5
        dy.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ops.msa_rope(x.detach(), r, pos)[0])
    assert torch.equal(g, ops.msa_rope(dy, r, pos, inverse=True)[0])
    for shape, p in (((0, 4, 64), pos[:0]), ((3, 0, 4, 64), None), ((0, 7, 4, 64), None)):
        (e,) = ops.msa_rope(torch.empty(shape, device="cuda"), r, p)
        assert tuple(e.shape) == shape
    assert ops.device_status() == 0


def test_refusals():
    x = randn((4, 2, 64), torch.bfloat16, 70)
    pos = torch.arange(4, device="cuda")
    r = ops.new_rope(64)
    bad = [
        (dict(xs=x.cpu(), rope=r, positions=pos), ValueError),
        (dict(xs=x, rope=ops.new_rope(64, device="cpu"), positions=pos), ValueError),
        (dict(xs=x, rope=r, positions=pos.float()), TypeError),
        (dict(xs=x, rope=r, positions=pos[:3]), ValueError),
        (dict(xs=x, rope=r, positions=pos.view(1, 1, 4)), ValueError),
        (dict(xs=x, rope=r, positions=pos.cpu()), ValueError),
        (dict(xs=(x, x.float()), rope=r, positions=pos), TypeError),
        (dict(xs=x.double(), rope=r, positions=pos), TypeError),
        (dict(xs=x[..., :32], rope=r, positions=pos), ValueError),
        (dict(xs=(x,) * 5, rope=r, positions=pos), ValueError),
        (dict(xs=(), rope=r, positions=pos), ValueError),
        (dict(xs=x, rope=None, positions=pos), TypeError),
        (dict(xs=x[0], rope=r), ValueError),
    ]
    for kw, err in bad:
        with pytest.raises(err):
            ops.msa_rope(**kw)
    y = x.clone().requires_grad_()
    with pytest.raises(ValueError):
        ops.msa_rope(y, r, pos, inplace=True)
    huge = torch.empty((1, 2000, 64), device="cuda", dtype=torch.bfloat16)
    from block_sparse_gqa_topk_gb300 import _lib
    with pytest.raises(_lib.MSAError):  # more heads than the kernel's index arithmetic serves
        ops.msa_rope(huge, r, pos[:1])
