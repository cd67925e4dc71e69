"""ops.msa_cache_append against what it joins: msa_rope and msa_cache_write on the same inputs, bit for
bit (outputs and every byte of the pool); and against the formula in 64 bits."""
import itertools

import numpy as np
import pytest
import torch

from block_sparse_gqa_topk_gb300 import _lib, ops
from test_gpu_cache import dev, randn, table_for

pytestmark = pytest.mark.gpu

KINDS = ({}, {"fp8": True}, {"fp4": True})


def marked(pages, H, page, d, di, kind):
    c = ops.new_paged_cache(pages, H, page_size=page, d=d, d_idx=di, **kind)
    for i, t in enumerate(c._pools):
        t.view(torch.uint8).fill_(0x30 + i)
    return c


def same_pools(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a._pools, b._pools))


def inputs(T, H_q, H, Hi, d, di, seed, fused=0):
    """q, k, v, q_idx, k_idx; fused: columns of one tensor, from column `fused` - 1 on."""
    rows = [(H_q, d), (H, d), (H, d)] + ([(Hi, di), (1, di)] if di else [])
    widths = [h * w for h, w in rows]
    if fused:
        flat = randn((T, sum(widths) + fused - 1), seed)[:, fused - 1:]
        xs = [x.unflatten(-1, r) for x, r in zip(torch.split(flat, widths, -1), rows)]
    else:
        xs = [randn((T, *r), seed + i) for i, r in enumerate(rows)]
    return xs[:4] + [xs[4].squeeze(-2)] if di else xs + [None, None]


def places(t, lens, new, page):
    """Position and pool row of every packed token."""
    out = []
    for b, (n, m) in enumerate(zip(lens, new)):
        out += [(p, int(t[b, p // page]) * page + p % page) for p in range(n - m, n)]
    return out


CASES = [  # page, H_q, H_kv, index heads, d, d_idx, rot, lens, new
    (16, 1, 1, 1, 64, 32, 32, [1], [1]),
    (16, 6, 2, 2, 64, 0, 64, [40, 17, 16, 1], [40, 1, 16, 1]),
    (48, 12, 3, 3, 128, 64, 64, [130, 48, 1, 97], [33, 48, 0, 2]),
    (128, 32, 8, 8, 128, 64, 16, [700, 1, 128, 129, 0], [300, 1, 1, 129, 0]),
    (256, 5, 5, 1, 128, 32, 2, [513], [257]),
    (16, 4, 2, 2, 128, 64, 34, [70, 33], [65, 33]),
    (16, 16, 1, 3, 64, 64, 48, [200, 3, 90], [7, 3, 1]),
    (64, 2, 2, 0, 128, 0, 126, [50], [50]),
    (64, 2, 1, 0, 128, 0, 128, [50], [49]),
    (128, 16, 4, 4, 128, 64, 64, [3000, 2500], [3000, 1300]),
]


@pytest.mark.parametrize("kind", range(3))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_is_rope_then_write(case, inter, kind):
    page, H_q, H, Hi, d, di, rot, lens, new = CASES[case]
    pages = sum((n + page - 1) // page for n in lens) + 2
    t = table_for(lens, page, pages, case)
    cu, T = dev(np.concatenate([[0], np.cumsum(new)])), sum(new)
    rope = ops.new_rope(rot, interleaved=inter, scaling={"type": "yarn", "factor": 4, "original_len": 64})
    own = torch.tensor([p for p, _ in places(t, lens, new, page)], device="cuda")
    far = torch.randint(-2 ** 40, 2 ** 40, (T,), generator=torch.Generator().manual_seed(case)).cuda()
    for fused, pos in itertools.product((0, 1, 4) if case % 2 else (0, 9), (None, own.int(), far)):
        q, k, v, qi, ki = inputs(T, H_q, H, Hi, d, di, 10 * case, fused)
        if T > 2:
            k = k.clone() if not fused else k
            k[1], k[2, 0] = 0, k[2, 0] * 2.0 ** -60
        a, b = (marked(pages, H, page, d, di, KINDS[kind]) for _ in "ab")
        y, yi = ops.msa_cache_append(a, dev(t), dev(lens), rope, q, k, v, qi, ki, positions=pos, cu_seqlens=cu)
        assert ops.device_status() == 0
        turned = ops.msa_rope([x for x in (q, k, qi, ki) if x is not None], rope, own if pos is None else pos)
        ops.msa_cache_write(b, dev(t), dev(lens), turned[1], v, turned[3] if di else None, cu_seqlens=cu)
        assert torch.equal(y, turned[0]) and (torch.equal(yi, turned[2]) if di else yi is None)
        assert y.is_contiguous() and same_pools(a, b), (fused, pos)


@pytest.mark.parametrize("kind", range(3))
def test_a_decode_step(kind):
    """One token a sequence, without cu_seqlens: empty slots get zero queries and no row."""
    page, H_q, H, d, di, rot, lens = 16, 8, 2, 128, 64, 64, [1, 0, 17, 40, 0, 16]
    t = table_for([40] * 6, page, 18, 3)
    a, b = (marked(18, H, page, d, di, KINDS[kind]) for _ in "ab")
    rope = ops.new_rope(rot)
    q, k, v, qi, ki = inputs(6, H_q, H, 2, d, di, 5)
    y, yi = ops.msa_cache_append(a, dev(t), dev(lens), rope, q, k, v, qi, ki)
    pos = torch.tensor(lens, device="cuda").clamp(min=1) - 1
    tq, tk, ti, tki = ops.msa_rope((q, k, qi, ki), rope, pos)
    ops.msa_cache_write(b, dev(t), dev(lens), tk, v, tki)
    live = torch.tensor(lens, device="cuda") > 0
    assert torch.equal(y[live], tq[live]) and torch.equal(yi[live], ti[live])
    assert not y[~live].any() and not yi[~live].any()
    assert same_pools(a, b) and ops.device_status() == 0


def test_against_the_formula():
    """bf16 cache: y1 = m (x1 cos a - x2 sin a) in 64 bits.  The angle's fraction of a turn is rounded to
    float (2^-24 of at most half a turn: pi 2^-24 radians), sine and cosine are good to 2 units of 2^-24
    and each of the products and the sum to one: 8 2^-24 (|x1| + |x2|) m in all, then half a bf16 step."""
    T, H, d, rot, m = 300, 2, 128, 64, 1.25
    rope = ops.new_rope(rot, mscale=m)
    c = ops.new_paged_cache(4, H, page_size=128, d=d, d_idx=64)
    q, k, v, qi, ki = inputs(T, 4, H, 2, d, 64, 1)
    pos = torch.randint(0, 1 << 20, (T,), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    y, yi = ops.msa_cache_append(c, dev([[2, 0, 3]]), dev([T]), rope, q, k, v, qi, ki, positions=pos,
                                 cu_seqlens=dev([0, T]))
    rows = torch.tensor([[2, 0, 3][p // 128] * 128 + p % 128 for p in range(T)], device="cuda")
    angle = pos.double()[:, None] * 10000.0 ** (-torch.arange(rot // 2, device="cuda").double() * 2 / rot)
    for x, got in ((q, y), (k, c.k.flatten(0, 1)[rows]), (qi, yi), (ki[:, None], c.k_idx.flatten(0, 1)[rows][:, None])):
        x1, x2 = x[..., :rot // 2].double(), x[..., rot // 2:rot].double()
        cos, sin = angle.cos()[:, None] * m, angle.sin()[:, None] * m
        want = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin, x[..., rot:].double()], -1)
        slack = 8 * 2.0 ** -24 * m * (x1.abs() + x2.abs())
        slack = torch.cat([slack, slack, torch.zeros_like(x[..., rot:].double())], -1)
        assert ((got.double() - want).abs() <= slack + 2.0 ** -8 * (want.abs() + slack)).all()
    assert torch.equal(c.v.flatten(0, 1)[rows], v) and ops.device_status() == 0


@pytest.mark.parametrize("kind", range(3))
def test_tokens_without_a_place(kind):
    """Page ids outside the pool, a length past the table, a negative one, more new tokens than length and
    a broken cu_seqlens: those tokens are dropped with zero queries, the status says so, the others
    are as they should be; rows behind the last sequence are zero and no error."""
    page, H, d, di = 16, 2, 64, 32
    rope = ops.new_rope(32)
    lens, new, t = [20, 17], [20, 17], np.array([[0, 1], [2, 3]], dtype=np.int32)
    q, k, v, qi, ki = inputs(40, 4, H, 2, d, di, 7)
    good = marked(4, H, page, d, di, KINDS[kind])
    y0, yi0 = ops.msa_cache_append(good, dev(t), dev(lens), rope, q, k, v, qi, ki, cu_seqlens=dev([0, 20, 37]))
    assert ops.device_status() == 0 and not y0[37:].any() and not yi0[37:].any() and y0[36].any()
    for table, ls, cu, lost in [
            ([[0, 9], [2, 3]], lens, [0, 20, 37], range(16, 20)), ([[0, -1], [2, 3]], lens, [0, 20, 37], range(16, 20)),
            (t, [20, 33], [0, 20, 37], range(20, 37)), (t, [-3, 17], [0, 20, 37], range(20)),
            (t, [12, 17], [0, 20, 37], range(8)), (t, [20, 2 ** 31 - 1], [0, 20, 37], range(20, 37)),
            (t, lens, [0, 20, 10], range(20, 40))]:
        c = marked(4, H, page, d, di, KINDS[kind])
        y, yi = ops.msa_cache_append(c, dev(table), dev(ls), rope, q, k, v, qi, ki, cu_seqlens=dev(cu))
        assert ops.device_status() == _lib.MSA_ERR_ARG
        assert not y[list(lost)].any() and not yi[list(lost)].any()
        kept = [i for i in range(20 if lost[0] >= 20 else 37) if i not in lost and (lost[0] < 20 or i < 20)]
        if ls != [12, 17]:
            assert torch.equal(y[kept], y0[kept]) and torch.equal(yi[kept], yi0[kept])
            if kept[-1] == 36:
                assert all(torch.equal(x[2:].view(torch.uint8), z[2:].view(torch.uint8))
                           for x, z in zip(c._pools, good._pools))


def test_captured_step_then_decode():
    """The serving step of a layer, captured: append, then attention over what it appended.  Prompts and
    tokens through msa_rope and msa_cache_write give the same bytes, and the same attention."""
    H_q, H, d, di, page, prompts = 8, 2, 128, 64, 16, [200, 1, 77]
    rope = ops.new_rope(64)
    for kind in KINDS:
        t = dev(table_for([240] * 3, page, 48, 2))
        a, b = (marked(48, H, page, d, di, kind) for _ in "ab")
        T, cu = sum(prompts), dev(np.concatenate([[0], np.cumsum(prompts)]))
        x = inputs(T, H_q, H, H, d, di, 3)
        ops.msa_cache_append(a, t, dev(prompts), rope, *x, cu_seqlens=cu)
        pos = torch.cat([torch.arange(n, device="cuda") for n in prompts])
        tq, tk, ti, tki = ops.msa_rope((x[0], x[1], x[3], x[4]), rope, pos)
        ops.msa_cache_write(b, t, dev(prompts), tk, x[2], tki, cu_seqlens=cu)
        lens = dev(prompts)
        new = inputs(3, H_q, H, H, d, di, 4)

        def step():
            y, yi = ops.msa_cache_append(a, t, lens, rope, *new)
            return y, yi, *ops.msa_decode_paged(y, yi, a, t, lens, 2), *ops.msa_decode_paged_dense(y, a, t, lens)

        def parts():
            tq, tk, ti, tki = ops.msa_rope((new[0], new[1], new[3], new[4]), rope, lens - 1)
            ops.msa_cache_write(b, t, lens, tk, new[2], tki)
            return tq, ti, *ops.msa_decode_paged(tq, ti, b, t, lens, 2), *ops.msa_decode_paged_dense(tq, b, t, lens)

        # both write over the prompts' last tokens, before the capture
        assert all(torch.equal(w, z) for w, z in zip(step(), parts())), kind
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for n in range(1, 20):
            lens += 1
            for w, z in zip(new, inputs(3, H_q, H, H, d, di, 100 + 10 * n)):
                w.copy_(z)
            graph.replay()
            assert all(torch.equal(w, z) for w, z in zip(out, parts())), (kind, n)
        assert same_pools(a, b)
        assert ops.device_status() == 0


def test_versions_streams_and_nothing_to_do():
    c = ops.new_paged_cache(4, 2, page_size=16, d=64, d_idx=32)
    rope, t = ops.new_rope(32), dev([[0, 1], [2, 3]])
    x = inputs(2, 4, 2, 2, 64, 32, 1)
    before = [p._version for p in c._pools]
    ops.msa_cache_append(c, t, dev([1, 1]), rope, *x)
    assert all(p._version > n for p, n in zip(c._pools, before))
    none = inputs(0, 4, 2, 2, 64, 32, 1)
    y, yi = ops.msa_cache_append(c, t, dev([1, 1]), rope, *none, cu_seqlens=dev([0, 0, 0]))
    assert y.shape == (0, 4, 64) and yi.shape == (0, 2, 32)
    y, yi = ops.msa_cache_append(c, t[:0], dev([]), rope, *x, cu_seqlens=dev([0]))
    assert not y.any() and not yi.any()
    want = ops.msa_cache_append(c, t, dev([3, 4]), rope, *x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ops.msa_cache_append(c, t, dev([3, 4]), rope, *x)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and ops.device_status() == 0


def test_refusals():
    c = ops.new_paged_cache(4, 2, page_size=16, d=64, d_idx=32)
    rope, t, lens = ops.new_rope(32), dev([[0, 1], [2, 3]]), dev([1, 2])
    x = inputs(2, 4, 2, 2, 64, 32, 1)

    def call(i=None, bad=None, cache=c, rope=rope, t=t, lens=lens, **kw):
        xs = [bad if j == i else z for j, z in enumerate(x)]
        return ops.msa_cache_append(cache, t, lens, rope, *xs, **kw)

    call()
    for i in range(5):
        for bad in (x[i].float(), x[i].cpu(), x[i][:1], x[i][..., :16], x[i].transpose(0, -1), None):
            with pytest.raises((TypeError, ValueError)):
                call(i, bad)
    for kw in (dict(rope=32), dict(rope=ops.new_rope(64)), dict(rope=ops.new_rope(32, device="cpu")), dict(cache=None),
               dict(lens=dev([1])), dict(lens=dev([1, 2]).long()), dict(t=t.long()), dict(t=t.cpu()),
               dict(positions=dev([1])), dict(positions=torch.zeros(2, device="cuda")),
               dict(positions=torch.zeros(2, dtype=torch.int32)), dict(positions=torch.zeros(2, 1, dtype=torch.int32).cuda()),
               dict(cu_seqlens=dev([0, 2])), dict(cu_seqlens=[0, 1, 2]), dict(t=t[:1], lens=dev([1]))):
        with pytest.raises((TypeError, ValueError)):
            call(**kw)
    plain = ops.new_paged_cache(4, 2, page_size=16, d=64, d_idx=0)
    with pytest.raises(ValueError):
        call(cache=plain)
    assert ops.msa_cache_append(plain, t, lens, ops.new_rope(64), *x[:3])[1] is None
    assert ops.device_status() == 0


@pytest.mark.parametrize("kind", range(3))
def test_a_pool_without_pages(kind):
    """No id is one of the pool's: tokens are dropped with zero queries, the status says so; an empty slot is none."""
    c = ops.new_paged_cache(0, 2, page_size=16, d=64, d_idx=32, **KINDS[kind])
    q, k, v, qi, ki = inputs(2, 4, 2, 2, 64, 32, 11)
    table, rope = dev([[0, 0], [0, 0]]), ops.new_rope(32)
    y, yi = ops.msa_cache_append(c, table, dev([20, 0]), rope, q, k, v, qi, ki)
    assert ops.device_status() == _lib.MSA_ERR_ARG and not y.any() and not yi.any()
    y, yi = ops.msa_cache_append(c, table, dev([0, 0]), rope, q, k, v, qi, ki)
    assert ops.device_status() == 0 and not y.any() and not yi.any()
