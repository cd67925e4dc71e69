"""Host-side checks of msa_cache_append (no GPU)."""
import pytest

from block_sparse_gqa_topk_gb300 import _lib
from test_serving_args import ARG, OK, SHAPE, UNSUP, cache, table


def append(rot=32, inter=0, bits=32, m=1.0, H_q=4, H_i=2, ps=1, q=(256, 64), k=(128, 64), v=(128, 64), qi=(64, 32), ki=32):
    return _lib.APPEND.pack(rot, inter, bits, m, H_q, H_i, ps, *q, *k, *v, *qi, ki)


def call(c=cache(), t=table(), lens=256, cu=None, T=1, a=append(), turns=256, pos=None, q=256, k=256, v=256, qi=256,
         ki=256, y=512, yi=512):
    return _lib.msa_cache_append(c, t, lens, cu, T, a, turns, pos, q, k, v, qi, ki, y, yi, None)


@pytest.mark.parametrize("kind", [{}, {"kind": 1, "ks": 256, "vs": 256}, {"kind": 2, "ks": 256, "vs": 256}])
def test_arguments(kind):
    c = lambda **kw: cache(**kind, **kw)  # noqa: E731
    for kw, code in [(dict(c=None), ARG), (dict(c=c(page=24)), UNSUP), (dict(c=c(k=0)), ARG), (dict(t=None), ARG),
                     (dict(t=table(ids=0)), ARG), (dict(t=table(n=1 << 28)), UNSUP), (dict(a=None), ARG),
                     (dict(T=-1), SHAPE), (dict(T=2), SHAPE), (dict(a=append(rot=0)), SHAPE), (dict(a=append(rot=33)), SHAPE),
                     (dict(a=append(rot=34)), SHAPE), (dict(a=append(H_q=0)), SHAPE), (dict(a=append(H_i=0)), SHAPE),
                     (dict(a=append(H_q=1025)), UNSUP), (dict(a=append(H_i=1025)), UNSUP),
                     (dict(a=append(m=float("nan"))), ARG), (dict(a=append(bits=16)), ARG), (dict(lens=None), ARG),
                     (dict(lens=258), ARG), (dict(cu=258), ARG), (dict(turns=None), ARG), (dict(turns=260), ARG),
                     (dict(pos=258), ARG), (dict(pos=260, a=append(bits=64)), ARG), (dict(q=None), ARG), (dict(q=257), ARG),
                     (dict(k=None), ARG), (dict(k=264), ARG), (dict(v=264), ARG), (dict(qi=None), ARG), (dict(ki=None), ARG),
                     (dict(ki=264), ARG), (dict(y=None), ARG), (dict(y=520), ARG), (dict(yi=None), ARG),
                     (dict(a=append(k=(130, 64))), ARG), (dict(a=append(v=(128, 60))), ARG), (dict(a=append(ki=36)), ARG),
                     (dict(c=c(di=0)), SHAPE), (dict(c=c(di=0), a=append(rot=66), qi=None, ki=None, yi=None), SHAPE),
                     (dict(t=table(B=0), T=0), OK), (dict(t=table(B=0), T=3, cu=256), OK), (dict(T=0, cu=256), OK)]:
        assert call(**({"c": c()} | kw)) == code, kw
