"""Host-side checks of the rotary and paged-cache calls (no GPU): frequencies against their
formulas, and every refusal that the C ABI makes before it touches the device."""
import fractions
import math

import pytest

from block_sparse_gqa_topk_gb300 import _lib, ops

OK, ARG, SHAPE, UNSUP, WS = (_lib.MSA_OK, _lib.MSA_ERR_ARG, _lib.MSA_ERR_SHAPE, _lib.MSA_ERR_UNSUPPORTED,
                             _lib.MSA_ERR_WORKSPACE)


def test_frequencies():
    f, m = ops.rope_frequencies(64)
    assert m == 1.0 and len(f) == 32 and f[0] == 1.0
    assert math.isclose(f[31], 10000.0 ** (-62 / 64), rel_tol=1e-15)
    g, m = ops.rope_frequencies(64, scaling={"type": "linear", "factor": 4})
    assert m == 1.0 and all(math.isclose(4 * b, a, rel_tol=1e-15) for a, b in zip(f, g))
    g, m = ops.rope_frequencies(64, scaling={"type": "ntk", "factor": 4})
    assert m == 1.0 and g[0] == 1.0  # the fastest pair stays, the slowest is divided by the factor
    assert math.isclose(g[31], f[31] / 4, rel_tol=1e-12)
    g, m = ops.rope_frequencies(64, scaling={"type": "yarn", "factor": 4, "original_len": 32768})
    assert math.isclose(m, 1 + 0.1 * math.log(4))
    for a, b in zip(f, g):
        turns = 32768 * a / (2 * math.pi)
        lo, hi = a / 4, a
        assert b == hi if turns >= 32 else math.isclose(b, lo) if turns <= 1 else lo < b < hi
    _, m = ops.rope_frequencies(64, scaling={"type": "yarn", "factor": 4, "original_len": 8, "mscale": 1.5})
    assert m == 1.5


def test_turns_are_the_exact_fractions():
    two_pi = fractions.Fraction(2 * 31415926535897932384626433832795028841971693993751, 10 ** 49)
    f = [1.0, 0.5, 1e-4, 7.0, -0.25, 0.0]
    r = ops.new_rope(12, inv_freq=f, device="cpu")
    for x, t in zip(f, r.turns.tolist()):
        exact = fractions.Fraction(x) / two_pi % 1 * 2 ** 64
        assert abs((t % 2 ** 64) - exact) <= fractions.Fraction(1, 2)


@pytest.mark.parametrize("args,kw", [
    ((0,), {}), ((63,), {}), ((514,), {}), ((64,), dict(base=0.0)), ((64,), dict(base=float("nan"))),
    ((64,), dict(scaling={"type": "other", "factor": 2})), ((64,), dict(scaling={"type": "linear"})),
    ((64,), dict(scaling={"type": "linear", "factor": 0})),
    ((64,), dict(scaling={"type": "linear", "factor": 2, "beta_fast": 3})),
    ((2,), dict(scaling={"type": "ntk", "factor": 2})),
    ((64,), dict(scaling={"type": "yarn", "factor": 2})),
    ((64,), dict(scaling={"type": "yarn", "factor": 2, "original_len": 8, "beta_fast": 1})),
    ((64,), dict(inv_freq=[1.0])), ((4,), dict(inv_freq=[1.0, float("inf")])),
    ((4,), dict(inv_freq=[1.0, 0.5], scaling={"type": "linear", "factor": 2})),
    ((64,), dict(mscale=float("nan"))),
])
def test_new_rope_refuses(args, kw):
    with pytest.raises(ValueError):
        ops.new_rope(*args, device="cpu", **kw)


def rope(B=1, N=4, rot=64, inter=0, inverse=0, dtype=0, bits=32, m=1.0):
    return _lib.ROPE.pack(B, N, rot, inter, inverse, dtype, bits, m, 0, 1)


def tensor(x=256, y=512, H=2, d=64):
    return _lib.ROPE_TENSOR.pack(x, y, 0, H * d, d, 0, H * d, d, H, d)


def test_rope_checks_its_arguments():
    call = lambda r=rope(), turns=256, pos=None, t=tensor(), n=1: _lib.msa_rope(r, turns, pos, t, n, None)  # noqa: E731
    assert call(r=None) == ARG and call(t=None) == ARG
    assert call(n=0) == ARG and call(n=5, t=tensor() * 5) == ARG
    for r, code in [(rope(B=-1), SHAPE), (rope(N=-1), SHAPE), (rope(rot=0), SHAPE), (rope(rot=63), SHAPE),
                    (rope(rot=1024), UNSUP), (rope(m=float("inf")), ARG), (rope(dtype=3), ARG),
                    (rope(bits=16), ARG), (rope(N=0), OK), (rope(B=0), OK)]:
        assert call(r=r, t=tensor(d=512)) == code, (r, code)
    assert call(t=tensor(d=32)) == SHAPE and call(t=tensor(H=0)) == SHAPE
    assert call(t=tensor(d=514)) == UNSUP and call(t=tensor(H=1025)) == UNSUP
    assert call(t=tensor(x=0)) == ARG and call(t=tensor(y=0)) == ARG and call(t=tensor(x=257)) == ARG
    assert call(turns=None) == ARG and call(turns=260) == ARG and call(pos=258) == ARG
    assert call(r=rope(bits=64), pos=260) == ARG
    assert call(t=tensor() + tensor(x=0), n=2) == ARG


def cache(P=4, page=16, H=2, d=64, di=32, kind=0, k=256, v=256, ki=256, ks=0, vs=0):
    return _lib.PAGED_CACHE.pack(P, page, H, d, di, kind, k, v, ki, ks, vs)


def table(ids=256, B=1, n=2, stride=2):
    return _lib.PAGE_TABLE.pack(ids, B, n, stride)


def test_cache_calls_check_their_arguments():
    def write(c=cache(), t=table(), lens=256, cu=None, T=1, k=256, v=256, ki=256, s=None):
        return _lib.msa_cache_write(c, t, lens, cu, T, k, v, ki, s, None)

    def read(c=cache(), t=table(), lens=256, cu=256, T=1, k=256, v=256, ki=256):
        return _lib.msa_cache_read(c, t, lens, cu, T, k, v, ki, None)

    for f in (write, read):
        for c, code in [(None, ARG), (cache(P=-1), SHAPE), (cache(page=0), SHAPE), (cache(H=0), SHAPE),
                        (cache(kind=2), ARG), (cache(page=24), UNSUP), (cache(d=96), UNSUP),
                        (cache(di=16), UNSUP), (cache(k=0), ARG), (cache(v=264), ARG), (cache(ki=0), ARG),
                        (cache(kind=1), ARG), (cache(kind=1, ks=256), ARG), (cache(di=0), SHAPE)]:
            assert f(c=c) == code, (f, c)
        assert f(t=None) == ARG and f(t=table(B=-1)) == SHAPE and f(t=table(ids=0)) == ARG
        assert f(t=table(ids=258)) == ARG and f(t=table(n=1 << 28)) == UNSUP and f(t=table(stride=-1)) == SHAPE
        assert f(T=-1) == SHAPE
        assert f(lens=None) == ARG and f(lens=258) == ARG and f(k=None) == ARG and f(v=264) == ARG
        assert f(ki=264) == ARG
        assert f(T=0, cu=256) == OK and f(t=table(B=0), T=0) == OK
    assert write(T=2) == SHAPE  # no cu_seqlens: one token a sequence
    assert write(cu=258) == ARG
    assert write(s=_lib.CACHE_STRIDES.pack(128, 64, 128, 60, 32)) == ARG
    assert read(cu=None) == ARG


def test_decode_calls_check_their_arguments():
    size = _lib.msa_decode_paged_workspace_size
    long = table(n=1024)
    need = size(cache(), long, 4, 4)  # the pooled scores grow with the table's length
    assert 0 < need < size(cache(), table(n=1 << 20), 4, 4) and size(cache(), long, 4, 0) > 0
    # short tables need none: up to 8 units (128 tokens, 64 with bf16 and d 128) a CTA of a
    # cluster of at most 8 (3 CTAs a SM hold all pairs' clusters at once; 16 units if one CTA is
    # a cluster and all tokens are read) and, sparse, 32 blocks
    for kw, tokens, groups in [(dict(), 8192, 1), (dict(d=128), 4096, 1), (dict(d=128, kind=1), 8192, 1),
                               (dict(H=57), 8192, 1), (dict(H=58), 4096, 1), (dict(H=115), 2048, 1),
                               (dict(H=229), 2048, 1), (dict(H=1000), 2048, 1), (dict(H=39, d=128), 4096, 8),
                               (dict(H=39, d=128), 2048, 16)]:
        H_q = groups * kw.get("H", 2)
        assert size(cache(**kw), table(n=tokens // 16), H_q, 0) == 0, kw
        assert size(cache(**kw), table(n=tokens // 16 + 1), H_q, 0) > 0, kw
    assert size(cache(), table(n=256), 4, 32) == 0 and size(cache(), table(n=257), 4, 1) > 0
    assert size(cache(H=300), table(n=256), 300, 8) == 0 and size(cache(H=300), table(n=256), 300, 9) > 0
    big = 1 << 40

    def dense(c=cache(), t=long, lens=256, H_q=4, scale=1.0, q=256, o=256, lse=256, ws=256, n=big):
        return _lib.msa_decode_paged_dense(c, t, lens, H_q, scale, q, o, lse, ws, n, None)

    def sparse(c=cache(), t=long, lens=256, H_q=4, topk=4, scale=1.0, q=256, qi=256, bi=256, o=256, lse=256,
               ws=256, n=big):
        return _lib.msa_decode_paged(c, t, lens, H_q, topk, scale, q, qi, bi, o, lse, ws, n, None)

    for f in (dense, sparse):
        for kw, code in [(dict(c=None), ARG), (dict(t=None), ARG), (dict(c=cache(d=96)), UNSUP),
                         (dict(c=cache(page=8)), UNSUP), (dict(c=cache(k=0)), ARG), (dict(t=table(ids=0)), ARG),
                         (dict(t=table(B=-1)), SHAPE), (dict(t=table(B=65536)), UNSUP),
                         (dict(t=table(n=1 << 28)), UNSUP), (dict(H_q=3), SHAPE), (dict(H_q=0), SHAPE),
                         (dict(H_q=34), UNSUP), (dict(scale=0.0), ARG), (dict(scale=float("nan")), ARG),
                         (dict(q=None), ARG), (dict(o=264), ARG), (dict(lse=None), ARG), (dict(lens=None), ARG),
                         (dict(lens=258), ARG), (dict(ws=None), WS), (dict(n=255), WS), (dict(ws=128), ARG),
                         (dict(t=table(B=0)), OK)]:
            assert f(**kw) == code, (f, kw)
    for kw, code in [(dict(topk=0), SHAPE), (dict(topk=33), UNSUP), (dict(c=cache(di=0)), SHAPE),
                     (dict(qi=None), ARG), (dict(bi=264), ARG), (dict(n=need - 1), WS)]:
        assert sparse(**kw) == code, kw
    # the work of a call is counted in 32 bits
    assert dense(t=table(B=60000, n=1 << 20, stride=1 << 20), c=cache(H=4)) == UNSUP
    assert size(cache(), table(), 4, -1) == 0 and size(cache(), table(), 3, 0) == 0
    assert size(cache(di=0), table(), 4, 4) == 0 and size(cache(k=0), table(ids=0, n=1024), 4, 4) > 0
