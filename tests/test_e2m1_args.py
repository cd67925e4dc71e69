"""Host-side checks of the paged calls over a 4-bit cache (no GPU)."""
from block_sparse_gqa_topk_gb300 import _lib
from test_serving_args import ARG, OK, SHAPE, UNSUP, WS, cache, table


def cache4(**kw):
    return cache(**({"kind": _lib.MSA_CACHE_E2M1, "ks": 256, "vs": 256} | kw))


def test_cache_calls():
    def write(c=cache4(), t=table(), T=1, k=256, v=256, ki=256):
        return _lib.msa_cache_write(c, t, 256, None, T, k, v, ki, None, None)

    def read(c=cache4(), t=table(), T=1, k=256, v=256, ki=256):
        return _lib.msa_cache_read(c, t, 256, 256, T, k, v, ki, None)

    for f in (write, read):
        for c, code in [(cache4(ks=0), ARG), (cache4(vs=0), ARG), (cache4(ks=264), ARG), (cache4(kind=3), ARG),
                        (cache4(d=96), UNSUP), (cache4(page=24), UNSUP), (cache4(di=0), SHAPE)]:
            assert f(c=c) == code, c
        assert f(t=table(B=0), T=0) == OK and f(T=-1) == SHAPE


def test_decode_calls():
    size = _lib.msa_decode_paged_workspace_size
    for kw, tokens in [(dict(), 8192), (dict(d=128), 8192), (dict(H=58), 4096)]:  # as with E4M3
        H_q = kw.get("H", 2)
        assert size(cache4(**kw), table(n=tokens // 16), H_q, 0) == 0
        assert size(cache4(**kw), table(n=tokens // 16 + 1), H_q, 0) > 0
    long = table(n=1024)

    def dense(c=cache4(), H_q=4, ws=256, n=1 << 40):
        return _lib.msa_decode_paged_dense(c, long, 256, H_q, 1.0, 256, 256, 256, ws, n, None)

    for kw, code in [(dict(c=cache4(ks=0)), ARG), (dict(c=cache4(d=96)), UNSUP), (dict(H_q=34), UNSUP),
                     (dict(H_q=3), SHAPE), (dict(ws=None), WS), (dict(n=255), WS)]:
        assert dense(**kw) == code, kw
