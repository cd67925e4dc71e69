"""Rotary positions, the paged cache and paged decode as a server runs them together: prompts
are rotated and written, each next token is rotated, written and decoded, in a captured step
whose batch has an empty slot.  Every decoded row must equal the training path's row on the same
rotated sequence (msa_index_topk + msa_fwd, and the dense set for the dense form), and a chunk
read back from the pages must give the training path's forward on it."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_topk_gb300 import ops
from parity import LSE_TOL, O_TOL

pytestmark = pytest.mark.gpu

H_q, H_kv, D, DI, TOPK, ROT = 8, 2, 64, 32, 3, 32


def dev(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def sequences(lens, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [[torch.randn(n, *s, generator=g, device="cuda").bfloat16()
             for s in ((H_q, D), (H_kv, D), (H_kv, D), (H_kv, DI), (DI,))] for n in lens]


def training_rows(seq, rope, fp8):
    """o, lse and block sets of every position, sparse and over the whole context."""
    q, k, v, qi, ki = (x[None] for x in seq)
    q, k, qi, ki = ops.msa_rope((q, k, qi, ki), rope)
    if fp8:  # the cache's values: codes times scales, which msa_fwd takes rounded to bf16
        k, v = ((c.view(torch.float8_e4m3fn).float() * s[..., None]).bfloat16()
                for c, s in (ops.msa_quantize_kv_fp8(k), ops.msa_quantize_kv_fp8(v)))
    out = []
    for topk in (TOPK, (k.shape[1] + 127) // 128):
        sets, _ = ops.msa_index_topk(qi, ki, topk, H_q=H_q, d=D)
        o, lse = ops.msa_fwd(q, k, v, sets, d_idx=DI)
        out.append((sets[0], o[0], lse[0]))
    return out


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_then_captured_decode(fp8):
    prompts, steps, page = [300, 517, 1], 9, 16
    # the training path takes a cached E4M3 key rounded to bf16, which moves a score by up to
    # scale * sum |q k| 2^-9 = 64^-0.5 * 64 * E|q k| (0.64) * 2^-9 = 1e-2, and the lse with it
    lse_tol = 2e-2 if fp8 else LSE_TOL
    seqs = sequences([n + steps for n in prompts], 1)
    rope = ops.new_rope(ROT, scaling={"type": "yarn", "factor": 4, "original_len": 256})
    want = [training_rows(s, rope, fp8) for s in seqs]
    slots = 4  # one stays empty
    pages = sum((n + steps + page - 1) // page for n in prompts)
    cache = ops.new_paged_cache(pages, H_kv, page_size=page, d=D, d_idx=DI, fp8=fp8)
    order, at = np.random.default_rng(2).permutation(pages), 0
    table = np.full((slots, (max(prompts) + steps + page - 1) // page), -1)
    rows = [0, 2, 3]  # slot of each sequence
    for r, n in zip(rows, prompts):
        m = (n + steps + page - 1) // page
        table[r, :m] = order[at:at + m]
        at += m
    table = dev(table)
    # prompts: packed, rotated at their positions, written
    lens = np.zeros(slots, dtype=np.int64)
    lens[rows] = prompts
    cu = dev(np.concatenate([[0], np.cumsum(lens)]))
    q, k, v, qi, ki = (torch.cat([s[i][:n] for s, n in zip(seqs, prompts)]) for i in range(5))
    pos = torch.cat([torch.arange(n, device="cuda") for n in prompts])
    q, k, qi, ki = ops.msa_rope((q, k, qi, ki), rope, pos)
    ops.msa_cache_write(cache, table, dev(lens), k, v, ki, cu_seqlens=cu)
    # the prompts read back: the training path's forward on them, as a packed batch
    gk, gv, gi = ops.msa_cache_read(cache, table, dev(lens), cu, sum(prompts))
    assert torch.equal(gi, ki)
    sets, _ = ops.msa_index_topk_varlen(qi, gi, cu, TOPK, max_seqlen=max(prompts), H_q=H_q, d=D)
    o, _ = ops.msa_fwd_varlen(q, gk, gv, sets, cu, TOPK, max_seqlen=max(prompts), d_idx=DI)
    first = 0
    for n, w in zip(prompts, want):
        assert (o[first:first + n].float() - w[0][1][:n].float()).abs().max() <= O_TOL
        first += n
    # decode: one captured step, its inputs filled in place
    n_t, pos_t = dev(np.zeros(slots)), torch.zeros(slots, dtype=torch.int64, device="cuda")
    new = [torch.zeros(slots, *x.shape[1:], dtype=torch.bfloat16, device="cuda") for x in seqs[0]]

    def step():
        rq, rk, rqi, rki = ops.msa_rope((new[0], new[1], new[3], new[4]), rope, pos_t)
        ops.msa_cache_write(cache, table, n_t, rk, new[2], rki)
        return (ops.msa_decode_paged(rq, rqi, cache, table, n_t, TOPK),
                ops.msa_decode_paged_dense(rq, cache, table, n_t))

    step()  # empty slots only: nothing is written
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (sets, o, lse), (o_dense, lse_dense) = step()
    for t in range(steps):
        for r, s, n in zip(rows, seqs, prompts):
            for x, y in zip(new, s):
                x[r] = y[n + t]
            n_t[r], pos_t[r] = n + t + 1, n + t
        graph.replay()
        torch.cuda.synchronize()
        assert ops.device_status() == 0
        assert (sets[1] == -1).all() and not o[1].any() and not o_dense[1].any()
        for r, n, (sparse, dense) in zip(rows, prompts, want):
            i = n + t
            assert torch.equal(sets[r], sparse[0][:, i])
            assert (o[r].float() - sparse[1][i].float()).abs().max() <= O_TOL
            assert (lse[r] - sparse[2][:, i]).abs().max() <= lse_tol
            assert (o_dense[r].float() - dense[1][i].float()).abs().max() <= O_TOL
            assert (lse_dense[r] - dense[2][:, i]).abs().max() <= lse_tol
