"""More of the serving operators around block-sparse attention, as cases to measure.

  append        a call's new tokens turned to their positions and stored: q and q_idx come back
                rotated, k and k_idx are rotated into a paged cache and v is written beside them
                (bf16, E4M3 codes, or E2M1 codes of 4 bits)
  cache         keys, values and index keys written into a cache of 4-bit codes and read back
  decode_dense  attention of one new token a sequence over its whole 4-bit cache
  decode_sparse block selection for one new token over the paged index keys, and attention over
                the selected blocks of a 4-bit cache

A row (one head's key or value of a token, d values) of a 4-bit cache is d / 2 bytes of E2M1 codes,
the even value in the low half of a byte, and 4 + d / 16 bytes of scales: a float32 power of two for
the row and an E4M3 number for each 16 values.  A value is code x block scale x row scale.  For a row
of largest magnitude a and a block of largest magnitude b:
  row scale   = the smallest power of two s with a <= 2688 s (2688 = 6 x 448; 1 for a row of zeros)
  block scale = the E4M3 number nearest to b / (6 s), at least 2^-9
  code        = the E2M1 number nearest to x / (block scale x s), ties to even

Sizes are those of the repository's workloads (tiny, 8k, 32k, 128k and the decode leg of the
benchmark: 8 caches of 128K tokens), with odd and ragged ones between them.  Ragged lengths belong
to a case (drawn from its `shape_seed`), so that its work is known; the values and the order of the
cache's pages come from the seed.
"""
import math
import random

import torch

own = False

BK = 128  # tokens of a selectable block


# ---------------------------------------------------------------------------- the cases
def listed():
    heads32 = {"H_q": 32, "H_kv": 8, "d": 128, "d_idx": 64}
    heads16 = {"H_q": 16, "H_kv": 4, "d": 128, "d_idx": 64}
    tiny = {"H_q": 8, "H_kv": 2, "d": 64, "d_idx": 32}
    plain = {"layout": "half", "scaling": "none", "fused": False, "far": 0}
    return [
        # one decode step of 8 sequences, every slot in use: latency
        {"name": "append_step_8", "op": "append", "B": 8, "L": 4096, "new": 1, **heads32, "kind": "bf16",
         "page": 128, "rot": 64, **plain, "shape_seed": 0},
        # one decode step of 64 ragged sequences with an empty slot, small pages of E4M3 codes,
        # positions of their own (a window that has moved on), frequencies stretched for long contexts
        {"name": "append_step_64_ragged", "op": "append", "B": 64, "L": 2000, "new": 1, **heads16,
         "kind": "e4m3", "page": 16, "rot": 32, "layout": "interleaved", "scaling": "yarn", "fused": True,
         "far": 1048576, "shape_seed": 21},
        # a chunk of each of three prompts into a 4-bit cache, the operands views of one projection
        {"name": "append_chunks_3x700", "op": "append", "B": 3, "L": 5000, "new": 700, **tiny, "kind": "e2m1",
         "page": 64, "rot": 32, "layout": "half", "scaling": "none", "fused": True, "far": 0, "shape_seed": 22},
        # a 32K prompt: the whole of it at once
        {"name": "append_prompt_32k", "op": "append", "B": 1, "L": 32768, "new": 32768, **heads32,
         "kind": "bf16", "page": 128, "rot": 64, **plain, "shape_seed": 0},
        # a 32K prompt written in 4 bits and read back as the context of the next chunk
        {"name": "cache_prompt_32k", "op": "cache", "mode": "both", "B": 1, "L": 32768, "new": 32768,
         **heads32, "page": 128, "shape_seed": 0},
        # ragged contexts of a mixed batch read back
        {"name": "cache_read_ragged", "op": "cache", "mode": "read", "B": 9, "L": 20000, "new": 0, **heads16,
         "page": 64, "shape_seed": 23},
        # one short sequence: latency
        {"name": "dense_1x700", "op": "dense", "B": 1, "L": 700, **tiny, "page": 16, "shape_seed": 0},
        # a mixed batch, one of its slots empty
        {"name": "dense_32_ragged", "op": "dense", "B": 32, "L": 8192, **heads16, "page": 64, "shape_seed": 24},
        # the long-context batch: 8 caches of 128K tokens
        {"name": "dense_8x128k", "op": "dense", "B": 8, "L": 131072, **heads32, "page": 128, "shape_seed": 0},
        # one tiny sequence: latency of the whole chain
        {"name": "sparse_1x2k", "op": "sparse", "B": 1, "L": 2048, **tiny, "topk": 4, "page": 128,
         "shape_seed": 0},
        # the decode leg of the benchmark over pages of 4-bit codes
        {"name": "sparse_8x128k", "op": "sparse", "B": 8, "L": 131072, **heads32, "topk": 16, "page": 128,
         "shape_seed": 0},
        # a mixed batch with few groups of many heads, small pages
        {"name": "sparse_16_ragged", "op": "sparse", "B": 16, "L": 40000, "H_q": 16, "H_kv": 2, "d": 128,
         "d_idx": 64, "topk": 16, "page": 16, "shape_seed": 25},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "cache", "dense", "sparse"])
    d = rng.choice([64, 128])
    d_idx = rng.choice([32, 64])
    H_kv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8, 16])
    while H_kv * G > 32:
        G //= 2
    case = {"op": op, "H_q": H_kv * G, "H_kv": H_kv, "d": d, "d_idx": d_idx,
            "page": rng.choice([16, 48, 64, 128, 256]), "shape_seed": rng.randrange(1, 1 << 20)}
    if op == "append":
        B = _log(rng, 1, 64)
        L = _log(rng, 1, 32000 // B + 1)
        return case | {"B": B, "L": L, "new": rng.choice([1, 1, L, max(1, L // 3)]),
                       "kind": rng.choice(["bf16", "e4m3", "e2m1"]),
                       "rot": rng.choice([d_idx // 2, d_idx // 2 + 2, d_idx, d_idx]),
                       "layout": rng.choice(["half", "interleaved"]),
                       "scaling": rng.choice(["none", "linear", "ntk", "yarn"]),
                       "fused": rng.random() < 0.4, "far": rng.choice([0, 0, 131072, 1048576])}
    if op == "cache":
        B = _log(rng, 1, 64)
        L = _log(rng, 1, 30000 // B + 1)
        mode = rng.choice(["read", "both"])
        return case | {"mode": mode, "B": B, "L": L, "new": 0 if mode == "read" else rng.choice([1, L, max(1, L // 3)])}
    B = _log(rng, 1, 64)
    L = _log(rng, 1, 400000 // B + 1)
    case |= {"B": B, "L": min(L, 131072)}
    if op == "sparse":
        case["topk"] = rng.choice([1, 4, 8, 16, 16, 20, 32])
    return case


def _lens(case):
    """Cache lengths of a case's sequences, the new tokens among them: all L where shape_seed is
    0, else spread over 1 .. L by their logarithm, with one full, one of a single token and (from 4
    sequences on) one empty slot."""
    B, L = case["B"], case["L"]
    if not case["shape_seed"]:
        return [L] * B
    r = random.Random(case["shape_seed"])
    lens = [_log(r, 1, L) for _ in range(B)]
    lens[r.randrange(B)] = L
    if B >= 4:
        a, b, c = r.sample(range(B), 3)
        lens[a], lens[b], lens[c] = L, 1, 0
    return lens


def _news(case):
    """Tokens of each sequence that are new in this call (none beyond its length)."""
    return [min(case["new"], n) for n in _lens(case)]


def _step(case):
    """A decode step: one token a slot, empty slots among them, and no cu_seqlens."""
    return case["op"] == "append" and case["new"] == 1


# ------------------------------------------------------------- frequencies of the rotations
def _base_scaling(case):
    return {"none": None, "linear": {"type": "linear", "factor": 4.0},
            "ntk": {"type": "ntk", "factor": 4.0},
            "yarn": {"type": "yarn", "factor": 4.0, "original_len": 32768}}[case["scaling"]]


def _frequencies(case):
    """Radians a position of each pair (64 bits), and the factor on the rotated values."""
    rot, base = case["rot"], 10000.0
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    s = _base_scaling(case)
    if s is None:
        return base ** (-2.0 * i / rot), 1.0
    if s["type"] == "ntk":
        return (base * s["factor"] ** (rot / (rot - 2))) ** (-2.0 * i / rot), 1.0
    f = base ** (-2.0 * i / rot)
    if s["type"] == "linear":
        return f / s["factor"], 1.0
    turns = s["original_len"] * f / (2 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0, 1)
    return f * keep + f / s["factor"] * (1 - keep), 0.1 * math.log(s["factor"]) + 1.0


# ------------------------------------------------------------------------------- inputs
def _prepare_pages(case, g):
    """A shuffled page table with a few pages that nobody holds, and pages full of values."""
    lens, page, H, d = _lens(case), case["page"], case["H_kv"], case["d"]
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
    table, at = torch.full((case["B"], (case["L"] + page - 1) // page), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    kind = case.get("kind", "e2m1")
    state = {"table": table.cuda(), "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
             "k_idx": torch.randn(pages, page, case["d_idx"], generator=g, device="cuda").bfloat16()}
    for n in ("k", "v"):
        if kind == "bf16":
            state[n] = torch.randn(pages, page, H, d, generator=g, device="cuda").bfloat16()
        elif kind == "e4m3":
            codes = (torch.randn(pages, page, H, d, generator=g, device="cuda") * 100).clamp(-448, 448)
            state[n] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
            state[n + "_scale"] = torch.rand(pages, page, H, generator=g, device="cuda") * 0.01 + 0.005
        else:  # values of about 1: blocks of 60 to 448, rows of 2^-9 and 2^-8
            state[n] = torch.randint(0, 256, (pages, page, H, d // 2), generator=g, device="cuda", dtype=torch.uint8)
            scale = torch.empty(pages, page, H, 4 + d // 16, dtype=torch.uint8, device="cuda")
            row = torch.randint(-9, -7, (pages, page, H, 1), generator=g, device="cuda").float()
            scale[..., :4] = torch.exp2(row).view(torch.uint8)
            scale[..., 4:] = torch.randint(0x67, 0x7F, (pages, page, H, d // 16), generator=g, device="cuda",
                                           dtype=torch.uint8)
            state[n + "_scale"] = scale
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case, **_prepare_pages(case, g)}
    B, H_q, H, d, di = (case[n] for n in ("B", "H_q", "H_kv", "d", "d_idx"))

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda").bfloat16()

    if case["op"] in ("append", "cache"):
        counts = _lens(case) if case.get("mode") == "read" else _news(case)
        state["total"] = sum(counts)
        state["cu"] = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        step = _step(case)
        state["live"] = torch.tensor([b for b, n in enumerate(counts) if n], device="cuda") if step else slice(None)
        T = B if step else sum(counts)
        if case["op"] == "append":
            rows = [(H_q, d), (H, d), (H, d), (H, di), (1, di)]
            widths = [h * w for h, w in rows]
            if case["fused"]:  # one projection's output, the operands its columns
                parts = torch.split(randn(T, sum(widths)), widths, dim=-1)
            else:
                parts = [randn(T, w) for w in widths]
            xs = [p.unflatten(-1, r) for p, r in zip(parts, rows)]
            state |= dict(zip(("q", "new_k", "new_v", "q_idx"), xs)) | {"new_k_idx": xs[4].squeeze(-2)}
            if case["far"]:
                state["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        elif case["mode"] == "both":
            state |= {"new_k": randn(T, H, d), "new_v": randn(T, H, d), "new_k_idx": randn(T, di)}
    else:
        state["q"] = randn(B, H_q, d)
        if case["op"] == "sparse":
            state["q_idx"] = randn(B, H, di)
    if own:
        from block_sparse_gqa_topk_gb300 import ops
        state["cache"] = ops.PagedCache(state["k"], state["v"], state["k_idx"], state.get("k_scale"),
                                        state.get("v_scale"))
        if case["op"] == "append":
            state["rope"] = ops.new_rope(case["rot"], interleaved=case["layout"] == "interleaved",
                                         scaling=_base_scaling(case))
    return state


# ---------------------------------------------------------------------------- plain forms
def _e2m1_table():
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    return torch.cat((half, -half))


def _e2m1_values(codes, scale):
    """Rows of 4-bit codes and their scales as 32-bit values."""
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    x = _e2m1_table()[both.int()].unflatten(-1, (-1, 16))
    block = scale[..., 4:].contiguous().view(torch.float8_e4m3fn).float()
    row = scale[..., :4].contiguous().view(torch.float32)
    return (x * block[..., None]).flatten(-2) * row


def _e2m1_codes(x):
    """Rows of 32-bit values as 4-bit codes and scales (a row scale is a power of two, so that the
    quotients by it are exact)."""
    part, exponent = torch.frexp(x.abs().amax(-1, keepdim=True))
    exponent = torch.where(part > 0, exponent - 12 + (part > 2688 / 4096).int(), 0)
    y = torch.ldexp(x, -exponent).unflatten(-1, (-1, 16))
    six = torch.full((), 6.0, device="cuda")  # a number here would be a product with 1 / 6
    block = (y.abs().amax(-1, keepdim=True) / six).clamp(min=2.0 ** -9).to(torch.float8_e4m3fn)
    y = y / block.float()
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
            + torch.signbit(y).to(torch.uint8) * 8).flatten(-2)
    row = torch.ldexp(torch.ones((), device="cuda"), exponent).contiguous()
    return (code[..., 0::2] | (code[..., 1::2] << 4),
            torch.cat((row.view(torch.uint8), block.squeeze(-1).view(torch.uint8)), -1))


def _places(s):
    """Pool rows (page * page_size + offset) of the tokens that a call stores or reads, and the
    tokens' places in their sequences."""
    page, cu, lens = s["case"]["page"], s["cu"].long(), s["lens"].long()
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = lens[b] - (cu[b + 1] - t)
    return s["table"].long()[b, pos // page] * page + pos % page, pos


def _store(s, rows, k, v, k_idx):
    kind = s["case"].get("kind", "e2m1")
    s["k_idx"].flatten(0, 1)[rows] = k_idx
    for n, x in (("k", k), ("v", v)):
        if kind == "bf16":
            s[n].flatten(0, 1)[rows] = x
            continue
        x = x.float()
        if kind == "e4m3":
            top = x.abs().amax(-1)
            most = torch.full((), 448.0, device="cuda")  # as above
            scale = torch.where(top > 0, top / most, 1.0)
            codes = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            codes, scale = _e2m1_codes(x)
        s[n].flatten(0, 1)[rows] = codes
        s[n + "_scale"].flatten(0, 1)[rows] = scale


def _values(s, name, cells, flat):
    """Cached keys or values as 32-bit numbers, of rows of the pool whose first `flat` axes are one."""
    x, kind = s[name].flatten(0, flat)[cells], s["case"].get("kind", "e2m1")
    if kind == "bf16":
        return x.float()
    scale = s[name + "_scale"].flatten(0, flat)[cells]
    return x.view(torch.float8_e4m3fn).float() * scale[..., None] if kind == "e4m3" else _e2m1_values(x, scale)


def _read(s, rows):
    return {"k": _values(s, "k", rows, 1).bfloat16(), "v": _values(s, "v", rows, 1).bfloat16(),
            "k_idx": s["k_idx"].flatten(0, 1)[rows]}


def _plain_cache(s):
    rows, _ = _places(s)
    if s["case"]["mode"] == "both":
        _store(s, rows, s["new_k"], s["new_v"], s["new_k_idx"])
    return _read(s, rows)


def _plain_append(s):
    case, live = s["case"], s["live"]
    rot, inter = case["rot"], case["layout"] == "interleaved"
    rows, pos = _places(s)
    if case["far"]:
        pos = s["positions"][live]
    freq, mul = _frequencies(case)
    angle = pos.double()[:, None] * freq
    cos, sin = (angle.cos() * mul).float()[:, None], (angle.sin() * mul).float()[:, None]

    def turn(x):  # [tokens, heads, width], in 32 bits, rounded once
        y = x.float()
        head, tail = y[..., :rot], y[..., rot:]
        a, b = (head[..., 0::2], head[..., 1::2]) if inter else (head[..., :rot // 2], head[..., rot // 2:])
        a, b = a * cos - b * sin, b * cos + a * sin
        head = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
        return torch.cat((head, tail), -1).bfloat16()

    out = {"q": torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda"),
           "q_idx": torch.zeros(s["q_idx"].shape, dtype=torch.bfloat16, device="cuda")}
    out["q"][live], out["q_idx"][live] = turn(s["q"][live]), turn(s["q_idx"][live])
    # a cache of codes codes the turned keys as they are in bf16
    _store(s, rows, turn(s["new_k"][live]), s["new_v"][live], turn(s["new_k_idx"][live][:, None])[:, 0])
    return out | ({n: s[n] for n in ("k", "v", "k_idx")} if case["kind"] == "bf16" else _read(s, rows))


def _softmax_join(scores, seen):
    """Weights of the seen scores and their log-sum-exp; none seen: no weight, -inf."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = (scores - top).exp()
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0), (top + total.log()).squeeze(-1)


def _plain_dense(s):
    case = s["case"]
    B, H, d, page = case["B"], case["H_kv"], case["d"], case["page"]
    G = case["H_q"] // H
    pos = torch.arange(case["L"], device="cuda")
    seen = pos < s["lens"][:, None]
    rows = s["table"].long().clamp(min=0)[:, pos // page] * page + pos % page  # [B, L]
    q = s["q"].float().view(B, H, G, d) / math.sqrt(d)
    w, lse = _softmax_join(q @ _values(s, "k", rows, 1).permute(0, 2, 3, 1), seen[:, None, None, :])
    o = w @ _values(s, "v", rows, 1).permute(0, 2, 1, 3)
    return {"o": o.view(B, H * G, d).bfloat16(), "lse": lse.view(B, H * G)}


def _plain_sparse(s):
    case = s["case"]
    B, H, d, page, topk = case["B"], case["H_kv"], case["d"], case["page"], case["topk"]
    G = case["H_q"] // H
    nb = (case["L"] + BK - 1) // BK
    pos = torch.arange(nb * BK, device="cuda")
    table, lens = s["table"].long().clamp(min=0), s["lens"].long()
    rows = table[:, (pos // page).clamp(max=table.shape[1] - 1)] * page + pos % page  # [B, nb * 128]
    # scores beside the border between taken and left blocks: 64 bits
    z = s["q_idx"].double() @ s["k_idx"].flatten(0, 1)[rows].double().transpose(1, 2)
    pooled = z.view(B, H, nb, BK).amax(-1)
    block = torch.arange(nb, device="cuda")
    mine = ((lens - 1).clamp(min=0) // BK)[:, None, None]
    pooled = pooled.masked_fill(block >= mine, -math.inf)
    pooled = pooled.masked_fill((block == mine) & (lens[:, None, None] > 0), math.inf)
    value, index = pooled.sort(dim=-1, descending=True, stable=True)  # equal scores: lower block first
    value, index = value[..., :topk], index[..., :topk]
    index = torch.where(value > -math.inf, index, nb).sort(-1).values
    if nb < topk:
        index = torch.nn.functional.pad(index, (0, topk - nb), value=nb)
    chosen = torch.where(index < nb, index, -1)  # [B, H, topk]
    at = (chosen.clamp(min=0)[..., None] * BK + torch.arange(BK, device="cuda")).flatten(-2)
    seen = (chosen >= 0).repeat_interleave(BK, -1) & (at < lens[:, None, None])
    batch = torch.arange(B, device="cuda")[:, None, None]
    head = torch.arange(H, device="cuda")[None, :, None]
    cell = (table[batch, (at // page).clamp(max=table.shape[1] - 1)] * page + at % page) * H + head
    q = s["q"].float().view(B, H, G, d) / math.sqrt(d)
    w, lse = _softmax_join(q @ _values(s, "k", cell, 2).transpose(-1, -2), seen[:, :, None, :])
    o = w @ _values(s, "v", cell, 2)
    return {"block_idx": chosen.int(), "o": o.view(B, H * G, d).bfloat16(), "lse": lse.view(B, H * G)}


# ------------------------------------------------------------------------ the framework's
def _own_run(s):
    from block_sparse_gqa_topk_gb300 import ops
    case = s["case"]
    if case["op"] == "append":
        q, q_idx = ops.msa_cache_append(s["cache"], s["table"], s["lens"], s["rope"], s["q"], s["new_k"], s["new_v"],
                                        s["q_idx"], s["new_k_idx"], positions=s.get("positions"),
                                        cu_seqlens=None if _step(case) else s["cu"])
        if case["kind"] == "bf16":
            return {"q": q, "q_idx": q_idx, "k": s["k"], "v": s["v"], "k_idx": s["k_idx"]}
        k, v, k_idx = ops.msa_cache_read(s["cache"], s["table"], s["lens"], s["cu"], s["total"])
        return {"q": q, "q_idx": q_idx, "k": k, "v": v, "k_idx": k_idx}
    if case["op"] == "cache":
        if case["mode"] == "both":
            ops.msa_cache_write(s["cache"], s["table"], s["lens"], s["new_k"], s["new_v"], s["new_k_idx"],
                                cu_seqlens=s["cu"])
        k, v, k_idx = ops.msa_cache_read(s["cache"], s["table"], s["lens"], s["cu"], s["total"])
        return {"k": k, "v": v, "k_idx": k_idx}
    if case["op"] == "dense":
        o, lse = ops.msa_decode_paged_dense(s["q"], s["cache"], s["table"], s["lens"])
        return {"o": o, "lse": lse}
    block_idx, o, lse = ops.msa_decode_paged(s["q"], s["q_idx"], s["cache"], s["table"], s["lens"], case["topk"])
    return {"block_idx": block_idx, "o": o, "lse": lse}


def run(state):
    if own:
        return _own_run(state)
    return {"append": _plain_append, "cache": _plain_cache, "dense": _plain_dense,
            "sparse": _plain_sparse}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- 64-bit values
def _exact_turns(case, pos):
    """Unit factors exp(i angle) x mscale of each position and pair."""
    rot = case["rot"]
    kind, factor = case["scaling"], 4.0
    base = 10000.0 * (factor ** (rot / (rot - 2.0)) if kind == "ntk" else 1.0)
    freqs, mul = [], 1.0
    for i in range(rot // 2):
        f = base ** (-(2.0 * i) / rot)
        if kind == "linear":
            f = f / factor
        elif kind == "yarn":
            g = min(1.0, max(0.0, (32768 / (2.0 * math.pi / f) - 1.0) / (32.0 - 1.0)))
            f = (1.0 - g) * (f / factor) + g * f
        freqs.append(f)
    if kind == "yarn":
        mul = 1.0 + 0.1 * math.log(factor)
    w = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    return torch.polar(torch.full((), mul, dtype=torch.float64, device="cuda"), pos.reshape(-1, 1).double() * w)


def _exact_turned(case, x, unit):
    rot, half = case["rot"], case["rot"] // 2
    y = x.double().reshape(unit.shape[0], -1, x.shape[-1]).clone()
    if case["layout"] == "interleaved":
        z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * unit[:, None, :]
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :half], y[..., half:rot]) * unit[:, None, :]
        y[..., :half], y[..., half:rot] = z.real, z.imag
    return y.reshape(x.shape)


def _small_float(codes, mantissa, bias):
    """Values of codes of a sign, an exponent and `mantissa` bits, from the format's fields (the
    sign bit is the caller's)."""
    c = codes.long()
    e, m = c >> mantissa, (c & ((1 << mantissa) - 1)).double()
    one = float(1 << mantissa)
    return torch.where(e == 0, m * 2.0 ** (1 - bias) / one, (one + m) / one * torch.exp2(e.double() - bias))


def _e4m3_value(c):
    mag = _small_float(c & 127, 3, 7)
    return torch.where(c >= 128, -mag, mag)


def _nearest(x, mantissa, least, most):
    """The nearest number with `mantissa` bits behind the first (ties to even), exponents from
    `least` on, magnitudes to `most`."""
    a = x.abs()
    floor = a.clamp(min=2.0 ** least)
    e = torch.floor(torch.log2(floor))
    e = torch.where(torch.exp2(e) > floor, e - 1, e)
    step = torch.exp2(e - mantissa)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=most)


def _exact_cached(kind, x):
    """The values that a cache holds for rows x (64 bits)."""
    if kind == "bf16":
        return x
    top = x.abs().amax(-1, keepdim=True)
    if kind == "e4m3":
        # a cached row's scale and the quotients that are coded have 32 bits by definition: in 64,
        # ties between two codes would fall the other way
        scale = torch.where(top > 0, top / 448.0, torch.ones_like(top)).float().double()
        return _nearest((x / scale).float().double(), 3, -6, 448.0) * scale
    row = torch.exp2(torch.ceil(torch.log2(top / 2688)))
    row = torch.where(row * 2688 < top, row * 2, torch.where(row * 1344 >= top, row / 2, row))
    row = torch.where(top > 0, row, 1.0)
    y = (x / row).unflatten(-1, (x.shape[-1] // 16, 16))
    block = _nearest(y.abs().amax(-1, keepdim=True) / 6, 3, -6, 448.0).clamp(min=2.0 ** -9)
    return (_nearest(y / block, 1, 0, 6.0) * block).reshape(x.shape) * row


def _exact_held(case, s, name, rows):
    """The values that rows of the pool hold."""
    x, kind = s[name].flatten(0, 1)[rows], case.get("kind", "e2m1")
    if kind == "bf16" or name == "k_idx":
        return x.double()
    scale = s[name + "_scale"].flatten(0, 1)[rows]
    if kind == "e4m3":
        return _e4m3_value(x) * scale.double()[..., None]
    low, high = x & 15, x >> 4
    y = torch.stack([torch.where(c >= 8, -1.0, 1.0) * _small_float(c & 7, 1, 1) for c in (low, high)], -1)
    y = y.flatten(-2).unflatten(-1, (x.shape[-1] // 8, 16)) * _e4m3_value(scale[..., 4:])[..., None]
    return y.flatten(-2) * scale[..., :4].contiguous().view(torch.float32).double()


def _sequence(s, b, n):
    """Pool rows of the first n tokens of sequence b, page after page."""
    page = s["case"]["page"]
    ids = s["table"][b, :(n + page - 1) // page].long()
    return (ids[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]


def _exact_cache(case, s):
    counts = _lens(case) if case["mode"] == "read" else _news(case)
    out = {"k": [], "v": [], "k_idx": []}
    at = 0
    for b, (n, c) in enumerate(zip(_lens(case), counts)):
        rows = _sequence(s, b, n)[n - c:]
        for name in out:
            if case["mode"] == "read":
                out[name].append(_exact_held(case, s, name, rows))
            else:
                x = s["new_" + name][at:at + c].double()
                out[name].append(x if name == "k_idx" else _exact_cached("e2m1", x))
        at += c
    return {n: torch.cat(p) for n, p in out.items()}


def _exact_append(case, s):
    names = ("k", "v", "k_idx")
    out = {"q": torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"),
           "q_idx": torch.zeros(s["q_idx"].shape, dtype=torch.float64, device="cuda")}
    pool = {n: s[n].double().flatten(0, 1) for n in names} if case["kind"] == "bf16" else None
    new = {n: [] for n in names}
    at = 0
    for b, (n, c) in enumerate(zip(_lens(case), _news(case))):
        if _step(case):
            at = b
        if c == 0:
            continue
        t = slice(at, at + c)
        unit = _exact_turns(case, s["positions"][t] if case["far"] else torch.arange(n - c, n, device="cuda"))
        for name in ("q", "q_idx"):
            out[name][t] = _exact_turned(case, s[name][t], unit)
        got = {"k": _exact_turned(case, s["new_k"][t], unit), "v": s["new_v"][t].double(),
               "k_idx": _exact_turned(case, s["new_k_idx"][t], unit)}
        if case["kind"] != "bf16":  # codes are those of the turned keys in bf16, by definition
            got = {m: x if m == "k_idx" else _exact_cached(case["kind"], x.bfloat16().double()) for m, x in got.items()}
        for m in names:
            if pool is None:
                new[m].append(got[m])
            else:
                pool[m][_sequence(s, b, n)[n - c:]] = got[m]
        at += c
    return out | ({n: torch.cat(p) for n, p in new.items()} if pool is None else
                  {n: p.view(s[n].shape) for n, p in pool.items()})


def _exact_attend(q, k, v):
    """Softmax attention of q [G, d] over k, v [n, d] (64 bits): values and log-sum-exp."""
    z = (q @ k.T) * (q.shape[-1] ** -0.5)
    lse = torch.logsumexp(z, -1)
    return torch.exp(z - lse[:, None]) @ v, lse


def _exact_decode(case, s):
    B, H_q, H, d = case["B"], case["H_q"], case["H_kv"], case["d"]
    G = H_q // H
    o = torch.zeros(B, H_q, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H_q), -math.inf, dtype=torch.float64, device="cuda")
    sets = torch.full((B, H, case.get("topk", 1)), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        rows = _sequence(s, b, n)
        own_block = (n - 1) // BK
        if case["op"] == "sparse":
            z = s["q_idx"][b].double() @ s["k_idx"].flatten(0, 1)[rows[:own_block * BK]].double().T
            best = z.view(H, own_block, BK).amax(-1) if own_block else z.new_zeros(H, 0)
        for g in range(H):
            use = rows
            if case["op"] == "sparse":
                take = sorted(torch.sort(best[g], dim=-1, descending=True, stable=True).indices[:case["topk"] - 1]
                              .tolist()) + [own_block]
                sets[b, g, :len(take)] = torch.tensor(take, dtype=torch.int32)
                use = torch.cat([rows[c * BK:(c + 1) * BK] for c in take])
            k, v = (_exact_held(case, s, name, (use, g)) for name in ("k", "v"))
            h = slice(g * G, (g + 1) * G)
            o[b, h], lse[b, h] = _exact_attend(s["q"][b, h].double(), k, v)
    return {"block_idx": sets, "o": o, "lse": lse} if case["op"] == "sparse" else {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"append": _exact_append, "cache": _exact_cache}.get(case["op"], _exact_decode)(case, s)


# ----------------------------------------------------------------------------------- work
def work(case):
    H_q, H, d, di = case["H_q"], case["H_kv"], case["d"], case["d_idx"]
    kind = case.get("kind", "e2m1")
    row = {"bf16": 2 * d, "e4m3": d + 4, "e2m1": d // 2 + d // 16 + 4}[kind]  # one head's cached key or value
    lens = _lens(case)
    stored = 2 * H * row + 2 * di  # a token in the cache, and as it comes
    given = 4 * H * d + 2 * di
    if case["op"] == "append":
        T = sum(_news(case))
        turned = (H_q * d + H * di) * 2
        return {"bytes": T * (2 * turned + given + stored + (0 if kind == "bf16" else stored + given)
                              + (4 if case["far"] else 0)),
                "flops": T * ((H_q + 2 * H + 1) * case["rot"] * 3 + (0 if kind == "bf16" else 6 * H * d))}
    if case["op"] == "cache":
        T, sides = (sum(lens), 1) if case["mode"] == "read" else (sum(_news(case)), 2)
        return {"bytes": sides * T * (given + stored), "flops": sides * T * 4 * H * d}
    G = H_q // H
    small = case["B"] * (2 * H_q * d * 2 + H_q * 4)  # q, o and lse
    if case["op"] == "dense":
        tokens = H * sum(lens)
        return {"bytes": tokens * 2 * row + small, "flops": tokens * G * 4 * d}
    keys = picked = 0
    for n in lens:
        if n:
            before = (n - 1) // BK
            keys += before * BK
            picked += min(case["topk"] - 1, before) * BK + n - before * BK
    return {"bytes": keys * di * 2 + picked * H * 2 * row + small + case["B"] * H * (di * 2 + case["topk"] * 4),
            "flops": keys * H * 2 * di + picked * H * G * 4 * d}
