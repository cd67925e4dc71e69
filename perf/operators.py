"""The serving and position operators around block-sparse attention, as cases to measure.

  rope          rotary positions of q, k, q_idx and k_idx in one call, with the gradient
  cache         keys, values and index keys written into a paged cache (bf16, or E4M3 codes
                with one scale a row) and read back in token order
  decode_dense  attention of one new token a sequence over its whole paged cache
  decode_sparse block selection for one new token over the paged index keys, and attention
                over the selected blocks

Sizes are those of the repository's workloads (tiny, 8k, 32k, 128k and the decode leg of the
benchmark: 8 caches of 128K tokens), with odd and ragged ones between them.  Ragged lengths
belong to a case (drawn from its `shape_seed`), so that its work is known; the values and the
order of the cache's pages come from the seed.
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
    return [
        # one decode step of 8 sequences: the four projections of each new token, rotated far out
        {"name": "rope_step_8", "op": "rope", "B": 0, "N": 8, **heads32, "rot": 64, "layout": "half",
         "scaling": "none", "dtype": "bf16", "fused": False, "grad": False, "far": 131072},
        # the 128K training workload: all four tensors, forward and backward
        {"name": "rope_train_128k", "op": "rope", "B": 1, "N": 131072, **heads32, "rot": 64,
         "layout": "half", "scaling": "none", "dtype": "bf16", "fused": False, "grad": True, "far": 0},
        # a packed fp16 batch of an odd length, interleaved pairs over the whole index head,
        # frequencies stretched for a longer context, views of one fused projection
        {"name": "rope_fused_5001", "op": "rope", "B": 0, "N": 5001, **heads16, "rot": 64,
         "layout": "interleaved", "scaling": "yarn", "dtype": "fp16", "fused": True, "grad": True,
         "far": 65536},
        # one decode step of 64 sequences: a token each into a bf16 cache of small pages
        {"name": "cache_step_64", "op": "cache", "mode": "write", "B": 64, "L": 1024, "new": 1,
         **heads32, "kind": "bf16", "page": 16, "shape_seed": 11},
        # a 32K prompt written as E4M3 and read back as the context of the next chunk
        {"name": "cache_prompt_32k", "op": "cache", "mode": "both", "B": 1, "L": 32768, "new": 32768,
         **heads32, "kind": "e4m3", "page": 128, "shape_seed": 0},
        # ragged contexts of a mixed batch read back from an E4M3 cache
        {"name": "cache_read_ragged", "op": "cache", "mode": "read", "B": 9, "L": 20000, "new": 0,
         **heads16, "kind": "e4m3", "page": 64, "shape_seed": 12},
        # one short sequence: latency
        {"name": "dense_1x700", "op": "dense", "B": 1, "L": 700, **tiny, "kind": "bf16", "page": 16,
         "shape_seed": 0},
        # a mixed batch, one of its slots empty, E4M3 cache
        {"name": "dense_32_ragged", "op": "dense", "B": 32, "L": 8192, **heads16, "kind": "e4m3",
         "page": 64, "shape_seed": 13},
        # the long-context batch: 8 caches of 128K tokens
        {"name": "dense_8x128k", "op": "dense", "B": 8, "L": 131072, **heads32, "kind": "bf16",
         "page": 128, "shape_seed": 0},
        # one tiny sequence: latency of the whole chain
        {"name": "sparse_1x2k", "op": "sparse", "B": 1, "L": 2048, **tiny, "topk": 4, "kind": "bf16",
         "page": 128, "shape_seed": 0},
        # the decode leg of the benchmark over pages
        {"name": "sparse_8x128k", "op": "sparse", "B": 8, "L": 131072, **heads32, "topk": 16,
         "kind": "bf16", "page": 128, "shape_seed": 0},
        # a mixed batch with few groups of many heads, small pages, E4M3 cache
        {"name": "sparse_16_ragged", "op": "sparse", "B": 16, "L": 40000, "H_q": 16, "H_kv": 2,
         "d": 128, "d_idx": 64, "topk": 16, "kind": "e4m3", "page": 16, "shape_seed": 14},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "cache", "dense", "sparse"])
    d = rng.choice([64, 128])
    d_idx = rng.choice([32, 64])
    H_kv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8, 16])
    while H_kv * G > 32:
        G //= 2
    case = {"op": op, "H_q": H_kv * G, "H_kv": H_kv, "d": d, "d_idx": d_idx}
    if op == "rope":
        B = rng.choice([0, 1, 2, 3])
        N = _log(rng, 1, 60000) // max(1, B) + 1
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        case |= {"B": B, "N": N, "rot": rng.choice([d_idx // 2, d_idx]),
                 "layout": rng.choice(["half", "interleaved"]),
                 "scaling": rng.choice(["none", "linear", "ntk", "yarn"]), "dtype": dtype,
                 "fused": rng.random() < 0.4, "grad": rng.random() < 0.6,
                 "far": rng.choice([0, 1000, 131072, 1048576])}
        return case
    case |= {"kind": rng.choice(["bf16", "e4m3"]), "page": rng.choice([16, 48, 64, 128, 256]),
             "shape_seed": rng.randrange(1, 1 << 20)}
    if op == "cache":
        mode = rng.choice(["write", "read", "both"])
        B = _log(rng, 1, 64)
        L = _log(rng, 1, 100000 // B + 1)
        new = 0 if mode == "read" else rng.choice([1, 1, L, max(1, L // 3)])
        return case | {"mode": mode if case["kind"] == "bf16" or mode != "write" else "both",
                       "B": B, "L": L, "new": new}
    B = _log(rng, 1, 64)
    L = _log(rng, 1, 400000 // B + 1)
    case |= {"B": B, "L": min(L, 131072)}
    if op == "sparse":
        case["topk"] = rng.choice([1, 4, 8, 16, 16, 20, 32])
    return case


def _lens(case):
    """Cache lengths of a case's sequences, the new token among them: all L where shape_seed is
    0, else spread over 1 .. L by their logarithm, with one full, one of a single token and
    (from 4 sequences on) one empty slot."""
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
_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _prepare_rope(case, g):
    dt = _DTYPES[case["dtype"]]
    lead = (case["N"],) if case["B"] == 0 else (case["B"], case["N"])
    rows = [(case["H_q"], case["d"]), (case["H_kv"], case["d"]), (case["H_kv"], case["d_idx"]),
            (1, case["d_idx"])]

    def tensors():
        if case["fused"]:  # one projection's output, the four operands its columns
            flat = torch.randn(*lead, sum(h * w for h, w in rows), generator=g, device="cuda",
                               dtype=torch.float32).to(dt)
            parts = torch.split(flat, [h * w for h, w in rows], dim=-1)
        else:
            parts = [torch.randn(*lead, h * w, generator=g, device="cuda", dtype=torch.float32).to(dt)
                     for h, w in rows]
        out = [p.unflatten(-1, r) for p, r in zip(parts, rows)]
        out[3] = out[3].squeeze(-2)  # k_idx has one head and no head axis
        return out

    xs = tensors()
    state = {"xs": xs}
    n = case["N"]
    if case["far"] or case["B"] == 0:  # tokens at any position, as a served batch has them
        state["positions"] = torch.randint(0, max(case["far"], n), lead, generator=g, device="cuda",
                                           dtype=torch.int32)
    else:
        state["positions"] = None
    if case["grad"]:
        state["dys"] = [torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float32).to(dt)
                        for x in xs]
    return state


def _prepare_pages(case, g):
    lens, page = _lens(case), case["page"]
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + 3  # a few pages that nobody holds
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["B"], (case["L"] + page - 1) // page), -1, dtype=torch.int32)
    order_host, at = order.cpu(), 0
    for b, n in enumerate(need):
        table[b, :n] = order_host[at:at + n]
        at += n
    shape = (pages, page, case["H_kv"], case["d"])

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    state = {"table": table.cuda(), "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
             "k_idx": randn(pages, page, case["d_idx"])}
    for n in ("k", "v"):
        if case["kind"] == "bf16":
            state[n] = randn(*shape)
        else:
            scale = torch.rand(shape[:3], generator=g, device="cuda") * 0.01 + 0.005
            codes = (torch.randn(shape, generator=g, device="cuda") * 100).clamp(-448, 448)
            state[n] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
            state[n + "_scale"] = scale
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "rope":
        state = _prepare_rope(case, g)
        if own:
            from block_sparse_gqa_topk_gb300 import ops
            state["rope"] = ops.new_rope(case["rot"], interleaved=case["layout"] == "interleaved",
                                         scaling=_base_scaling(case))
        for x in state["xs"]:
            x.requires_grad_(case["grad"])
        return {"case": case, **state}
    state = {"case": case, **_prepare_pages(case, g)}
    B, bf = case["B"], torch.bfloat16
    if case["op"] == "cache":
        counts = _lens(case) if case["mode"] == "read" else _news(case)
        T = sum(counts)
        state["total"] = T
        state["cu"] = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        if case["mode"] != "read":
            for n, s in (("new_k", (T, case["H_kv"], case["d"])), ("new_v", (T, case["H_kv"], case["d"])),
                         ("new_k_idx", (T, case["d_idx"]))):
                state[n] = torch.randn(*s, generator=g, device="cuda").to(bf)
    else:
        state["q"] = torch.randn(B, case["H_q"], case["d"], generator=g, device="cuda").to(bf)
        if case["op"] == "sparse":
            state["q_idx"] = torch.randn(B, case["H_kv"], case["d_idx"], generator=g, device="cuda").to(bf)
    if own:
        from block_sparse_gqa_topk_gb300 import ops
        state["cache"] = ops.PagedCache(state["k"], state["v"], state["k_idx"], state.get("k_scale"),
                                        state.get("v_scale"))
    return state


# ---------------------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, rot, interleaved, back):
    """x [.., d] rotated by cos, sin [.., rot / 2] in 32 bits, rounded once."""
    y = x.float()
    head, tail = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
    if back:
        sin = -sin
    a, b = a * cos - b * sin, b * cos + a * sin
    head = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((head, tail), -1).to(x.dtype)


def _plain_rope(s):
    case = s["case"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(case["N"], device="cuda").expand(case["B"], -1)
    freq, mul = _frequencies(case)
    angle = pos.double()[..., None] * freq
    cos, sin = (angle.cos() * mul).float(), (angle.sin() * mul).float()
    inter = case["layout"] == "interleaved"

    def turn(x, back):
        heads = x.dim() > cos.dim()
        return _rotate(x, cos.unsqueeze(-2) if heads else cos, sin.unsqueeze(-2) if heads else sin,
                       case["rot"], inter, back)

    with torch.no_grad():
        q, k, qi, ki = s["xs"]
        out = {"y": [turn(q, False), turn(k, False), turn(qi, False), turn(ki, False)]}
        if case["grad"]:
            q, k, qi, ki = s["dys"]
            out["dx"] = [turn(q, True), turn(k, True), turn(qi, True), turn(ki, True)]
    return out


def _rows(s):
    """Pool rows (page * page_size + offset) of the packed tokens of a cache call."""
    page, cu, lens = s["case"]["page"], s["cu"].long(), s["lens"].long()
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = lens[b] - (cu[b + 1] - t)
    return s["table"].long()[b, pos // page] * page + pos % page


def _plain_cache(s):
    case = s["case"]
    rows = _rows(s)
    f8 = case["kind"] == "e4m3"
    if case["mode"] != "read":
        s["k_idx"].flatten(0, 1)[rows] = s["new_k_idx"]
        if f8:
            xk, xv = s["new_k"].float(), s["new_v"].float()
            ak, av = xk.abs().amax(-1), xv.abs().amax(-1)
            most = torch.full((), 448.0, device="cuda")  # a number here would be a product with 1 / 448
            sk, sv = torch.where(ak > 0, ak / most, 1.0), torch.where(av > 0, av / most, 1.0)
            s["k"].flatten(0, 1)[rows] = (xk / sk[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            s["v"].flatten(0, 1)[rows] = (xv / sv[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            s["k_scale"].flatten(0, 1)[rows] = sk
            s["v_scale"].flatten(0, 1)[rows] = sv
        else:
            s["k"].flatten(0, 1)[rows] = s["new_k"]
            s["v"].flatten(0, 1)[rows] = s["new_v"]
    if case["mode"] == "write":
        return {"k": s["k"], "v": s["v"], "k_idx": s["k_idx"]}
    k, v = s["k"].flatten(0, 1)[rows], s["v"].flatten(0, 1)[rows]
    if f8:
        k = (k.view(torch.float8_e4m3fn).float() * s["k_scale"].flatten(0, 1)[rows][..., None]).bfloat16()
        v = (v.view(torch.float8_e4m3fn).float() * s["v_scale"].flatten(0, 1)[rows][..., None]).bfloat16()
    return {"k": k, "v": v, "k_idx": s["k_idx"].flatten(0, 1)[rows]}


def _gathered(s, name, rows):
    """Cache rows as 32-bit values."""
    x = s[name].flatten(0, 1)[rows]
    if s["case"]["kind"] == "e4m3" and name != "k_idx":
        return x.view(torch.float8_e4m3fn).float() * s[name + "_scale"].flatten(0, 1)[rows][..., None]
    return x.float()


def _softmax_join(scores, seen):
    """Weights of the seen scores and their log-sum-exp; none seen: no weight, -inf."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = (scores - top).exp()
    total = e.sum(-1, keepdim=True)
    w = e / torch.where(total > 0, total, 1.0)
    return w, (top + total.log()).squeeze(-1)


def _plain_dense(s):
    case = s["case"]
    B, H_kv, d, page = case["B"], case["H_kv"], case["d"], case["page"]
    G = case["H_q"] // H_kv
    pos = torch.arange(case["L"], device="cuda")
    seen = pos < s["lens"][:, None]
    rows = s["table"].long().clamp(min=0)[:, pos // page] * page + pos % page  # [B, L]
    q = s["q"].float().view(B, H_kv, G, d) / math.sqrt(d)
    k = _gathered(s, "k", rows).permute(0, 2, 3, 1)  # [B, H_kv, d, L]
    w, lse = _softmax_join(q @ k, seen[:, None, None, :])
    v = _gathered(s, "v", rows).permute(0, 2, 1, 3)  # [B, H_kv, L, d]
    o = w @ v
    return {"o": o.view(B, H_kv * G, d).bfloat16(), "lse": lse.view(B, H_kv * G)}


def _plain_sparse(s):
    case = s["case"]
    B, H_kv, d, page, topk = case["B"], case["H_kv"], case["d"], case["page"], case["topk"]
    G = case["H_q"] // H_kv
    nb = (case["L"] + BK - 1) // BK
    pos = torch.arange(nb * BK, device="cuda")
    table = s["table"].long().clamp(min=0)
    lens = s["lens"].long()
    page_of = (pos // page).clamp(max=table.shape[1] - 1)
    rows = table[:, page_of] * page + pos % page  # [B, nb * 128]
    # scores beside the border between taken and left blocks: 64 bits
    ki = s["k_idx"].flatten(0, 1)[rows].double()
    z = s["q_idx"].double() @ ki.transpose(1, 2)  # [B, H_kv, nb * 128]
    pooled = z.view(B, H_kv, nb, BK).amax(-1)
    block = torch.arange(nb, device="cuda")
    mine = ((lens - 1).clamp(min=0) // BK)[:, None, None]
    pooled = pooled.masked_fill(block >= mine, -math.inf)
    pooled = pooled.masked_fill((block == mine) & (lens[:, None, None] > 0), math.inf)
    value, index = pooled.sort(dim=-1, descending=True, stable=True)  # equal scores: lower block first
    value, index = value[..., :topk], index[..., :topk]
    index = torch.where(value > -math.inf, index, nb).sort(-1).values
    if nb < topk:
        index = torch.nn.functional.pad(index, (0, topk - nb), value=nb)
    chosen = torch.where(index < nb, index, -1)  # [B, H_kv, topk]
    at = (chosen.clamp(min=0)[..., None] * BK + torch.arange(BK, device="cuda")).flatten(-2)
    seen = (chosen >= 0).repeat_interleave(BK, -1) & (at < lens[:, None, None])
    batch = torch.arange(B, device="cuda")[:, None, None]
    head = torch.arange(H_kv, device="cuda")[None, :, None]
    at_page = (at // page).clamp(max=table.shape[1] - 1)
    cell = (table[batch, at_page] * page + at % page) * H_kv + head  # row of one head

    def selected(n):
        x = s[n].flatten(0, 2)[cell]
        if case["kind"] == "e4m3":
            return x.view(torch.float8_e4m3fn).float() * s[n + "_scale"].flatten()[cell][..., None]
        return x.float()

    q = s["q"].float().view(B, H_kv, G, d) / math.sqrt(d)
    w, lse = _softmax_join(q @ selected("k").transpose(-1, -2), seen[:, :, None, :])
    o = w @ selected("v")
    return {"block_idx": chosen.int(), "o": o.view(B, H_kv * G, d).bfloat16(),
            "lse": lse.view(B, H_kv * G)}


# ------------------------------------------------------------------------ the framework's
def _own_run(s):
    from block_sparse_gqa_topk_gb300 import ops
    case = s["case"]
    if case["op"] == "rope":
        if not case["grad"]:
            return {"y": list(ops.rope(s["xs"], s["rope"], s["positions"]))}
        y = ops.rope(s["xs"], s["rope"], s["positions"])
        dx = torch.autograd.grad(y, s["xs"], s["dys"])
        return {"y": [t.detach() for t in y], "dx": list(dx)}
    if case["op"] == "cache":
        if case["mode"] != "read":
            ops.msa_cache_write(s["cache"], s["table"], s["lens"], s["new_k"], s["new_v"], s["new_k_idx"],
                                cu_seqlens=s["cu"])
        if case["mode"] == "write":
            return {"k": s["k"], "v": s["v"], "k_idx": s["k_idx"]}
        k, v, k_idx = ops.msa_cache_read(s["cache"], s["table"], s["lens"], s["cu"], s["total"])
        return {"k": k, "v": v, "k_idx": k_idx}
    if case["op"] == "dense":
        o, lse = ops.msa_decode_paged_dense(s["q"], s["cache"], s["table"], s["lens"])
        return {"o": o, "lse": lse}
    block_idx, o, lse = ops.msa_decode_paged(s["q"], s["q_idx"], s["cache"], s["table"], s["lens"],
                                             case["topk"])
    return {"block_idx": block_idx, "o": o, "lse": lse}


def run(state):
    if own:
        return _own_run(state)
    return {"rope": _plain_rope, "cache": _plain_cache, "dense": _plain_dense,
            "sparse": _plain_sparse}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- 64-bit values
def _exact_rope(case, s):
    rot, half = case["rot"], case["rot"] // 2
    kind, factor = case["scaling"], 4.0
    base = 10000.0 * (factor ** (rot / (rot - 2.0)) if kind == "ntk" else 1.0)
    freqs, mul = [], 1.0
    for i in range(half):
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
    pos = s["positions"]
    lead = s["xs"][0].shape[:-2]
    if pos is None:
        pos = torch.arange(case["N"], device="cuda").repeat(case["B"], 1)
    # rows as complex numbers times exp(i angle); the gradient turns the other way
    unit = torch.polar(torch.full((), mul, dtype=torch.float64, device="cuda"),
                       pos.reshape(-1, 1).double() * w)

    def turned(x, sign):
        d = x.shape[-1]
        y = x.detach().double().reshape(unit.shape[0], -1, d).clone()
        if case["layout"] == "interleaved":
            z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2])
        else:
            z = torch.complex(y[..., :half], y[..., half:rot])
        z = z * (unit if sign > 0 else unit.conj())[:, None, :]
        if case["layout"] == "interleaved":
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            y[..., :half], y[..., half:rot] = z.real, z.imag
        return y.reshape(x.shape)

    assert tuple(lead) == tuple(pos.shape)
    out = {"y": [turned(x, 1) for x in s["xs"]]}
    if case["grad"]:
        out["dx"] = [turned(x, -1) for x in s["dys"]]
    return out


def _e4m3_value(codes):
    """Values of E4M3 codes from the format's fields."""
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
    return torch.where(c >= 128, -mag, mag)


def _e4m3_round(x):
    """The nearest E4M3 value (ties to even, at most 448) of each value of x (64 bits)."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(-6, 8)
    e = torch.where(torch.exp2(e) > a.clamp(min=2.0 ** -6), e - 1, e)
    step = torch.exp2(e - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def _sequence(s, b, n):
    """Pool rows of the first n tokens of sequence b, page after page."""
    page = s["case"]["page"]
    ids = s["table"][b, :(n + page - 1) // page].long()
    return (ids[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]


def _exact_cache(case, s):
    lens = _lens(case)
    counts = lens if case["mode"] == "read" else _news(case)
    out = {"k": [], "v": [], "k_idx": []}
    pool = {}
    if case["mode"] == "write":
        pool = {n: s[n].double().flatten(0, 1) for n in ("k", "v", "k_idx")}
    at = 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        rows = _sequence(s, b, n)[n - c:]
        for name in ("k", "v", "k_idx"):
            if case["mode"] == "read":
                x = s[name].flatten(0, 1)[rows]
                if case["kind"] == "e4m3" and name != "k_idx":
                    x = _e4m3_value(x) * s[name + "_scale"].flatten(0, 1)[rows].double()[..., None]
                x = x.double()
            else:
                x = s["new_" + name][at:at + c].double()
                if case["kind"] == "e4m3" and name != "k_idx":
                    top = x.abs().amax(-1, keepdim=True)
                    # a cached row's scale and the quotients that are coded have 32 bits by
                    # definition: in 64, ties between two codes would fall the other way
                    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top)).float().double()
                    x = _e4m3_round((x / scale).float().double()) * scale
            if case["mode"] == "write":
                pool[name][rows] = x
            else:
                out[name].append(x)
        at += c
    if case["mode"] == "write":
        return {n: p.view(s[n].shape) for n, p in pool.items()}
    return {n: torch.cat(p) for n, p in out.items()}


def _exact_attend(q, k, v):
    """Softmax attention of q [G, d] over k, v [n, d] (64 bits): values and log-sum-exp."""
    z = (q @ k.T) * (q.shape[-1] ** -0.5)
    lse = torch.logsumexp(z, -1)
    return torch.exp(z - lse[:, None]) @ v, lse


def _exact_decode(case, s):
    B, H_q, H_kv, d = case["B"], case["H_q"], case["H_kv"], case["d"]
    G = H_q // H_kv
    o = torch.zeros(B, H_q, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H_q), -math.inf, dtype=torch.float64, device="cuda")
    sets = torch.full((B, H_kv, case.get("topk", 1)), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        rows = _sequence(s, b, n)
        own_block = (n - 1) // BK
        if case["op"] == "sparse":
            z = s["q_idx"][b].double() @ s["k_idx"].flatten(0, 1)[rows[:own_block * BK]].double().T
            best = z.view(H_kv, own_block, BK).amax(-1) if own_block else z.new_zeros(H_kv, 0)
        for g in range(H_kv):
            use = rows
            if case["op"] == "sparse":
                take = sorted(torch.sort(best[g], dim=-1, descending=True, stable=True).indices[:case["topk"] - 1]
                              .tolist()) + [own_block]
                sets[b, g, :len(take)] = torch.tensor(take, dtype=torch.int32)
                use = torch.cat([rows[c * BK:(c + 1) * BK] for c in take])
            kv = []
            for name in ("k", "v"):
                x = s[name].flatten(0, 1)[use, g]
                if case["kind"] == "e4m3":
                    x = _e4m3_value(x) * s[name + "_scale"].flatten(0, 1)[use, g].double()[:, None]
                kv.append(x.double())
            h = slice(g * G, (g + 1) * G)
            o[b, h], lse[b, h] = _exact_attend(s["q"][b, h].double(), *kv)
    if case["op"] == "sparse":
        return {"block_idx": sets, "o": o, "lse": lse}
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "rope":
            return _exact_rope(case, s)
        if case["op"] == "cache":
            return _exact_cache(case, s)
        return _exact_decode(case, s)


# ----------------------------------------------------------------------------------- work
def work(case):
    H_q, H_kv, d, di = case["H_q"], case["H_kv"], case["d"], case["d_idx"]
    if case["op"] == "rope":
        n = max(1, case["B"]) * case["N"]
        passes = 2 if case["grad"] else 1
        size = 4 if case["dtype"] == "fp32" else 2
        row = (H_q + H_kv) * d + (H_kv + 1) * di
        given = case["far"] or case["B"] == 0
        return {"bytes": passes * n * (2 * row * size + (4 if given else 0)),
                "flops": passes * n * (H_q + 2 * H_kv + 1) * case["rot"] * 3}
    row = d * 2 if case["kind"] == "bf16" else d + 4  # one head's cached key or value
    lens = _lens(case)
    if case["op"] == "cache":
        total = sum(lens) if case["mode"] == "read" else sum(_news(case))
        cached, plain = 2 * H_kv * row + 2 * di, 2 * H_kv * 2 * d + 2 * di
        sides = 2 if case["mode"] == "both" else 1
        return {"bytes": sides * total * (cached + plain), "flops": sides * total * 2 * H_kv * d}
    G = H_q // H_kv
    small = case["B"] * (2 * H_q * d * 2 + H_q * 4)  # q, o and lse
    if case["op"] == "dense":
        tokens = H_kv * sum(lens)
        return {"bytes": tokens * 2 * row + small, "flops": tokens * G * 4 * d}
    keys = picked = 0
    for n in lens:
        if n:
            before = (n - 1) // BK
            keys += before * BK
            picked += min(case["topk"] - 1, before) * BK + n - before * BK
    return {"bytes": keys * di * 2 + picked * H_kv * 2 * row + small + case["B"] * H_kv * (di * 2 + case["topk"] * 4),
            "flops": keys * H_kv * 2 * di + picked * H_kv * G * 4 * d}
