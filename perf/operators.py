"""The sequence operators as a user's program calls them, and in plain torch.

Four operators that stand next to the dense attention of this package and are
used together: the rotary position embedding (forward and backward), the write
of new tokens into a paged KV cache (rotating q and k on the way), attention
over prompts packed one behind the other (forward and backward), and attention
of a chunk of new tokens, or of single ones, over the paged cache.

Layouts: packed tokens are [T, heads, d]; sequence s owns the tokens
cu[s] .. cu[s+1]-1. A paged cache is [pages, page, kv_heads, d] and a table
[sequences, most pages] of page numbers (-1 where a sequence has no page).
Causal masks are bottom-right aligned: the last query sees every key.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEVICE = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a training step's or a long prompt's queries: 32 heads, positions far beyond the trained
        # length, frequencies blended for a longer context
        {"name": "rotary prompt", "op": "rotary", "tokens": 32768, "heads": 32, "d": 128, "rot": 128,
         "interleaved": False, "dtype": "bf16", "stretch": 8.0, "first": 98304},
        # a small odd batch of a model that turns half of each head, pairs side by side
        {"name": "rotary partial", "op": "rotary", "tokens": 777, "heads": 5, "d": 64, "rot": 32,
         "interleaved": True, "dtype": "fp16", "stretch": 1.0, "first": 0},
        # the gradient of a training step's queries, kept in 32 bits
        {"name": "rotary gradient", "op": "rotary_grad", "tokens": 8192, "heads": 32, "d": 128, "rot": 128,
         "interleaved": False, "dtype": "fp32", "stretch": 1.0, "first": 0},
        # one decode step of 16 requests: their new token goes into the cache
        {"name": "append decode", "op": "append", "q_lens": "1*16", "kv_lens": "1024*4+700*6+97*6",
         "heads": 32, "kv_heads": 8, "d": 128, "rot": 128, "interleaved": False, "page": 64, "dtype": "bf16"},
        # a prefill step that mixes a long chunk, an odd one and a single token
        {"name": "append chunk", "op": "append", "q_lens": "2048+511+1", "kv_lens": "4096+511+900",
         "heads": 32, "kv_heads": 8, "d": 128, "rot": 64, "interleaved": True, "page": 16, "dtype": "fp16"},
        # a handful of short prompts in one call: latency
        {"name": "packed short", "op": "packed", "q_lens": "1+17+64+129+300", "k_lens": "", "heads": 4,
         "kv_heads": 2, "d": 64, "causal": True, "dtype": "fp16"},
        # long prompts of different lengths, 32768 tokens in all
        {"name": "packed prompts", "op": "packed", "q_lens": "16384+9001+5120+2263", "k_lens": "", "heads": 32,
         "kv_heads": 8, "d": 128, "causal": True, "dtype": "bf16"},
        # gradients between two short packed sides of different lengths, three query heads to a key head
        {"name": "packed gradient short", "op": "packed_grad", "q_lens": "33+200+1+77", "k_lens": "150+128+65+12",
         "heads": 6, "kv_heads": 2, "d": 64, "causal": False, "dtype": "fp16"},
        # a training step's gradients over packed documents
        {"name": "packed gradient", "op": "packed_grad", "q_lens": "8192+4097+2048+1270+777", "k_lens": "",
         "heads": 32, "kv_heads": 8, "d": 128, "causal": True, "dtype": "bf16"},
        # one decode step of 16 requests with 65536 cached tokens each
        {"name": "paged decode", "op": "paged", "q_lens": "1*16", "kv_lens": "65536*16", "heads": 32,
         "kv_heads": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # one decode step of three short requests: latency
        {"name": "paged decode short", "op": "paged", "q_lens": "1*3", "kv_lens": "700+1+4097", "heads": 16,
         "kv_heads": 2, "d": 64, "page": 16, "dtype": "fp16"},
        # a serving step: a long prompt's next chunk, a short prompt, a few drafted tokens, single tokens
        {"name": "paged mixed", "op": "paged", "q_lens": "2048+513+8+1*12", "kv_lens": "30000+513+4099+8192*6+1500*6",
         "heads": 32, "kv_heads": 8, "d": 128, "page": 32, "dtype": "bf16"},
    ]


def _log(rng, low, high):
    """A whole number spread over the logarithm of [low, high]."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    return kv * rng.choice([1, 2, 3, 4, 5, 8]), kv


def _lens(rng, n, low, high, most):
    out, left = [], most
    for _ in range(n):
        v = _log(rng, low, max(low, min(high, left)))
        out.append(v)
        left = max(low, left - v)
    return out


def draw(rng):
    op = rng.choice(["rotary", "rotary_grad", "append", "packed", "packed_grad", "paged", "packed", "paged"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    heads, kv = _heads(rng)
    if op in ("rotary", "rotary_grad"):
        heads = rng.randint(1, 32)
        d = rng.choice([64, 80, 96, 128, 256])
        return {"op": op, "tokens": _log(rng, 1, min(32768, 32768 * 32 * 128 // (heads * d))), "heads": heads, "d": d,
                "rot": rng.choice([d, d // 2, d // 4]), "interleaved": rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "stretch": rng.choice([1.0, 4.0, 16.0]),
                "first": rng.choice([0, rng.randint(1, 1000000)])}
    if op == "append":
        q = _lens(rng, rng.randint(1, 20), 1, 2048, 4096)
        k = [v + (0 if rng.random() < 0.3 else _log(rng, 1, 2000)) for v in q]
        return {"op": op, "q_lens": "+".join(map(str, q)), "kv_lens": "+".join(map(str, k)), "heads": heads,
                "kv_heads": kv, "d": d, "rot": rng.choice([d, d // 2]), "interleaved": rng.random() < 0.5,
                "page": rng.choice([16, 32, 64, 128]), "dtype": dtype}
    if op == "packed":
        q = _lens(rng, rng.randint(1, 12), 1, 12000, 16000)
        return {"op": op, "q_lens": "+".join(map(str, q)), "k_lens": "", "heads": heads, "kv_heads": kv, "d": d,
                "causal": rng.random() < 0.8, "dtype": dtype}
    if op == "packed_grad":
        q = _lens(rng, rng.randint(1, 8), 1, 5000, 8000)
        k = [v + _log(rng, 1, 1000) for v in q] if rng.random() < 0.4 else q
        return {"op": op, "q_lens": "+".join(map(str, q)), "k_lens": "+".join(map(str, k)) if k != q else "",
                "heads": heads, "kv_heads": kv, "d": d, "causal": rng.random() < 0.7, "dtype": dtype}
    n = rng.randint(1, 24)
    q = [1] * n if rng.random() < 0.5 else [_log(rng, 1, 1500) if rng.random() < 0.4 else 1 for _ in range(n)]
    k = [v + (0 if rng.random() < 0.1 else _log(rng, 1, 30000)) for v in q]
    return {"op": op, "q_lens": "+".join(map(str, q)), "kv_lens": "+".join(map(str, k)), "heads": heads,
            "kv_heads": kv, "d": d, "page": rng.choice([16, 32, 64, 128, 256]), "dtype": dtype}


def _numbers(text):
    """"3+5*2" is [3, 5, 5]."""
    parts = [p.split("*") for p in text.split("+")]
    return [int(p[0]) for p in parts for _ in range(int(p[1]) if len(p) > 1 else 1)]


# --------------------------------------------------------------- inputs
def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEVICE)


def _rows(gen, n, heads, d, dtype):
    """Projected activations: unit variance around a mean of each channel's own."""
    mean = 0.5 * torch.randn(1, heads, d, generator=gen, device=DEVICE)
    return (torch.randn(n, heads, d, generator=gen, device=DEVICE) + mean).to(DTYPES[dtype])


def _frequencies(rot, stretch):
    """Angle a position adds to each pair, 64 bits: base 10000, and for a context `stretch` times as long the slow pairs
    slowed by it, the fast ones kept, a straight line between (over the pairs that turn 1 to 32 times in 8192 tokens)."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEVICE)
    freq = 10000.0 ** (-2.0 * i / rot)
    if stretch == 1.0:
        return freq, 1.0
    turns = 8192.0 * freq / (2.0 * math.pi)
    kept = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return freq * kept + freq / stretch * (1.0 - kept), 0.1 * math.log(stretch) + 1.0


def _pages(gen, case, kv_lens):
    """A cache whose pages lie in no order, the table of each sequence, and three pages nobody owns."""
    page = case["page"]
    need = [-(-n // page) for n in kv_lens]
    total = sum(need) + 3
    shape = (total, page, case["kv_heads"], case["d"])
    dtype = DTYPES[case["dtype"]]
    k = torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.bfloat16).to(dtype)
    k += (0.5 * torch.randn(1, 1, *shape[2:], generator=gen, device=DEVICE)).to(dtype)
    v = torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.bfloat16).to(dtype)
    order = torch.randperm(total, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.full((len(need), max(need) + 1), -1, dtype=torch.int32, device=DEVICE)
    start = 0
    for s, n in enumerate(need):
        table[s, :n] = order[start:start + n]
        start += n
    return k, v, table


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("rotary", "rotary_grad"):
        s["x"] = _rows(gen, case["tokens"], case["heads"], case["d"], case["dtype"])
        s["positions"] = case["first"] + torch.arange(case["tokens"], dtype=torch.int64, device=DEVICE)
        s["freq"], s["mscale"] = _frequencies(case["rot"], case["stretch"])
        return s
    q_lens = _numbers(case["q_lens"])
    k_lens = _numbers(case.get("kv_lens") or case.get("k_lens") or case["q_lens"])
    total = sum(q_lens)
    s |= {"q_lens": q_lens, "k_lens": k_lens, "cu_q": _cu(q_lens)}
    s["q"] = _rows(gen, total, case["heads"], case["d"], case["dtype"])
    if op in ("append", "paged"):
        s["k_pages"], s["v_pages"], s["table"] = _pages(gen, case, k_lens)
        s["kv_lens"] = torch.tensor(k_lens, dtype=torch.int32, device=DEVICE)
    if op == "append":
        s["k"] = _rows(gen, total, case["kv_heads"], case["d"], case["dtype"])
        s["v"] = _rows(gen, total, case["kv_heads"], case["d"], case["dtype"])
        s["freq"], s["mscale"] = _frequencies(case["rot"], 1.0)
        owner = torch.repeat_interleave(torch.arange(len(q_lens), device=DEVICE), torch.tensor(q_lens, device=DEVICE))
        s["owner"] = owner
    if op in ("packed", "packed_grad"):
        s["cu_k"] = _cu(k_lens)
        s["k"] = _rows(gen, sum(k_lens), case["kv_heads"], case["d"], case["dtype"])
        s["v"] = _rows(gen, sum(k_lens), case["kv_heads"], case["d"], case["dtype"])
    if op == "packed_grad":
        s["o"], s["lse"] = _packed(s)
        s["dout"] = torch.randn(total, case["heads"], case["d"], generator=gen, device=DEVICE).to(DTYPES[case["dtype"]])
    return s


# ---------------------------------------------------------- plain forms
def _turn(x, positions, freq, mscale, interleaved, back=False):
    """x [T, heads, d] turned by its tokens' positions; `back`: the transposed turn, which is the gradient's."""
    rot = 2 * freq.numel()
    angle = positions.double()[:, None] * freq[None, :]
    cos = (angle.cos() * mscale).float()[:, None, :]
    sin = (angle.sin() * (-mscale if back else mscale)).float()[:, None, :]
    y = x.float().clone()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    first, second = a * cos - b * sin, a * sin + b * cos
    a.copy_(first)
    b.copy_(second)
    return y.to(x.dtype)


def _append(s):
    case = s["case"]
    token = torch.arange(s["q"].shape[0], device=DEVICE)
    new = s["cu_q"][1:] - s["cu_q"][:-1]
    position = token - s["cu_q"][s["owner"]] + (s["kv_lens"] - new)[s["owner"]]
    turn = (position, s["freq"], s["mscale"], case["interleaved"])
    page = s["table"][s["owner"], position // case["page"]].long()
    slot = position % case["page"]
    s["k_pages"][page, slot] = _turn(s["k"], *turn)
    s["v_pages"][page, slot] = s["v"]
    return _turn(s["q"], *turn), s["k_pages"], s["v_pages"]


def _chunks(rows, per_row):
    """Row ranges of a score matrix that fit into about 4 GB of 32-bit scores."""
    step = max(1, min(rows, (1 << 30) // max(1, per_row)))
    return [(r, min(rows, r + step)) for r in range(0, rows, step)]


def _attend(q, k, v, causal):
    """Attention of one sequence: q [n, Hq, d], k, v [m, Hkv, d]; o in q's type, lse [n, Hq]."""
    n, heads, d = q.shape
    m, kv = k.shape[0], k.shape[1]
    kt, vt = k.float().permute(1, 2, 0), v.float().transpose(0, 1)
    o = torch.zeros_like(q)
    lse = torch.full((n, heads), -math.inf, device=q.device)
    for r0, r1 in _chunks(n, heads * m):
        seen = min(m, r1 + m - n) if causal else m
        if seen <= 0:
            continue
        rows = q[r0:r1].float().reshape(r1 - r0, kv, heads // kv, d).permute(1, 2, 0, 3).reshape(kv, -1, d)
        x = torch.matmul(rows * (1.0 / math.sqrt(d)), kt[:, :, :seen]).view(kv, heads // kv, r1 - r0, seen)
        if causal:
            last = torch.arange(r0, r1, device=q.device) + (m - n)
            x.masked_fill_(torch.arange(seen, device=q.device)[None, :] > last[:, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
        total = x.sum(-1, keepdim=True)
        y = torch.matmul(x.view(kv, -1, seen), vt[:, :seen]).view(kv, heads // kv, r1 - r0, d)
        y = torch.where(total > 0, y / total, 0.0)
        o[r0:r1] = y.permute(2, 0, 1, 3).reshape(r1 - r0, heads, d).to(q.dtype)
        lse[r0:r1] = (top + total.log()).permute(2, 0, 1, 3).reshape(r1 - r0, heads)
    return o, lse


def _spans(lens):
    start = 0
    for n in lens:
        yield start, start + n
        start += n


def _packed(s):
    parts = [_attend(s["q"][a:b], s["k"][c:e], s["v"][c:e], s["case"]["causal"])
             for (a, b), (c, e) in zip(_spans(s["q_lens"]), _spans(s["k_lens"]))]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def _attend_grad(q, k, v, o, lse, dout, causal):
    n, heads, d = q.shape
    m, kv = k.shape[0], k.shape[1]
    scale = 1.0 / math.sqrt(d)
    group = heads // kv
    kt, vt = k.float().transpose(0, 1), v.float().transpose(0, 1)
    dq = torch.zeros_like(q)
    dk, dv = torch.zeros_like(kt), torch.zeros_like(vt)
    by_head = lambda t: t.float().reshape(t.shape[0], kv, group, -1).permute(1, 2, 0, 3).reshape(kv, group * t.shape[0], -1)  # noqa: E731
    for r0, r1 in _chunks(n, heads * m):
        seen = min(m, r1 + m - n) if causal else m
        if seen <= 0:
            continue
        rows, grad = by_head(q[r0:r1]), by_head(dout[r0:r1])
        x = torch.matmul(rows * scale, kt[:, :seen].transpose(1, 2))
        x = x.sub_(by_head(lse[r0:r1])).exp_()
        if causal:
            last = (torch.arange(r0, r1, device=q.device) + (m - n)).repeat(group)
            x.masked_fill_(torch.arange(seen, device=q.device)[None, :] > last[:, None], 0.0)
        dv[:, :seen] += torch.matmul(x.transpose(1, 2), grad)
        ds = torch.matmul(grad, vt[:, :seen].transpose(1, 2))
        ds = ds.sub_((grad * by_head(o[r0:r1])).sum(-1, keepdim=True)).mul_(x).mul_(scale)
        dk[:, :seen] += torch.matmul(ds.transpose(1, 2), rows)
        dq[r0:r1] = torch.matmul(ds, kt[:, :seen]).view(kv, group, r1 - r0, d).permute(2, 0, 1, 3).reshape(r1 - r0, heads, d).to(q.dtype)
    return dq, dk.transpose(0, 1).to(k.dtype), dv.transpose(0, 1).to(v.dtype)


def _packed_grad(s):
    parts = [_attend_grad(s["q"][a:b], s["k"][c:e], s["v"][c:e], s["o"][a:b], s["lse"][a:b], s["dout"][a:b], s["case"]["causal"])
             for (a, b), (c, e) in zip(_spans(s["q_lens"]), _spans(s["k_lens"]))]
    return tuple(torch.cat([p[i] for p in parts]) for i in range(3))


def _cached(pages, table, i, n):
    """The first n cached rows of sequence i, [n, Hkv, d]."""
    page = pages.shape[1]
    return pages[table[i, :-(-n // page)].long()].flatten(0, 1)[:n]


def _paged(s):
    parts = [_attend(s["q"][a:b], _cached(s["k_pages"], s["table"], i, n), _cached(s["v_pages"], s["table"], i, n), True)
             for i, ((a, b), n) in enumerate(zip(_spans(s["q_lens"]), s["k_lens"]))]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import dynamic_block_sparse_tiled_b200 as bl
        if op == "rotary":
            return bl.rotary(s["x"], s["freq"], s["positions"], interleaved=case["interleaved"], mscale=s["mscale"])
        if op == "rotary_grad":
            return bl.rotary_backward(s["x"], s["freq"], s["positions"], interleaved=case["interleaved"], mscale=s["mscale"])
        if op == "append":
            q = bl.paged_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"], s["cu_q"],
                                inv_freq=s["freq"], interleaved=case["interleaved"], mscale=s["mscale"])
            return q, s["k_pages"], s["v_pages"]
        if op == "packed":
            return bl.attention_packed(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=case["causal"])
        if op == "packed_grad":
            return bl.attention_packed_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"], s["cu_q"], s["cu_k"],
                                                causal=case["causal"])
        return bl.attention_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"], s["cu_q"])
    if op in ("rotary", "rotary_grad"):
        return _turn(s["x"], s["positions"], s["freq"], s["mscale"], case["interleaved"], back=op == "rotary_grad")
    return {"append": _append, "packed": _packed, "packed_grad": _packed_grad, "paged": _paged}[op](s)


# ------------------------------------------------- what a pass has to do
def _pairs(q_lens, k_lens, causal):
    """(query, key) pairs that the mask leaves."""
    total = 0
    for n, m in zip(q_lens, k_lens):
        if not causal:
            total += n * m
        else:
            first = max(1, m - n + 1)  # keys the first query with any sees
            total += (first + m) * (m - first + 1) // 2
    return total


def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op in ("rotary", "rotary_grad"):
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["d"] * size + 8 * case["tokens"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    q_lens = _numbers(case["q_lens"])
    k_lens = _numbers(case.get("kv_lens") or case.get("k_lens") or case["q_lens"])
    d, hq, hk, t, tk = case["d"], case["heads"], case["kv_heads"], sum(q_lens), sum(k_lens)
    index = 8 * len(q_lens)
    if op == "append":
        pages = 4 * sum(-(-k // case["page"]) - (k - n) // case["page"] for n, k in zip(q_lens, k_lens))
        return {"bytes": 2 * t * (hq + 2 * hk) * d * size + index + pages + 4 * case["rot"], "flops": 3 * t * (hq + hk) * case["rot"]}
    if op == "packed":
        return {"bytes": (2 * t * hq + 2 * tk * hk) * d * size + 4 * t * hq + index,
                "flops": 4 * d * hq * _pairs(q_lens, k_lens, case["causal"])}
    if op == "packed_grad":
        return {"bytes": (4 * t * hq + 4 * tk * hk) * d * size + 4 * t * hq + index,
                "flops": 10 * d * hq * _pairs(q_lens, k_lens, case["causal"])}
    pages = 4 * sum(-(-k // case["page"]) for k in k_lens)
    return {"bytes": (2 * t * hq + 2 * tk * hk) * d * size + 4 * t * hq + index + pages,
            "flops": 4 * d * hq * _pairs(q_lens, k_lens, True)}


# ------------------------------------------- from the definition, 64 bits
def _turn_exact(x, positions, freq, mscale, interleaved, sign):
    rot = 2 * freq.numel()
    wide = x.double()
    part = wide[..., :rot]
    pair = part.unflatten(-1, (rot // 2, 2)) if interleaved else torch.stack(part.split(rot // 2, -1), -1)
    angle = sign * positions.double()[:, None, None] * freq
    turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * torch.polar(torch.full_like(angle, mscale), angle))
    turned = turned.flatten(-2) if interleaved else torch.cat([turned[..., 0], turned[..., 1]], -1)
    return torch.cat([turned, wide[..., rot:]], -1)


def _score_exact(q, k, n, m, causal, rows):
    """Scores of one head's query rows, 64 bits, and the pairs that count."""
    x = torch.einsum("id,jd->ij", q.double(), k.double()) / math.sqrt(q.shape[-1])
    at = torch.arange(*rows, device=q.device)[:, None] + (m - n)
    seen = torch.arange(m, device=q.device)[None, :] <= at if causal else torch.ones_like(x, dtype=torch.bool)
    return x, seen


def _blocks(n, m):
    step = max(1, (1 << 28) // max(1, m))
    return [(r, min(n, r + step)) for r in range(0, n, step)]


def _attend_exact(q, k, v, causal):
    n, heads, d = q.shape
    m = k.shape[0]
    group = heads // k.shape[1]
    o = torch.zeros(n, heads, d, dtype=torch.float64, device=q.device)
    lse = torch.full((n, heads), -math.inf, dtype=torch.float64, device=q.device)
    for h in range(heads):
        for a, b in _blocks(n, m):
            x, seen = _score_exact(q[a:b, h], k[:, h // group], n, m, causal, (a, b))
            x = torch.where(seen, x, -math.inf)
            lse[a:b, h] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[a:b, h].nan_to_num(neginf=0.0)[:, None])
            o[a:b, h] = torch.einsum("ij,jd->id", p, v[:, h // group].double())
    return o, lse


def _grad_exact(q, k, v, o, lse, dout, causal):
    n, heads, d = q.shape
    m, group = k.shape[0], heads // k.shape[1]
    dq = torch.zeros(n, heads, d, dtype=torch.float64, device=q.device)
    dk = torch.zeros(m, k.shape[1], d, dtype=torch.float64, device=q.device)
    dv = torch.zeros_like(dk)
    for h in range(heads):
        kh, vh = k[:, h // group].double(), v[:, h // group].double()
        for a, b in _blocks(n, m):
            x, seen = _score_exact(q[a:b, h], kh, n, m, causal, (a, b))
            p = torch.where(seen, torch.exp(x - lse[a:b, h].double()[:, None]), 0.0)
            g = dout[a:b, h].double()
            dv[:, h // group] += torch.einsum("ij,id->jd", p, g)
            ds = p * (torch.einsum("id,jd->ij", g, vh) - torch.einsum("id,id->i", g, o[a:b, h].double())[:, None]) / math.sqrt(d)
            dq[a:b, h] = torch.einsum("ij,jd->id", ds, kh)
            dk[:, h // group] += torch.einsum("ij,id->jd", ds, q[a:b, h].double())
    return dq, dk, dv


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rotary", "rotary_grad"):
        return _turn_exact(s["x"], s["positions"], s["freq"], s["mscale"], case["interleaved"], -1 if op == "rotary_grad" else 1)
    spans = list(_spans(s["q_lens"]))
    if op == "append":
        q = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
        pages = [s["k_pages"].double(), s["v_pages"].double()]
        for i, ((a, b), n) in enumerate(zip(spans, s["k_lens"])):
            at = torch.arange(n - (b - a), n, device=DEVICE)
            q[a:b] = _turn_exact(s["q"][a:b], at, s["freq"], s["mscale"], case["interleaved"], 1)
            where = (s["table"][i].long()[at // case["page"]], at % case["page"])
            pages[0][where] = _turn_exact(s["k"][a:b], at, s["freq"], s["mscale"], case["interleaved"], 1)
            pages[1][where] = s["v"][a:b].double()
        return q, pages[0], pages[1]
    parts = []
    start = 0
    for i, ((a, b), n) in enumerate(zip(spans, s["k_lens"])):
        if op == "paged":
            k, v = (_cached(s[name], s["table"], i, n) for name in ("k_pages", "v_pages"))
        else:
            k, v = s["k"][start:start + n], s["v"][start:start + n]
        start += n
        if op == "packed_grad":
            parts.append(_grad_exact(s["q"][a:b], k, v, s["o"][a:b], s["lse"][a:b], s["dout"][a:b], case["causal"]))
        else:
            parts.append(_attend_exact(s["q"][a:b], k, v, case.get("causal", True)))
    return tuple(torch.cat([p[i] for p in parts]) for i in range(len(parts[0])))
