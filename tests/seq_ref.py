"""The operators over sequences of different lengths in 64 bits, for the tests.

Tolerances. u = eps / 2 of the inputs' type bounds one rounding. With S the
32-bit scores, their error is at most d 2^-23 times A_s = scale |q|.|k| (the sum
of a score's terms), so every P carries a relative error e = d 2^-23 max A_s +
2^-20 (the exponential and the 32-bit sums), far under u.
  o      P is rounded once and o once: |err| <= (2 u + 2 e) sum_j p |v|, plus
         n 2^-25 max|v| for fp16 P below its normal numbers (the sum is >= 1);
  lse    e + 2^-23 |lse|;
  dv     P and dv rounded once: (2 u + 2 e) sum_i P |dO|;
  dk, dq dS and the result rounded once: (2 u + 4 e) times the same sums over
         scale P (|dO|.|v| + |dO|.|o|) |q| (or |k|), which count the terms of
         dP - D also where the difference cancels;
each plus the smallest number of the type, where a result is subnormal.
"""
import math

import torch


def spans(lens):
    out, at = [], 0
    for n in lens:
        out.append((at, at + n))
        at += n
    return out


def cu(lens, first=0, device="cuda"):
    return torch.tensor([first + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=device)


def turn(x, positions, freq, mscale=1.0, interleaved=False, inverse=False):
    """x [..., T, H, d] turned by positions [T], in 64 bits."""
    rot = 2 * freq.numel()
    a = positions.double()[:, None] * freq
    c, s = (a.cos() * mscale)[:, None, :], (a.sin() * (-mscale if inverse else mscale))[:, None, :]
    y = x.double().clone()
    p, q = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, w = p * c - q * s, p * s + q * c
    p.copy_(u)
    q.copy_(w)
    return y


def heads(t, g):
    """Key heads repeated for their query heads."""
    return t.double().repeat_interleave(g, dim=1)


def attend(q, k, v, causal, scale=None):
    """One sequence: (o, lse, bound of o, bound of lse); n x m scores per head."""
    n, hq, d = q.shape
    m, g = k.shape[0], hq // k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    u = torch.finfo(q.dtype).eps / 2 if q.dtype != torch.float64 else 0.0
    if m == 0:
        z = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
        return z, torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device), z, z[..., 0]
    qq, kk, vv = q.double().transpose(0, 1), heads(k, g).transpose(0, 1), heads(v, g).transpose(0, 1)
    s = scale * qq @ kk.transpose(1, 2)
    if causal:
        hidden = torch.arange(m, device=q.device)[None, :] > torch.arange(n, device=q.device)[:, None] + (m - n)
        s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    e = d * 2.0 ** -23 * scale * float((qq.abs() @ kk.abs().transpose(1, 2)).max()) + 2.0 ** -20
    o = p @ vv
    b_o = (2 * u + 2 * e) * (p @ vv.abs()) + m * 2.0 ** -25 * float(vv.abs().max()) + torch.finfo(q.dtype).tiny
    b_l = e + 2.0 ** -23 * torch.where(lse == -math.inf, 0.0, lse).abs()
    return o.transpose(0, 1), lse.t(), b_o.transpose(0, 1), b_l.t()


def grads(q, k, v, o, lse, dout, causal, scale=None):
    """One sequence: (dq, dk, dv) and their bounds."""
    n, hq, d = q.shape
    m, hkv = k.shape[0], k.shape[1]
    g = hq // hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    u = torch.finfo(q.dtype).eps / 2
    if n == 0 or m == 0:
        r = [torch.zeros(t.shape, dtype=torch.float64, device=q.device) for t in (q, k, v)]
        return r, r
    qq, kk, vv = q.double().transpose(0, 1), heads(k, g).transpose(0, 1), heads(v, g).transpose(0, 1)
    oo, go = o.double().transpose(0, 1), dout.double().transpose(0, 1)
    p = torch.exp(scale * qq @ kk.transpose(1, 2) - lse.double().t()[..., None])
    seen = torch.ones(n, m, dtype=torch.bool, device=q.device)
    if causal:
        seen = torch.arange(m, device=q.device)[None, :] <= torch.arange(n, device=q.device)[:, None] + (m - n)
    p = torch.where(seen, p, 0.0)
    ds = scale * p * (go @ vv.transpose(1, 2) - (go * oo).sum(-1, keepdim=True))
    a_ds = scale * p * (go.abs() @ vv.abs().transpose(1, 2) + (go * oo).abs().sum(-1, keepdim=True))
    e = d * 2.0 ** -23 * scale * float((qq.abs() @ kk.abs().transpose(1, 2)).max()) + 2.0 ** -20
    fold = lambda t: t.reshape(hkv, g, m, d).sum(1).transpose(0, 1)  # noqa: E731
    tiny = torch.finfo(q.dtype).tiny
    r = [(ds @ kk).transpose(0, 1), fold(ds.transpose(1, 2) @ qq), fold(p.transpose(1, 2) @ go)]
    b = [(2 * u + 4 * e) * (a_ds @ kk.abs()).transpose(0, 1) + tiny,
         (2 * u + 4 * e) * fold(a_ds.transpose(1, 2) @ qq.abs()) + tiny,
         (2 * u + 2 * e) * fold(p.transpose(1, 2) @ go.abs()) + tiny]
    return r, b


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)  # NaN is bad
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst {float((err / bound)[bad].max()):.3g} x, "
        f"first {[int(i) for i in bad.nonzero()[0]]}: {float(got[bad][0])} for {float(want[bad][0])}")


def check_packed(got, q, k, v, q_lens, k_lens, causal, scale=None, what=""):
    o, lse = got
    for i, ((a, b), (c, e)) in enumerate(zip(spans(q_lens), spans(k_lens))):
        if a == b:
            continue
        ro, rl, bo, bl_ = attend(q[a:b], k[c:e], v[c:e], causal, scale)
        empty = rl == -math.inf
        assert bool((lse[a:b].double()[empty] == -math.inf).all()), f"{what} sequence {i}: lse of empty rows"
        assert bool((o[a:b][empty] == 0).all()), f"{what} sequence {i}: o of empty rows"
        within(o[a:b], ro, bo, f"{what} sequence {i} o")
        within(lse[a:b][~empty], rl[~empty], bl_[~empty], f"{what} sequence {i} lse")


def check_grads(got, q, k, v, o, lse, dout, q_lens, k_lens, causal, scale=None, what=""):
    for i, ((a, b), (c, e)) in enumerate(zip(spans(q_lens), spans(k_lens))):
        r, bd = grads(q[a:b], k[c:e], v[c:e], o[a:b], lse[a:b], dout[a:b], causal, scale)
        for name, t, (x, y), want, bound in zip(("dq", "dk", "dv"), got, ((a, b), (c, e), (c, e)), r, bd):
            if x < y:
                within(t[x:y], want, bound, f"{what} sequence {i} {name}")


def paged(kv_lens, page, hkv, d, dtype, gen, head_major=False, spare=3):
    """A cache whose pages lie in no order and whose unowned rows are NaN, its
    table (-1 behind a sequence's pages), and each sequence's keys and values."""
    need = [-(-n // page) for n in kv_lens]
    total = sum(need) + spare
    shape = (total, hkv, page, d) if head_major else (total, page, hkv, d)
    pools = []
    for _ in range(2):
        t = torch.full(shape, math.nan, dtype=dtype, device="cuda")
        pools.append(t.transpose(1, 2) if head_major else t)
    order = torch.randperm(total, generator=gen, device="cuda").int()
    table = torch.full((len(kv_lens), max(need + [0]) + 2), -1, dtype=torch.int32, device="cuda")
    rows, at = [], 0
    for s, (n, c) in enumerate(zip(kv_lens, need)):
        table[s, :c] = order[at:at + c]
        at += c
        kv = [torch.randn(n, hkv, d, generator=gen, device="cuda").to(dtype) for _ in range(2)]
        j = torch.arange(n, device="cuda")
        for pool, t in zip(pools, kv):
            pool[table[s].long()[j // page], j % page] = t
        rows.append(kv)
    return pools[0], pools[1], table, rows
