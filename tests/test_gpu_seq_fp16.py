"""The range of fp16 in the operators over sequences: P and dS are rounded to it
before their products, so small ones must keep their bits wherever they make up
a result."""
import math

import pytest

import seq_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bl():
    from dynamic_block_sparse_tiled_b200 import build
    build.build()
    import dynamic_block_sparse_tiled_b200 as m
    return m


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def with_sink(g, q_lens, k_lens, hq, hkv, d, over, where):
    """fp16 q, k, v of packed sequences. One key of each (the first, or the last)
    scores `over` nats more than the others do on average; its value is 0."""
    import torch
    q, k, v = (torch.randn(sum(n), h, d, generator=g, device="cuda") for n, h in ((q_lens, hq), (k_lens, hkv), (k_lens, hkv)))
    v = 64 * (1 + 0.25 * v)
    q[..., 0] = 16.0
    k[..., 0] = 0.0
    for a, b in R.spans(k_lens):
        at = a if where == "first" else b - 1
        k[at] = 0.0
        k[at, :, 0] = over * math.sqrt(d) / 16
        v[at] = 0.0
    return q.half(), k.half(), v.half()


def check_sink(o, q, k, v, q_lens, k_lens, causal):
    """Element by element: P of a row, the reference 2^7 under its maximum, is off
    by 2^-11 of itself or 2^-25 (half a step of its subnormals) of 2^7, o by 2^-11
    of itself or 2^-25; scores by e (seq_ref).
    And on the whole: the model rounds P so and o, all else in 64 bits, and its
    error's norm is the kernel's expected one (a stream or range that does not see
    the strong key is nearer); 1.25 leaves eight times the spread of a norm over
    500 independent rows (3 %)."""
    import torch
    off = model = 0.0
    for (a, b), (c, e) in zip(R.spans(q_lens), R.spans(k_lens)):
        n, m, hq = b - a, e - c, q.shape[1]
        qq = q[a:b].double().transpose(0, 1)
        kk, vv = (R.heads(t[c:e], hq // k.shape[1]).transpose(0, 1) for t in (k, v))
        s = qq @ kk.transpose(1, 2) / math.sqrt(q.shape[2])
        if causal:
            s = s.masked_fill(torch.ones(n, m, dtype=torch.bool, device="cuda").triu(1 + m - n), -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        l = p.sum(-1, keepdim=True)
        want = p @ vv / l
        rounded = ((p * 128).half().double() / 128 @ vv / l).half().double()
        got = o[a:b].double().transpose(0, 1)
        err = q.shape[2] * 2.0 ** -23 * float((qq.abs() @ kk.abs().transpose(1, 2)).max()) / math.sqrt(q.shape[2]) + 2.0 ** -20
        bound = (2 * 2.0 ** -11 + 2 * err) * (p @ vv.abs()) / l + m * 2.0 ** -32 * float(vv.abs().max()) + 2.0 ** -25
        R.within(got, want, bound, "o")
        off += float((got - want).square().sum())
        model += float((rounded - want).square().sum())
    assert off <= 1.25 ** 2 * model, (off / model) ** 0.5


@pytest.mark.parametrize("over", [14, 16, 18, 20])
@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("d", [64, 128])
def test_small_weights_beside_a_strong_key(bl, over, where, d):
    """A key that outweighs all others and has no value of its own: o is made of the
    small weights. Few keys in all (whole items), and many (the shared list)."""
    g = gen(40)
    for q_lens, k_lens in (([150], [1000]), ([200, 33], [4096, 900])):
        q, k, v = with_sink(g, q_lens, k_lens, 4, 2, d, over, where)
        o, _ = bl.attention_packed(q, k, v, R.cu(q_lens), R.cu(k_lens), causal=False)
        assert bl.blasst_check() == 0
        check_sink(o, q, k, v, q_lens, k_lens, False)
    lens = [700, 129]
    q, k, v = with_sink(g, lens, lens, 4, 2, d, over, "first")
    o, _ = bl.attention_packed(q, k, v, R.cu(lens), causal=True)
    assert bl.blasst_check() == 0
    check_sink(o, q, k, v, lens, lens, True)


@pytest.mark.parametrize("over", [14, 18, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_small_weights_beside_a_strong_key_over_the_cache(bl, over, d):
    """The same for single tokens (the kernel for few rows), cut by ranges and not."""
    import torch
    g = gen(41)
    for kv_lens in ([300 + 7 * i for i in range(70)], [3000 + 11 * i for i in range(64)]):
        ones, n = [1] * len(kv_lens), sum(kv_lens)
        q, k, v = with_sink(g, ones, kv_lens, 8, 2, d, over, "first")
        page = 16
        need = [-(-m // page) for m in kv_lens]
        table = torch.full((len(ones), max(need)), -1, dtype=torch.int32, device="cuda")
        kp, vp = (torch.zeros(sum(need), page, 2, d, dtype=q.dtype, device="cuda") for _ in range(2))
        order, at = torch.randperm(sum(need), generator=g, device="cuda").int(), 0
        for s, ((a, b), c) in enumerate(zip(R.spans(kv_lens), need)):
            table[s, :c] = order[at:at + c]
            at += c
            j = torch.arange(b - a, device="cuda")
            kp[table[s].long()[j // page], j % page] = k[a:b]
            vp[table[s].long()[j // page], j % page] = v[a:b]
        lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
        o, _ = bl.attention_paged(q, kp, vp, table, lens, R.cu(ones))
        assert bl.blasst_check() == 0 and n == k.shape[0]
        check_sink(o, q, k, v, ones, kv_lens, True)


@pytest.mark.parametrize("step", [0.02, 0.2])
@pytest.mark.parametrize("rows", [300, 20, 1])
def test_references_that_move(bl, step, rows):
    """Scores that grow along the row, so that the softmax's reference moves in every
    block, in the kernel for few rows too (20 rows, 1 row)."""
    import torch
    g = gen(42)
    q, k, v = (torch.randn(n, h, 64, generator=g, device="cuda").half() for n, h in ((rows, 2), (600, 1), (600, 1)))
    q[..., 0] = 8.0
    k[..., 0] = (torch.arange(600, device="cuda") * step)[:, None].half()
    for causal in (False, True):
        got = bl.attention_packed(q, k, v, R.cu([rows]), R.cu([600]), causal=causal)
        assert bl.blasst_check() == 0
        R.check_packed(got, q, k, v, [rows], [600], causal)


# ---------------------------------------------------------------- gradients
def grads_fp16(q, k, v, o, lse, dout, causal):
    """One sequence's (dq, dk, dv) in 64 bits with their bounds, and with P and dS
    and the results rounded as fp16 has them.

    As in seq_ref, but what is under fp16's normal numbers is counted as it is:
    P is kept as 2^14 P, so it is off by 2^-11 of itself or 2^-39; dS as 2^k dS with
    2^14 / 2 < 2^k N <= 2^14 for N >= |dO| |v| (of the row for dQ, of all rows for
    dK; N is found to 2^-8), so it is off by 2^-11 of itself or 2^-25 2^-13 N; the
    results by 2^-11 of themselves or 2^-25."""
    import torch
    n, hq, d = q.shape
    m, hkv = k.shape[0], k.shape[1]
    g, scale = hq // hkv, 1 / math.sqrt(d)
    qq, oo, go = (t.double().transpose(0, 1) for t in (q, o, dout))
    kk, vv = (R.heads(t, g).transpose(0, 1) for t in (k, v))
    p = torch.exp(scale * qq @ kk.transpose(1, 2) - lse.double().t()[..., None])
    if causal:
        p = p.masked_fill(torch.ones(n, m, dtype=torch.bool, device="cuda").triu(1 + m - n), 0.0)
    ds = p * (go @ vv.transpose(1, 2) - (go * oo).sum(-1, keepdim=True))
    a_ds = p * (go.abs() @ vv.abs().transpose(1, 2) + (go * oo).abs().sum(-1, keepdim=True))
    e = d * 2.0 ** -23 * scale * float((qq.abs() @ kk.abs().transpose(1, 2)).max()) + 2.0 ** -20
    fold = lambda t: t.reshape(hkv, g, m, d).sum(1).transpose(0, 1)  # noqa: E731
    big = lambda t: t.norm(dim=-1)  # noqa: E731
    of_v = big(v.double()).amax(0).repeat_interleave(g)  # per query head
    of_do = big(go)                                      # [hq, n]
    of_do_all = of_do.amax(1).view(hkv, g).amax(1).repeat_interleave(g)
    row, key = 2.0 ** -38 * 1.01 * of_do * of_v[:, None], 2.0 ** -38 * 1.01 * of_do_all * of_v
    u = 2.0 ** -11
    want = [scale * (ds @ kk).transpose(0, 1), scale * fold(ds.transpose(1, 2) @ qq), fold(p.transpose(1, 2) @ go)]
    bound = [scale * ((2 * u + 4 * e) * (a_ds @ kk.abs()) + row[..., None] * kk.abs().sum(1, keepdim=True)).transpose(0, 1),
             scale * fold((2 * u + 4 * e) * (a_ds.transpose(1, 2) @ qq.abs()) + (key[:, None] * qq.abs().sum(1))[:, None]),
             fold((2 * u + 2 * e) * (p.transpose(1, 2) @ go.abs()) + 2.0 ** -39 * go.abs().sum(1, keepdim=True))]

    def kept(x, size):
        """x rounded as fp16 holds 2^k x, 2^14 / 2 < 2^k size <= 2^14."""
        k2 = torch.exp2(14 - torch.ceil(torch.log2(size.clamp(min=1e-300))))
        return (x * k2).half().double() / k2

    p16 = kept(p, torch.ones((), dtype=torch.float64, device="cuda"))
    dq16, dk16 = kept(ds, (of_do * of_v[:, None])[..., None]), kept(ds, (of_do_all * of_v)[:, None, None])
    # (what dS's roundings lose in a row is not in dQ: seen at its largest where keys have much in common)
    model = [scale * (dq16 @ kk).transpose(0, 1), scale * fold(dk16.transpose(1, 2) @ qq), fold(p16.transpose(1, 2) @ go)]
    return want, [b + 2.0 ** -25 for b in bound], [t.half().double() for t in model]


def check_fp16(got, q, k, v, o, lse, dout, q_lens, k_lens, causal, what=""):
    """Every element within its bound; and each sequence's errors, relative to the
    sums of |terms| of their token and head (a few large ones would hide the others;
    the gradient itself can cancel to less than the 32-bit roundings of dP and D,
    which the model leaves out), have the model's norm, with 1.25 for its spread."""
    import torch
    for i, ((a, b), (c, e)) in enumerate(zip(R.spans(q_lens), R.spans(k_lens))):
        want, bound, model = grads_fp16(q[a:b], k[c:e], v[c:e], o[a:b], lse[a:b], dout[a:b], causal)
        for name, t, (x, y), w, bd, md in zip(("dq", "dk", "dv"), got, ((a, b), (c, e), (c, e)), want, bound, model):
            R.within(t[x:y], w, bd, f"{what} sequence {i} {name}")
            size = (bd - 2.0 ** -25).norm(dim=-1, keepdim=True) * 2.0 ** 10
            size = torch.where(size == 0, 1.0, size)
            off, most = float(((t[x:y].double() - w) / size).norm()), float(((md - w) / size).norm())
            assert off <= 1.25 * most, f"{what} sequence {i} {name}: {off / most:.3g} times the model's error"


@pytest.mark.parametrize("over", [14, 16, 18])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_gradients_of_small_weights(bl, over, d, causal):
    """Values that only small weights touch: their gradients are sums of those."""
    import torch
    g = gen(43)
    lens = [1500, 700]
    q, k, v = with_sink(g, lens, lens, 4, 2, d, over, "first")
    dout = (256 * torch.randn(sum(lens), 4, d, generator=g, device="cuda")).half()
    cu = R.cu(lens)
    o, lse = bl.attention_packed(q, k, v, cu, causal=causal)
    got = bl.attention_packed_backward(q, k, v, o, lse, dout, cu, causal=causal)
    assert bl.blasst_check() == 0
    check_fp16(got, q, k, v, o, lse, dout, lens, lens, causal)


@pytest.mark.parametrize("d,hq,hkv,causal", [(64, 4, 2, True), (128, 3, 1, False), (128, 8, 2, True)])
@pytest.mark.parametrize("of", ["dout", "v", "both"])
def test_sequences_of_different_sizes(bl, d, hq, hkv, causal, of):
    """Sequences whose dO or v differ by up to 2^16 (a mean over many tokens beside
    one over few): each one's gradients are as near as alone, and the same bits."""
    import torch
    g = gen(44)
    q_lens, k_lens = [90, 0, 333, 1, 40, 129], [200, 77, 333, 60, 0, 300]
    if not causal:
        q_lens[0], k_lens[1] = 64, 0
    sizes = [2.0 ** -8, 1.0, 2.0 ** 8, 2.0 ** -7, 1.0, 2.0 ** 3]
    q, k, v = (torch.randn(sum(n), h, d, generator=g, device="cuda") for n, h in ((q_lens, hq), (k_lens, hkv), (k_lens, hkv)))
    dout = torch.randn(sum(q_lens), hq, d, generator=g, device="cuda")
    for (a, b), (c, e), x in zip(R.spans(q_lens), R.spans(k_lens), sizes):
        if of != "v":
            dout[a:b] *= x
        if of != "dout":
            v[c:e] *= min(x, 16.0)  # (dO v stays a number of fp16)
    q, k, v, dout = (t.half() for t in (q, k, v, dout))
    cq, ck = R.cu(q_lens), R.cu(k_lens)
    o, lse = bl.attention_packed(q, k, v, cq, ck, causal=causal)
    got = bl.attention_packed_backward(q, k, v, o, lse, dout, cq, ck, causal=causal)
    for i, ((a, b), (c, e)) in enumerate(zip(R.spans(q_lens), R.spans(k_lens))):
        if a == b or c == e:
            continue
        one = [q[a:b], k[c:e], v[c:e], o[a:b], lse[a:b].clone(), dout[a:b]]  # (lse lies on 16 bytes)
        check_fp16([t[x:y] for t, (x, y) in zip(got, ((a, b), (c, e), (c, e)))], *one, [b - a], [e - c], causal, f"{i}:")
        alone = bl.attention_packed_backward(*one, R.cu([b - a]), R.cu([e - c]), causal=causal)
        assert all(torch.equal(t[x:y], s) for t, (x, y), s in zip(got, ((a, b), (c, e), (c, e)), alone)), i
    assert bl.blasst_check() == 0


@pytest.mark.parametrize("some", [(3, 0, 1, 17, 2, 70), (1, 0, 1, 1, 2)])
def test_more_sequences_than_a_block_of_rows(bl, some):
    """Many short sequences, so that a block of the row pass holds rows of several, or
    of more than a warp has lanes."""
    import torch
    g = gen(45)
    lens = [some[i % len(some)] for i in range(150)]
    q, k, v, dout = (torch.randn(sum(lens), h, 64, generator=g, device="cuda") for h in (4, 2, 2, 4))
    for i, (a, b) in enumerate(R.spans(lens)):
        dout[a:b] *= 2.0 ** (i % 5 * 4 - 8)
        v[a:b] *= 2.0 ** (i % 3 - 1)
    q, k, v, dout = (t.half() for t in (q, k, v, dout))
    cu = R.cu(lens)
    o, lse = bl.attention_packed(q, k, v, cu)
    got = bl.attention_packed_backward(q, k, v, o, lse, dout, cu)
    for a, b in [x for x in R.spans(lens) if x[0] < x[1]]:
        want, bound, _ = grads_fp16(q[a:b], k[a:b], v[a:b], o[a:b], lse[a:b], dout[a:b], True)
        for t, w, bd in zip(got, want, bound):
            R.within(t[a:b], w, bd, f"tokens {a}-{b}")
    for a, b in R.spans(lens)[3:12]:
        alone = bl.attention_packed_backward(q[a:b], k[a:b], v[a:b], o[a:b], lse[a:b], dout[a:b], R.cu([b - a]))
        assert all(torch.equal(t[a:b], s) for t, s in zip(got, alone))
    assert bl.blasst_check() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_different_sizes(bl, d):
    """Rows of dO that are 2^16 smaller than others of their sequence: their dQ is as
    near as the others'."""
    import torch
    g = gen(46)
    lens = [500, 260]
    q, k, v, dout = (torch.randn(sum(lens), h, d, generator=g, device="cuda") for h in (4, 2, 2, 4))
    dout *= torch.exp2(torch.randint(-8, 9, (sum(lens), 4, 1), generator=g, device="cuda").float())
    q, k, v, dout = (t.half() for t in (q, k, v, dout))
    cu = R.cu(lens)
    o, lse = bl.attention_packed(q, k, v, cu)
    got = bl.attention_packed_backward(q, k, v, o, lse, dout, cu)
    check_fp16(got, q, k, v, o, lse, dout, lens, lens, True)
    assert bl.blasst_check() == 0


def test_a_sequence_that_is_not_finite(bl):
    """Infinities and NaN in one sequence's dO and v leave the others' bits alone."""
    import torch
    g = gen(47)
    lens = [70, 150, 30]
    q, k, v, dout = (torch.randn(sum(lens), h, 64, generator=g, device="cuda").half() for h in (4, 2, 2, 4))
    cu = R.cu(lens)

    def grads():
        o, lse = bl.attention_packed(q, k, v, cu)
        return bl.attention_packed_backward(q, k, v, o, lse, dout, cu)

    want = grads()
    dout[100, 1, 5], dout[101, 0, 0], v[90, 0, 3], v[200, 1, 2] = math.inf, math.nan, math.nan, -math.inf
    got = grads()
    for own in (slice(0, 70), slice(220, 250)):
        assert all(torch.equal(a[own], b[own]) for a, b in zip(got, want))
    assert bl.blasst_check() == 0
