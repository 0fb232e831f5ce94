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
