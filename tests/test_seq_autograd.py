"""The operators over sequences beside autograd: a gradient that is asked for is
recorded by a function around the calls, or refused; never lost without a word."""
import math

import pytest

import seq_ref as R


@pytest.fixture(scope="module")
def bl():
    from dynamic_block_sparse_tiled_b200 import build
    build.build()
    import dynamic_block_sparse_tiled_b200 as m
    return m


def calls(bl, x, f, cu, pool, table, lse):
    return {"rotary": lambda: bl.rotary(x, f), "rotary_backward": lambda: bl.rotary_backward(x, f),
            "packed": lambda: bl.attention_packed(x, x, x, cu),
            "packed_backward": lambda: bl.attention_packed_backward(x, x, x, x, lse, x, cu),
            "paged": lambda: bl.attention_paged(x, pool, pool, table, cu[1:], cu),
            "append": lambda: bl.paged_append(x, x, x, pool, pool, table, cu[1:], cu)}


def inputs(bl, device):
    import torch
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=device)
    f, _ = bl.rope_frequencies(64, device=device)
    cu = torch.tensor([0, 3], dtype=torch.int32, device=device)
    pool = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=device)
    return x, f, cu, pool, torch.zeros(1, 2, dtype=torch.int32, device=device), torch.zeros(3, 2, device=device)


@pytest.mark.parametrize("name", ["rotary", "rotary_backward", "packed", "packed_backward", "paged", "append"])
def test_refused_before_anything_else(bl, name):
    import torch
    x, *rest = inputs(bl, "cpu")
    x.requires_grad_()
    with pytest.raises(ValueError, match="requires a gradient"):
        calls(bl, x, *rest)[name]()
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):
        calls(bl, x, *rest)[name]()


@pytest.mark.gpu
def test_refused_on_any_argument(bl):
    import torch
    x, f, cu, pool, table, lse = inputs(bl, "cuda")
    y = torch.zeros_like(x).requires_grad_()
    page = torch.zeros_like(pool).requires_grad_()
    wanted = [lambda: bl.rotary(x, f, out=y), lambda: bl.rotary(y * 1, f), lambda: bl.attention_packed(x, y, x, cu),
              lambda: bl.attention_packed(x, x, y * 2, cu), lambda: bl.attention_packed_backward(x, x, x, x, lse, y, cu),
              lambda: bl.attention_packed_backward(x, x, x, x, lse.clone().requires_grad_(), x, cu),
              lambda: bl.attention_paged(x, page, pool, table, cu[1:], cu),
              lambda: bl.paged_append(x, y, x, pool, pool, table, cu[1:], cu),
              lambda: bl.paged_append(x, x, x, pool, pool, table, cu[1:], cu, q_out=y)]
    for call in wanted:
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad():
            call()
    for call in calls(bl, x, f, cu, pool, table, lse).values():  # none asks for a gradient
        call()
    assert bl.blasst_check() == 0


@pytest.mark.gpu
def test_a_function_around_the_calls(bl):
    """rotary and packed attention in one autograd function; its gradients against
    64-bit autograd of the formula."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(51)
    lens, hq, hkv, d = [90, 30], 4, 2, 64
    freq, _ = bl.rope_frequencies(d)
    cu, pos = R.cu(lens), torch.cat([torch.arange(n, device="cuda") for n in lens])

    class Attention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v):
            tq, tk = bl.rotary(q, freq, pos), bl.rotary(k, freq, pos)
            o, lse = bl.attention_packed(tq, tk, v, cu)
            ctx.save_for_backward(tq, tk, v, o, lse)
            return o

        @staticmethod
        def backward(ctx, dout):
            dq, dk, dv = bl.attention_packed_backward(*ctx.saved_tensors, dout.contiguous(), cu)
            return bl.rotary_backward(dq, freq, pos), bl.rotary_backward(dk, freq, pos), dv

    leaf = [torch.randn(120, h, d, generator=g, device="cuda").bfloat16().requires_grad_() for h in (hq, hkv, hkv)]
    dout = torch.randn(120, hq, d, generator=g, device="cuda").bfloat16()
    Attention.apply(*leaf).backward(dout)
    wide = [t.detach().double().requires_grad_() for t in leaf]
    a = pos.double()[:, None] * freq

    def turn(x):
        p, r = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([p * a.cos()[:, None] - r * a.sin()[:, None], p * a.sin()[:, None] + r * a.cos()[:, None]], -1)

    loss = 0.0
    for x, y in R.spans(lens):
        s = turn(wide[0])[x:y].transpose(0, 1) @ turn(wide[1])[x:y].repeat_interleave(2, 1).transpose(0, 1).transpose(1, 2)
        s = (s / math.sqrt(d)).masked_fill(torch.ones(y - x, y - x, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        loss = loss + (s.softmax(-1) @ wide[2][x:y].repeat_interleave(2, 1).transpose(0, 1) * dout[x:y].double().transpose(0, 1)).sum()
    loss.backward()
    # four bf16 roundings in a row (turned inputs, P or dS, the gradient before and behind the turn), each at
    # most u of the sums of their terms; norm-wise against the gradient's own norm twice that
    for t, w in zip(leaf, wide):
        assert float((t.grad.double() - w.grad).norm()) <= 8 * 2.0 ** -8 * float(w.grad.norm())
    assert bl.blasst_check() == 0
