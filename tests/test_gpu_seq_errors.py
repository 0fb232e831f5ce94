"""Index errors of the operators over sequences concern the sequences that have
them: other calls made before blasst_check compute, and a wait that gives up is
reported all the same."""
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


def bad_page(bl, g):
    """An attention call over the cache whose table names a page that is not there."""
    import torch
    kp, vp, table, _ = R.paged([100], 16, 2, 64, torch.bfloat16, g)
    table[0, 1] = kp.shape[0]
    q = torch.randn(1, 4, 64, generator=g, device="cuda").bfloat16()
    bl.attention_paged(q, kp, vp, table, torch.tensor([100], dtype=torch.int32, device="cuda"), R.cu([1]))


def dense(q, k, v):
    """[B, H, L, d] causal attention in 64 bits."""
    import torch
    q, k, v = (t.double() for t in (q, k, v))
    s = q @ k.repeat_interleave(q.shape[1] // k.shape[1], 1).transpose(2, 3) / math.sqrt(q.shape[-1])
    n, m = s.shape[-2:]
    s = s.masked_fill(torch.ones(n, m, dtype=torch.bool, device="cuda").triu(1 + m - n), -math.inf)
    return s.softmax(-1) @ v.repeat_interleave(q.shape[1] // v.shape[1], 1)


def test_dense_calls_after_an_index_error(bl):
    """The prefill, the split decode and the backward compute what they compute
    without the error, bit for bit (dQ is added by several CTAs in any order: up to
    300 fp32 terms, 2^-24 each of sums that cancel to a sixteenth at most)."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    q, k, v, dout = (torch.randn(1, h, 300, 128, generator=g, device="cuda").bfloat16() for h in (4, 2, 2, 4))
    one = q[:, :, -1:].contiguous()

    def calls():
        o, lse, _ = bl.attention_prefill(q, k, v)
        return [o, lse, *bl.attention_decode(one, k, v)[:2], *bl.attention_backward(q, k, v, o, lse, dout)]

    want = calls()
    assert bl.blasst_check() == 0
    # every P, then o rounded once to bf16 (eps / 2 each), and the two exponentials' 1.1e-4
    assert float((want[0].double() - dense(q, k, v)).abs().max()) <= (2 * 2.0 ** -8 + 2.2e-4) * float(v.abs().max())
    bad_page(bl, g)
    got = calls()
    assert bl.blasst_check() == bl.BLASST_EINDEX
    assert bl.blasst_check() == 0
    for i, (a, b) in enumerate(zip(got, want)):
        if i == 4:
            assert float((a.double() - b.double()).norm()) <= 16 * 300 * 2.0 ** -24 * float(b.double().norm())
        else:
            assert torch.equal(a, b), i


def test_calls_over_sequences_after_an_index_error(bl):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(32)
    lens = [70, 200]
    q, k, v = (torch.randn(270, h, 64, generator=g, device="cuda").bfloat16() for h in (4, 2, 2))
    bad_page(bl, g)
    got = bl.attention_packed(q, k, v, R.cu(lens))
    assert bl.blasst_check() == bl.BLASST_EINDEX
    R.check_packed(got, q, k, v, lens, lens, True)


@pytest.mark.parametrize("first", ["index", "wait"])
def test_a_wait_that_gives_up_is_not_hidden(bl, first):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(33)
    if first == "index":
        bad_page(bl, g)
    bl.blasst_selftest_timeout(1_000_000)  # 1 ms
    if first == "wait":
        # (calls after the wait do nothing; their index errors change nothing)
        bad_page(bl, g)
    assert bl.blasst_check() == bl.BLASST_ETIMEOUT
    assert bl.blasst_check() == 0
