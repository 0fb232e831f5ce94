"""Attention over sequences where a resident grid takes whole items from a list: what
long prompts and batches of many short ones run through. Each case asserts that
it gets there."""
import math

import pytest

import seq_ref as R

pytestmark = pytest.mark.gpu

TYPES = ["bfloat16", "float16"]


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


def by_list(tokens, n_seq, hq, hkv, most_keys):
    """(the list is used, by the kernel for few rows): the host's rule, from the sizes
    of a call alone. Places: full items and one per sequence; whole items where full
    ones fill the SMs eight times or no sequence can have over 1024 keys; the list
    where their places are more than two per SM."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    g = hq // hkv
    few = g <= 32 and tokens * g <= 32 * n_seq
    full = tokens // (128 // g * (1 if few else 2))
    whole = full * hkv >= 8 * sms or most_keys <= 1024
    return whole and (full + n_seq) * hkv > 2 * sms, few


def qkv(g, q_lens, k_lens, hq, hkv, d, dtype):
    import torch
    return [(torch.randn(sum(n), h, d, generator=g, device="cuda") + m).to(getattr(torch, dtype))
            for n, h, m in ((q_lens, hq, 0.0), (k_lens, hkv, 0.3), (k_lens, hkv, -0.2))]


# (name, lengths of q, of the keys, heads, key heads, kernel for few rows)
PACKED = [
    ("one or two tokens, few keys", [i % 3 for i in range(400)], [(5 * i) % 6 for i in range(400)], 4, 2, True),
    ("one or two tokens and some of 70, few keys", [70 if i % 97 == 5 else 1 + i % 2 for i in range(300)], [i % 7 for i in range(300)], 4, 2, True),
    ("many rows per token, few keys", [51] * 20, [51 if i % 3 else (0, 20, 102)[i // 3 % 3] for i in range(20)], 64, 4, False),
    ("prompts", [300, 17, 0, 333, 256, 1, 700, 129] * 11, None, 16, 2, False),
    ("prompts of other lengths than their keys", [300, 17, 0, 333, 256, 1, 700, 129] * 11, [100, 60, 9, 500, 0, 40, 701, 128] * 11, 16, 2, False),
    ("prompts of one head each", [1200, 130, 1, 257] * 24, None, 8, 8, False),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", PACKED, ids=[c[0] for c in PACKED])
def test_packed(bl, dtype, d, causal, case):
    import torch
    name, q_lens, k_lens, hq, hkv, few = case
    k_lens = q_lens if k_lens is None else k_lens
    assert by_list(sum(q_lens), len(q_lens), hq, hkv, sum(k_lens)) == (True, few)
    g = gen(60)
    q, k, v = qkv(g, q_lens, k_lens, hq, hkv, d, dtype)
    cq, ck = R.cu(q_lens), R.cu(k_lens)
    got = bl.attention_packed(q, k, v, cq, ck, causal=causal)
    assert bl.blasst_check() == 0
    R.check_packed(got, q, k, v, q_lens, k_lens, causal)
    # the same bits whoever takes which item, from a workspace that holds anything
    ws = torch.full((bl.blasst_seq_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        again = bl.attention_packed(q, k, v, cq, ck, causal=causal, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(again, got))
    assert bl.blasst_check() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,d,page,few", [
    # single tokens of large groups over caches of very different lengths
    ([1] * 600, [1 + (37 * i) % 90 + (i % 97 == 5) * 1500 for i in range(600)], 256, 8, 64, 16, True),
    # single tokens, two tokens and none, short caches
    ([(1, 1, 2, 0)[i % 4] for i in range(500)], [2 + (29 * i) % 200 for i in range(500)], 8, 4, 128, 8, True),
    # chunks beside single tokens
    ([600, 1, 1, 333, 1, 40] * 20, [900, 700, 3, 1500, 129, 40] * 20, 16, 2, 128, 32, False),
    ([600, 1, 1, 333, 1, 40] * 20, [900, 700, 3, 1500, 129, 40] * 20, 16, 2, 64, 64, False),
])
@pytest.mark.parametrize("causal", [True, False])
def test_paged(bl, dtype, q_lens, kv_lens, hq, hkv, d, page, few, causal):
    import torch
    g = gen(61)
    kp, vp, table, rows = R.paged(kv_lens, page, hkv, d, getattr(torch, dtype), g)
    assert by_list(sum(q_lens), len(q_lens), hq, hkv, table.shape[1] * page) == (True, few)
    q = torch.randn(sum(q_lens), hq, d, generator=g, device="cuda").to(kp.dtype)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    got = bl.attention_paged(q, kp, vp, table, lens, R.cu(q_lens), causal=causal)
    assert bl.blasst_check() == 0
    k, v = (torch.cat([r[i] for r in rows]) for i in range(2))
    R.check_packed(got, q, k, v, q_lens, kv_lens, causal)
    again = bl.attention_paged(q, kp, vp, table, lens, R.cu(q_lens), causal=causal)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("few", [True, False])
def test_replayed_with_other_lengths(bl, dtype, few):
    """A captured call: the list is cleared by every replay, and follows the lengths."""
    import torch
    g = gen(62)
    n, total, hq, hkv, d = (400, 500, 4, 2, 64) if few else (40, 20000, 16, 2, 64)
    keys = 900 if few else total
    assert by_list(total, n, hq, hkv, keys) == (True, few)

    def lens(seed, whole):
        cuts = torch.randint(0, whole + 1, (n - 1,), generator=gen(seed), device="cuda").sort()[0].tolist()
        return [b - a for a, b in zip([0, *cuts], [*cuts, whole])]

    q, k, v = qkv(g, [total], [keys], hq, hkv, d, dtype)
    cq, ck = R.cu(lens(1, total)), R.cu(lens(2, keys))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        bl.attention_packed(q, k, v, cq, ck)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = bl.attention_packed(q, k, v, cq, ck)
    for seed in (1, 3, 5):
        q_lens, k_lens = lens(seed, total), lens(seed + 1, keys)
        cq.copy_(R.cu(q_lens))
        ck.copy_(R.cu(k_lens))
        for t in got:
            t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        R.check_packed(got, q, k, v, q_lens, k_lens, True, what=f"seed {seed}")
    assert bl.blasst_check() == 0


def test_two_streams_at_once(bl):
    """Two calls at the same time, each with a list of its own."""
    import torch
    q_lens = [300, 17, 0, 333, 256, 1, 700, 129] * 11
    g = gen(63)
    sets = [qkv(g, q_lens, q_lens, 16, 2, 64, "bfloat16") for _ in range(2)]
    cu = R.cu(q_lens)
    want = [bl.attention_packed(*s, cu) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(bl.attention_packed(*sets[i], cu))
    torch.cuda.synchronize()
    for w, calls in zip(want, got):
        for c in calls:
            assert all(torch.equal(a, b) for a, b in zip(c, w))
    assert bl.blasst_check() == 0
