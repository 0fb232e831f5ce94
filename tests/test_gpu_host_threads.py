"""Calls from host threads that have made no CUDA call before, as autograd's and a
server's workers: the device's context is bound when a call needs it."""
import threading

import pytest

import seq_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bl():
    from dynamic_block_sparse_tiled_b200 import build
    build.build()
    import dynamic_block_sparse_tiled_b200 as m
    return m


def in_thread(f):
    """f() in a new thread; its result, or its exception."""
    got = []

    def run():
        try:
            got.append((f(), None))
        except Exception as e:  # noqa: BLE001
            got.append((None, e))

    t = threading.Thread(target=run)
    t.start()
    t.join(60)
    value, error = got[0]
    if error is not None:
        raise error
    return value


@pytest.mark.parametrize("name", ["prefill", "prefill fp32", "decode", "mla", "backward", "select", "packed",
                                  "packed backward", "paged", "append", "rotary"])
def test_first_call_of_a_thread(bl, name):
    """The same bits from a new thread as from this one (the dense dQ, added by several
    CTAs in any order, to its rounding)."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(70)
    r = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    q, k, v, dout = r(1, 4, 300, 128), r(1, 2, 300, 128), r(1, 2, 300, 128), r(1, 4, 300, 128)
    o, lse, _ = bl.attention_prefill(q, k, v)
    lens = [100, 200]
    cu = R.cu(lens)
    x, y, z, w = r(300, 4, 128), r(300, 2, 128), r(300, 2, 128), r(300, 4, 128)
    po, pl = bl.attention_packed(x, y, z, cu)
    kp, vp, table, _ = R.paged([100, 200], 16, 2, 128, torch.bfloat16, g)
    kv = torch.tensor([100, 200], dtype=torch.int32, device="cuda")
    two = R.cu([1, 1])
    freq, _ = bl.rope_frequencies(128)
    f32 = [r(1, 2, 200, 64, dtype=torch.float32) for _ in range(3)]
    mq, mc = r(1, 128, 576), r(1, 500, 576)
    call = {"prefill": lambda: bl.attention_prefill(q, k, v)[:2],
            "prefill fp32": lambda: bl.attention_prefill(*f32, Bc=64)[:2],
            "decode": lambda: bl.attention_decode(q[:, :, :1].contiguous(), k, v)[:2],
            "mla": lambda: bl.attention_decode_mla(mq, mc)[:2],
            "backward": lambda: bl.attention_backward(q, k, v, o, lse, dout),
            "select": lambda: bl.select_blocks(q, k),
            "packed": lambda: bl.attention_packed(x, y, z, cu),
            "packed backward": lambda: bl.attention_packed_backward(x, y, z, po, pl, w, cu),
            "paged": lambda: bl.attention_paged(x[:2], kp, vp, table, kv, two),
            "append": lambda: (bl.paged_append(x[:2], y[:2], z[:2], kp, vp, table, kv, two, inv_freq=freq),),
            "rotary": lambda: (bl.rotary(x, freq),)}[name]
    want = call()
    assert bl.blasst_check() == 0
    stream = torch.cuda.current_stream()
    torch.cuda.synchronize()

    def work():
        with torch.cuda.stream(stream):
            return call()

    got = in_thread(work)
    assert in_thread(bl.blasst_check) == 0
    for i, (a, b) in enumerate(zip(got, want)):
        if name == "backward" and i == 0:
            assert float((a - b).norm()) <= 16 * 300 * 2.0 ** -24 * float(b.norm())
        else:
            assert torch.equal(a, b), i


def test_threads_at_once(bl):
    """Several threads, each with a stream of its own, beginning together."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(71)
    lens = [100, 333, 7]
    q, k, v, dout = (torch.randn(440, h, 64, generator=g, device="cuda").half() for h in (4, 2, 2, 4))
    cu = R.cu(lens)
    o, lse = bl.attention_packed(q, k, v, cu)
    want = (o, lse, *bl.attention_packed_backward(q, k, v, o, lse, dout, cu))
    torch.cuda.synchronize()
    start, got = threading.Barrier(6, timeout=60), [None] * 6

    def run(i):
        start.wait()
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                a, b = bl.attention_packed(q, k, v, cu)
                got[i] = (a, b, *bl.attention_packed_backward(q, k, v, a, b, dout, cu))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    for result in got:
        assert result is not None and all(torch.equal(a, b) for a, b in zip(result, want))
    assert bl.blasst_check() == 0
