"""The operators over sequences of different lengths against their definitions in
64 bits (tests/seq_ref.py, which derives the bounds)."""
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


def rand(g, *shape, dtype, mean=0.0):
    import torch
    return (torch.randn(*shape, generator=g, device="cuda") + mean).to(getattr(torch, dtype) if isinstance(dtype, str) else dtype)


def qkv(seed, q_lens, k_lens, hq, hkv, d, dtype):
    g = gen(seed)
    return (rand(g, sum(q_lens), hq, d, dtype=dtype), rand(g, sum(k_lens), hkv, d, dtype=dtype, mean=0.3),
            rand(g, sum(k_lens), hkv, d, dtype=dtype, mean=-0.2), g)


# ------------------------------------------------------------------- rotary
@pytest.mark.parametrize("dtype", TYPES + ["float32"])
@pytest.mark.parametrize("tokens,heads,d,rot", [(1, 1, 2, 2), (3, 5, 64, 64), (37, 3, 80, 20), (130, 8, 128, 128),
                                                (700, 32, 128, 64), (9, 2, 1024, 1000), (5, 7, 33, 6)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(bl, dtype, tokens, heads, d, rot, interleaved, inverse):
    import torch
    g = gen(1)
    x = rand(g, tokens, heads, d, dtype=dtype)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda")
    freq, m = bl.rope_frequencies(rot, scaling="linear", factor=3.0)
    call = bl.rotary_backward if inverse else bl.rotary
    y = call(x, freq, pos, interleaved=interleaved, mscale=1.25)
    want = R.turn(x, pos, freq, 1.25, interleaved, inverse)
    # one rounding; sine and cosine of an angle reduced in 64 bits: its rounding to 32 bits (2^-24 of up to
    # pi), their own error (2 units) and the two products
    u = torch.finfo(x.dtype).eps / 2
    size = 1.25 * x.double().abs().amax() * math.sqrt(2)
    R.within(y, want, (u * want.abs() + size * 2.0 ** -21 + torch.finfo(x.dtype).tiny), "rotary")
    assert torch.equal(y[..., rot:], x[..., rot:])
    assert bl.blasst_check() == 0


def test_rotary_layouts_in_place_positions(bl):
    import torch
    g = gen(2)
    freq, _ = bl.rope_frequencies(64)
    x = rand(g, 2, 6, 50, 64, dtype="bfloat16")  # [B, H, L, d]
    flat = lambda t, b: t[b].transpose(0, 1)  # noqa: E731
    # no positions: 0, 1, ...; one row for all; a row each
    rows = torch.randint(0, 5000, (2, 50), generator=g, device="cuda", dtype=torch.int32)
    for pos, of in ((None, lambda b: torch.arange(50, device="cuda")), (rows[0], lambda b: rows[0]), (rows, lambda b: rows[b]),
                    (rows.long(), lambda b: rows[b])):
        y = bl.rotary(x, freq, pos)
        for b in range(2):
            want = bl.rotary(flat(x, b).contiguous(), freq, of(b).long())
            assert torch.equal(flat(y, b), want)
    # strided input (every second head, an odd token offset), given output, in place
    wide = rand(g, 61, 12, 72, dtype="float16")
    view = wide[5:, ::2, 3:67]
    want = bl.rotary(view.contiguous(), freq)
    assert torch.equal(bl.rotary(view, freq), want)
    out = torch.zeros(56, 6, 80, dtype=torch.float16, device="cuda")
    got = bl.rotary(view, freq, out=out[..., 8:72])
    assert torch.equal(got, want) and bool((out[..., :8] == 0).all()) and bool((out[..., 72:] == 0).all())
    before = wide.clone()
    bl.rotary(view, freq, out=view)
    assert torch.equal(view, want)
    before[5:, ::2, 3:67] = want
    assert torch.equal(wide, before)
    # there and back
    z = rand(g, 100, 4, 64, dtype="float32")
    pos = torch.arange(100, device="cuda") + 70000
    assert float((bl.rotary_backward(bl.rotary(z, freq, pos), freq, pos) - z).abs().max()) < 2e-5
    assert bl.rotary(z[:0], freq).shape == (0, 4, 64)
    assert bl.blasst_check() == 0


def test_rotary_refusals(bl):
    import torch
    freq, _ = bl.rope_frequencies(64)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: bl.rotary(x.double(), freq), lambda: bl.rotary(x, freq.float()), lambda: bl.rotary(x[0], freq),
                lambda: bl.rotary(x.transpose(1, 2), freq), lambda: bl.rotary(x, freq, torch.arange(3, device="cuda")),
                lambda: bl.rotary(x, freq, torch.arange(4, device="cuda").float()), lambda: bl.rotary(x, freq.cpu()),
                lambda: bl.rotary(x, freq, out=x[:3]), lambda: bl.rotary(x, freq, torch.arange(4))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(bl.BlasstError):
        bl.rotary(x[..., :62], freq)  # rot > d
    with pytest.raises(bl.BlasstError):
        bl.rotary(x, freq, mscale=0.0)


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", TYPES + ["float32"])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,d,rot,page,interleaved,head_major", [
    ([1], [1], 1, 1, 64, 64, 16, False, False),
    ([1] * 9, [5, 16, 17, 64, 1, 33, 200, 128, 129], 8, 2, 128, 128, 16, False, True),
    ([40, 0, 7, 300], [40, 12, 100, 431], 5, 5, 64, 32, 64, True, False),
    ([3, 70], [90, 71], 4, 1, 80, 20, 7, True, True),
    ([2] * 300, [3 + (5 * i) % 60 for i in range(300)], 2, 1, 64, 64, 8, False, False),
    ([12, 5], [12, 30], 3, 3, 33, 6, 5, False, False),
])
def test_append(bl, dtype, q_lens, kv_lens, hq, hkv, d, rot, page, interleaved, head_major):
    import torch
    g = gen(3)
    dt = getattr(torch, dtype)
    kp, vp, table, rows = R.paged(kv_lens, page, hkv, d, dt, g, head_major)
    T = sum(q_lens)
    q, k, v = (rand(g, T, h, d, dtype=dt) for h in (hq, hkv, hkv))
    freq, _ = bl.rope_frequencies(rot)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    want_k, want_v = kp.clone(), vp.clone()
    got = bl.paged_append(q, k, v, kp, vp, table, lens, R.cu(q_lens), inv_freq=freq, interleaved=interleaved, mscale=1.5)
    for i, ((a, b), n) in enumerate(zip(R.spans(q_lens), kv_lens)):
        pos = torch.arange(n - (b - a), n, device="cuda")
        args = (pos, freq) if b > a else None
        if args is None:
            continue
        # the same turn as blasst_rotary's, bit for bit
        turned = [bl.rotary(t[a:b], freq, pos, interleaved=interleaved, mscale=1.5) for t in (q, k)]
        assert torch.equal(got[a:b], turned[0])
        want_k[table[i].long()[pos // page], pos % page] = turned[1]
        want_v[table[i].long()[pos // page], pos % page] = v[a:b]
    # every page that the new tokens do not name is as it was (NaN among them)
    assert torch.equal(kp.view(dt).nan_to_num(777.0), want_k.nan_to_num(777.0))
    assert torch.equal(vp.nan_to_num(777.0), want_v.nan_to_num(777.0))
    # nothing to turn, q in place
    kp2, vp2 = want_k.clone(), want_v.clone()
    q2 = q.clone()
    assert bl.paged_append(q2, k, v, kp2, vp2, table, lens, R.cu(q_lens), q_out=q2).data_ptr() == q2.data_ptr()
    assert torch.equal(q2, q)
    for i, ((a, b), n) in enumerate(zip(R.spans(q_lens), kv_lens)):
        pos = torch.arange(n - (b - a), n, device="cuda")
        assert torch.equal(kp2[table[i].long()[pos // page], pos % page], k[a:b])
    assert bl.blasst_check() == 0


def test_append_bad_places_write_nothing(bl):
    import torch
    g = gen(4)
    q_lens, kv_lens = [2, 3, 1], [20, 9, 40]
    kp, vp, table, _ = R.paged(kv_lens, 16, 2, 64, torch.bfloat16, g)
    q = rand(g, 6, 4, 64, dtype="bfloat16")
    k, v = rand(g, 6, 2, 64, dtype="bfloat16"), rand(g, 6, 2, 64, dtype="bfloat16")
    lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    for change in ("page", "negative page", "length", "short length"):
        t, n = table.clone(), lens.clone()
        if change == "page":
            t[0, 1] = kp.shape[0]
        elif change == "negative page":
            t[0, 1] = -1
        elif change == "length":
            n[0] = 16 * table.shape[1] + 2
        else:
            n[0] = 1
        a, b = kp.clone(), vp.clone()
        bl.paged_append(q, k, v, a, b, t, n, R.cu(q_lens))
        assert bl.blasst_check() == bl.BLASST_EINDEX, change
        assert bl.blasst_check() == 0
        # sequence 0's places that are out of range are not written, the others' are
        ok_k, ok_v = kp.clone(), vp.clone()
        for i, ((c, e), m) in enumerate(zip(R.spans(q_lens), kv_lens)):
            pos = torch.arange(m - (e - c), m, device="cuda")
            if i == 0:
                if change != "short length":
                    continue
                pos, c = torch.tensor([0], device="cuda"), 1  # its second token has place 0
            ok_k[table[i].long()[pos // 16], pos % 16] = k[c:e]
            ok_v[table[i].long()[pos // 16], pos % 16] = v[c:e]
        assert torch.equal(a.nan_to_num(7.0), ok_k.nan_to_num(7.0)), change
        assert torch.equal(b.nan_to_num(7.0), ok_v.nan_to_num(7.0)), change


# ---------------------------------------------------- packed, with gradients
PACKED = [
    ([1], None, 1, 1, 64, True), ([1, 1, 1], None, 4, 2, 128, True), ([0, 5, 0, 130, 1, 0], None, 4, 4, 64, True),
    ([127, 128, 129, 63, 64, 65], None, 2, 1, 128, True), ([300, 17, 255, 256, 257], None, 6, 2, 64, True),
    ([300, 17, 255, 1], None, 3, 1, 128, False), ([700], None, 8, 1, 64, True), ([513, 200], None, 5, 1, 128, True),
    ([33, 200, 1, 77], [150, 128, 65, 12], 6, 2, 64, False), ([33, 200, 1, 77], [150, 128, 65, 12], 8, 2, 128, True),
    ([300, 140, 3], [7, 140, 0], 4, 1, 64, True), ([5, 0, 9], [0, 300, 200], 2, 2, 128, False),
    ([3] * 70, [(7 * i) % 50 for i in range(70)], 4, 2, 64, True), ([40, 2], [1000, 2100], 128, 1, 64, True),
    ([9, 1, 1], [2500, 700, 3000], 40, 8, 128, True), ([1500, 2], None, 16, 2, 128, True),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_lens,k_lens,hq,hkv,d,causal", PACKED)
def test_packed_and_gradients(bl, dtype, q_lens, k_lens, hq, hkv, d, causal):
    import torch
    kl = q_lens if k_lens is None else k_lens
    q, k, v, g = qkv(5, q_lens, kl, hq, hkv, d, dtype)
    cu_q, cu_k = R.cu(q_lens), None if k_lens is None else R.cu(kl)
    o, lse = bl.attention_packed(q, k, v, cu_q, cu_k, causal=causal)
    assert bl.blasst_check() == 0
    R.check_packed((o, lse), q, k, v, q_lens, kl, causal)
    dout = rand(g, sum(q_lens), hq, d, dtype=dtype)
    got = bl.attention_packed_backward(q, k, v, o, lse, dout, cu_q, cu_k, causal=causal)
    assert bl.blasst_check() == 0
    R.check_grads(got, q, k, v, o, lse, dout, q_lens, kl, causal)
    # the same bits again
    again = bl.attention_packed_backward(q, k, v, o, lse, dout, cu_q, cu_k, causal=causal)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    o2, lse2 = bl.attention_packed(q, k, v, cu_q, cu_k, causal=causal)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,hq,hkv,d,causal,mean", [
    ([40], 12, 4, 128, True, 0.5), ([5, 17, 3, 90, 33], 8, 4, 64, True, 0.5), ([600], 4, 2, 128, True, 0.5),
    ([300, 20], 3, 1, 128, False, 0.5), ([40, 200], 8, 2, 128, True, 3.0)])
def test_error_of_query_gradients(bl, dtype, lens, hq, hkv, d, causal, mean):
    """dQ is as near as rounding dS and the result makes it, also where few keys
    are seen or the keys have much in common. The model: both rounded, all else in
    64 bits; its error's norm is the kernel's expected one, and 1.1 leaves ten times
    the spread of a norm over thousands of independent roundings (2e4 values: 1 %)."""
    import torch
    q, k, v, g = qkv(23, lens, lens, hq, hkv, d, dtype)
    k = (k + mean * torch.randn(1, hkv, d, generator=g, device="cuda")).to(k.dtype)
    cu = R.cu(lens)
    o, lse = bl.attention_packed(q, k, v, cu, causal=causal)
    dout = rand(g, sum(lens), hq, d, dtype=dtype)
    dq = bl.attention_packed_backward(q, k, v, o, lse, dout, cu, causal=causal)[0]
    assert bl.blasst_check() == 0
    off = model = 0.0
    for a, b in R.spans(lens):
        qq, kk, vv = q[a:b].double().transpose(0, 1), *(R.heads(t[a:b], hq // hkv).transpose(0, 1) for t in (k, v))
        go = dout[a:b].double().transpose(0, 1)
        p = torch.exp(qq @ kk.transpose(1, 2) * d ** -0.5 - lse[a:b].double().t()[..., None])
        if causal:
            p = p.tril()
        ds = p * (go @ vv.transpose(1, 2) - (go * o[a:b].double().transpose(0, 1)).sum(-1, keepdim=True))
        want = (ds @ kk) * d ** -0.5
        # (fp16 holds dS scaled, so that it has all its bits)
        scale = 2.0 ** 10 if dtype == "float16" else 1.0
        rounded = ((ds * scale).to(q.dtype).double() / scale @ kk) * d ** -0.5
        off += float((dq[a:b].double().transpose(0, 1) - want).square().sum())
        model += float((rounded.to(q.dtype).double() - want).square().sum())
    assert off <= 1.1 ** 2 * model, (off / model) ** 0.5


@pytest.mark.parametrize("first", [0, 333])
def test_many_sequences(bl, first):
    """More sequences than one look of a warp covers, empty ones among them, through
    both ways of dealing out the work (few keys in all, and many)."""
    import torch
    g = gen(20)
    n = 1500
    q_lens = [(0, 1, 2, 7, 1, 0, 40)[i % 7] for i in range(n)]
    for k_lens in (q_lens, [(3 * i) % 25 for i in range(n)], [1 + (i == 700) * 3000 for i in range(n)]):
        t, tk = sum(q_lens) + first, sum(k_lens) + first
        q, k, v = rand(g, t, 2, 64, dtype="bfloat16"), rand(g, tk, 1, 64, dtype="bfloat16"), rand(g, tk, 1, 64, dtype="bfloat16")
        cq, ck = R.cu(q_lens, first), R.cu(k_lens, first)
        o, lse = bl.attention_packed(q, k, v, cq, ck)
        dout = rand(g, t, 2, 64, dtype="bfloat16")
        got = bl.attention_packed_backward(q, k, v, o, lse, dout, cq, ck)
        assert bl.blasst_check() == 0
        own = slice(first, None)
        R.check_packed((o[own], lse[own]), q[own], k[own], v[own], q_lens, k_lens, True)
        R.check_grads([x[own] for x in got], q[own], k[own], v[own], o[own], lse[own], dout[own], q_lens, k_lens, True)
    kv_lens = [1 + (37 * i) % 90 + (i % 97 == 5) * 1500 for i in range(700)]
    ones = [1 + (i % 50 == 3) for i in range(700)]
    kp, vp, table, rows = R.paged(kv_lens, 16, 1, 64, torch.float16, g)
    q = rand(g, sum(ones), 4, 64, dtype="float16")
    got = bl.attention_paged(q, kp, vp, table, torch.tensor(kv_lens, dtype=torch.int32, device="cuda"), R.cu(ones))
    assert bl.blasst_check() == 0
    k, v = (torch.cat([r[i] for r in rows]) for i in range(2))
    R.check_packed(got, q, k, v, ones, kv_lens, True)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_side_without_tokens(bl, dtype):
    import torch
    q, k, v, g = qkv(21, [5, 9], [5, 9], 4, 2, 64, dtype)
    cu, none = R.cu([5, 9]), R.cu([0, 0])
    o, lse = bl.attention_packed(q, k[:0], v[:0], cu, none)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    got = bl.attention_packed_backward(q, k[:0], v[:0], o, lse, torch.ones_like(q), cu, none)
    assert bool((got[0] == 0).all()) and got[1].shape == (0, 2, 64)
    o, lse = bl.attention_packed(q[:0], k, v, none, cu)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    got = bl.attention_packed_backward(q[:0], k, v, o, lse, q[:0], none, cu)
    assert bool((got[1] == 0).all()) and bool((got[2] == 0).all())
    o, lse = bl.attention_packed(q, k, v, cu[:1])  # no sequence at all
    assert o.shape == q.shape
    assert bl.blasst_check() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_packed_strides_scale_and_unowned_tokens(bl, dtype):
    """One projection's q, k and v side by side, tokens before the first and behind
    the last sequence that are NaN, a scale of its own."""
    import torch
    g = gen(6)
    hq, hkv, d, lens, first, behind = 6, 2, 64, [50, 0, 131, 9], 11, 40
    total = first + sum(lens) + behind
    wide = rand(g, total, (hq + 2 * hkv) * d + 16, dtype=dtype)
    wide[:first] = math.nan
    wide[first + sum(lens):] = math.nan
    q = wide[:, 8:8 + hq * d].unflatten(1, (hq, d))
    k = wide[:, 8 + hq * d:8 + (hq + hkv) * d].unflatten(1, (hkv, d))
    v = wide[:, 8 + (hq + hkv) * d:8 + (hq + 2 * hkv) * d].unflatten(1, (hkv, d))
    cu = R.cu(lens, first)
    o, lse = bl.attention_packed(q, k, v, cu, causal=True, scale=0.31)
    own = slice(first, first + sum(lens))
    R.check_packed((o[own], lse[own]), q[own], k[own], v[own], lens, lens, True, 0.31)
    # the gradient with heads before tokens
    dout = rand(g, hq, total, d, dtype=dtype).transpose(0, 1)
    dout[:first] = math.nan
    dout[first + sum(lens):] = math.nan
    got = bl.attention_packed_backward(q, k, v, o, lse, dout, cu, causal=True, scale=0.31)
    R.check_grads([t[own] for t in got], q[own], k[own], v[own], o[own], lse[own], dout[own], lens, lens, True, 0.31)
    assert bl.blasst_check() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [True, False])
def test_unowned_outputs_are_left(bl, dtype, causal):
    """Through the C ABI with outputs of the caller's: rows of no sequence stay."""
    import ctypes as C

    import torch
    from test_seq_host import struct_of
    lib = bl.load_library()
    hq, hkv, d, lens, first, behind = 4, 2, 128, [70, 200], 3, 5
    total = first + sum(lens) + behind
    q, k, v, g = qkv(7, [total], [total], hq, hkv, d, dtype)
    dout = rand(g, total, hq, d, dtype=dtype)
    cu = R.cu(lens, first)
    outs = {n: torch.full((total, h, d), 7.0, dtype=q.dtype, device="cuda") for n, h in
            (("o", hq), ("dq", hq), ("dk", hkv), ("dv", hkv))}
    lse = torch.full((total, hq), 7.0, device="cuda")
    ws = torch.empty(max(bl.blasst_seq_workspace_bytes(d), bl.blasst_packed_bwd_workspace_bytes(total, hq, hkv)),
                     dtype=torch.uint8, device="cuda")
    common = dict(q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), lse=lse.data_ptr(), cu_q=cu.data_ptr(),
                  cu_k=cu.data_ptr(), n_seq=2, Tq=total, Tk=total, Hq=hq, Hkv=hkv, d=d, q_st=hq * d, q_sh=d,
                  k_st=hkv * d, k_sh=d, v_st=hkv * d, v_sh=d, causal=int(causal), dtype=0 if dtype == "bfloat16" else 2,
                  workspace=ws.data_ptr(), workspace_bytes=ws.numel(), stream=torch.cuda.current_stream().cuda_stream,
                  o=outs["o"].data_ptr())
    assert lib.blasst_packed_fwd(C.byref(struct_of("blasst_packed_args")(**common))) == 0
    args = dict(common, dout=dout.data_ptr(), o_st=hq * d, o_sh=d, do_st=hq * d, do_sh=d,
                **{n: outs[n].data_ptr() for n in ("dq", "dk", "dv")})
    assert lib.blasst_packed_bwd(C.byref(struct_of("blasst_packed_bwd_args")(**args))) == 0
    assert bl.blasst_check() == 0
    own = slice(first, first + sum(lens))
    for t in list(outs.values()) + [lse]:
        assert bool((t[:first] == 7).all()) and bool((t[first + sum(lens):] == 7).all())
    R.check_packed((outs["o"][own], lse[own]), q[own], k[own], v[own], lens, lens, causal)
    R.check_grads([outs[n][own] for n in ("dq", "dk", "dv")], q[own], k[own], v[own], outs["o"][own], lse[own],
                  dout[own], lens, lens, causal)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [2.0 ** -12, 1.0, 2.0 ** 9])
def test_gradient_sizes(bl, dtype, size):
    """Gradients far from 1 (a mean over many tokens, a scaled loss): fp16 dS is
    scaled by the largest rows, so it neither overflows nor fades."""
    lens = [200, 700]
    q, k, v, g = qkv(8, lens, lens, 4, 2, 64, dtype)
    dout = (rand(g, 900, 4, 64, dtype="float32") * size).to(q.dtype)
    o, lse = bl.attention_packed(q, k, v, R.cu(lens))
    got = bl.attention_packed_backward(q, k, v, o, lse, dout, R.cu(lens))
    R.check_grads(got, q, k, v, o, lse, dout, lens, lens, True)
    assert bl.blasst_check() == 0


def test_large_scores_and_references_that_move(bl):
    """Keys whose scores grow along the row: the softmax's reference moves in
    every block, in either half of it."""
    import torch
    for step in (0.02, 0.2):
        lens = [600]
        q, k, v, g = qkv(9, lens, lens, 2, 1, 64, "bfloat16")
        k = k + q[:, :1] * 0  # (same device and type)
        ramp = (torch.arange(600, device="cuda") * step)[:, None, None]
        q[..., 0] = 8.0
        k[..., 0] = ramp[..., 0].to(k.dtype)
        o, lse = bl.attention_packed(q, k, v, R.cu(lens), causal=False)
        R.check_packed((o, lse), q, k, v, lens, lens, False)
        o, lse = bl.attention_packed(q[:3], k, v, R.cu([3]), R.cu(lens), causal=True)
        R.check_packed((o, lse), q[:3], k, v, [3], lens, True)
    assert bl.blasst_check() == 0


def test_gradient_against_differences(bl):
    """<gradient, direction> against central differences of the definition."""
    import torch
    lens, kl = [60, 33], [75, 20]
    q, k, v, g = qkv(10, lens, kl, 4, 2, 64, "float16")
    dout = rand(g, 93, 4, 64, dtype="float16")
    o, lse = bl.attention_packed(q, k, v, R.cu(lens), R.cu(kl))
    got = bl.attention_packed_backward(q, k, v, o, lse, dout, R.cu(lens), R.cu(kl))

    def loss(x, y, z):
        t = 0.0
        for (a, b), (c, e) in zip(R.spans(lens), R.spans(kl)):
            t += float((R.attend(x[a:b], y[c:e], z[c:e], True)[0] * dout[a:b].double()).sum())
        return t

    base = [t.double() for t in (q, k, v)]
    for i in range(3):
        way = torch.randn(base[i].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        up = [t + h * way if j == i else t for j, t in enumerate(base)]
        down = [t - h * way if j == i else t for j, t in enumerate(base)]
        slope = (loss(*up) - loss(*down)) / (2 * h)
        bound = 0.0
        for (a, b), (c, e) in zip(R.spans(lens), R.spans(kl)):
            bd = R.grads(q[a:b], k[c:e], v[c:e], o[a:b], lse[a:b], dout[a:b], True)[1][i]
            x, y = (a, b) if i == 0 else (c, e)
            # errors of single elements have random signs: their root sum of squares, times 4
            bound += float((bd * way[x:y]).square().sum())
        # (o and with it D is rounded too: counted by the same bound)
        assert abs(float((got[i].double() * way).sum()) - slope) <= 4 * math.sqrt(bound) + 1e-6 * abs(slope)


def test_index_errors(bl):
    import torch
    q, k, v, g = qkv(11, [100], [100], 2, 1, 64, "bfloat16")
    dout = torch.zeros_like(q)
    for bad in ([0, 60, 101], [0, -1, 100], [0, 80, 60], [-5, 50, 100]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        o, lse = bl.attention_packed(q, k, v, cu)
        assert bl.blasst_check() == bl.BLASST_EINDEX
        bl.attention_packed_backward(q, k, v, o, lse, dout, cu)
        assert bl.blasst_check() == bl.BLASST_EINDEX
    o, lse = bl.attention_packed(q, k, v, R.cu([40, 60]))
    assert bl.blasst_check() == 0
    R.check_packed((o, lse), q, k, v, [40, 60], [40, 60], True)


def test_attention_refusals(bl):
    import torch
    q, k, v, g = qkv(12, [8], [8], 4, 2, 64, "bfloat16")
    cu = R.cu([8])
    o, lse = bl.attention_packed(q, k, v, cu)
    pool, table, lens = torch.zeros(4, 16, 2, 64, dtype=q.dtype, device="cuda"), cu.new_zeros(1, 4), R.cu([8])[1:]
    value = [lambda: bl.attention_packed(q, k.half(), v, cu), lambda: bl.attention_packed(q, k, v[:7], cu),
             lambda: bl.attention_packed(q, k, v, cu.long()), lambda: bl.attention_packed(q, k, v, cu, R.cu([4, 4])),
             lambda: bl.attention_packed(q[0], k, v, cu), lambda: bl.attention_packed(q, k.cpu(), v, cu),
             lambda: bl.attention_packed(q.double(), k.double(), v.double(), cu),
             lambda: bl.attention_packed(q, k, v, cu[:0]),
             lambda: bl.attention_packed(q, k, v, cu, workspace=torch.zeros(8, 8, device="cuda").t()[:, :4]),
             lambda: bl.attention_packed_backward(q, k, v, o[:7], lse, o, cu),
             lambda: bl.attention_packed_backward(q, k, v, o, lse.half(), o, cu),
             lambda: bl.attention_packed_backward(q, k, v, o, lse.t().contiguous().t(), o, cu),
             lambda: bl.attention_packed_backward(q, k, v, o, lse, o.half(), cu),
             lambda: bl.attention_paged(q, pool, pool[:3], table, lens, cu),
             lambda: bl.attention_paged(q, pool, pool, table.expand(2, 4), lens, cu),
             lambda: bl.attention_paged(q, pool, pool, table.long(), lens, cu),
             lambda: bl.attention_paged(q, pool, pool, table, cu, cu),
             lambda: bl.attention_paged(q[..., :32], pool, pool, table, lens, cu),
             lambda: bl.paged_append(q, k, v[:, :1], pool, pool, table, lens, cu),
             lambda: bl.paged_append(q, k, v, pool, pool, table, lens, cu, q_out=q[:4])]
    for f in value:
        with pytest.raises(ValueError):
            f()
    status = [lambda: bl.attention_packed(q[..., :48], k[..., :48], v[..., :48], cu),          # d
              lambda: bl.attention_packed(q[:, :3], k, v, cu),                                 # groups
              lambda: bl.attention_packed(q.float(), k.float(), v.float(), cu),                # type
              lambda: bl.attention_packed_backward(q, k, v, o, lse, torch.ones_like(q[:1, :1]).expand(8, 4, 64), cu),
              lambda: bl.attention_packed(q, k, v, cu, workspace=torch.zeros(64, device="cuda")),
              lambda: bl.attention_packed(q, k, v, cu, scale=math.nan),
              lambda: bl.attention_paged(q, pool[:, :12], pool[:, :12], table, lens, cu)]      # page size
    for f in status:
        with pytest.raises(bl.BlasstError):
            f()
    assert bl.blasst_check() == 0


# -------------------------------------------------------------------- paged
PAGED = [
    ([1], [1], 1, 1, 64, 16, True), ([1] * 5, [700, 1, 4097, 128, 129], 16, 2, 64, 16, True),
    ([1] * 5, [127, 5000, 2, 300, 64], 32, 8, 128, 64, True), ([1, 1], [3000, 9], 5, 1, 128, 24, True),
    ([1] * 40, [(97 * i) % 900 + 1 for i in range(40)], 4, 2, 128, 8, True),
    ([3, 8, 1, 2], [3, 900, 70, 2000], 8, 1, 64, 32, True), ([4, 4], [200, 6000], 8, 1, 128, 128, True),
    ([200, 1, 0, 65, 1], [1000, 300, 50, 65, 8], 4, 1, 128, 32, True), ([130, 5], [130, 1200], 3, 1, 64, 256, False),
    ([1, 1, 2], [500, 0, 1], 4, 4, 64, 200, True), ([1, 30], [40, 2000], 128, 1, 64, 16, True),
    ([1] * 3, [900, 20, 333], 80, 2, 128, 16, False), ([700, 1, 1], [3000, 5, 2500], 2, 2, 64, 16, True),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,d,page,causal", PAGED)
@pytest.mark.parametrize("head_major", [False, True])
def test_paged(bl, dtype, q_lens, kv_lens, hq, hkv, d, page, causal, head_major):
    import torch
    g = gen(13)
    dt = getattr(torch, dtype)
    kp, vp, table, rows = R.paged(kv_lens, page, hkv, d, dt, g, head_major)
    q = rand(g, sum(q_lens), hq, d, dtype=dt)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    got = bl.attention_paged(q, kp, vp, table, lens, R.cu(q_lens), causal=causal)
    assert bl.blasst_check() == 0
    k, v = (torch.cat([r[i] for r in rows]) for i in range(2))
    R.check_packed(got, q, k, v, q_lens, kv_lens, causal)
    again = bl.attention_paged(q, kp, vp, table, lens, R.cu(q_lens), causal=causal)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_paged_bad_pages_and_lengths(bl):
    import torch
    g = gen(14)
    kv_lens = [300, 40]
    kp, vp, table, rows = R.paged(kv_lens, 16, 2, 64, torch.float16, g)
    q = rand(g, 2, 8, 64, dtype="float16")
    lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    for change in ("page", "negative page", "length", "negative length"):
        t, n = table.clone(), lens.clone()
        if change == "page":
            t[0, 3] = kp.shape[0]
        elif change == "negative page":
            t[0, 3] = -2
        elif change == "length":
            n[0] = 16 * table.shape[1] + 1
            t[0] = table[0, 0]  # (the length is clamped to the table: give it pages)
        else:
            n[0] = -4
        o, lse = bl.attention_paged(q, kp, vp, t, n, R.cu([1, 1]))
        assert bl.blasst_check() == bl.BLASST_EINDEX, change
        # the other sequence's row is right all the same
        R.check_packed((o[1:], lse[1:]), q[1:], rows[1][0], rows[1][1], [1], [40], True, what=change)
    assert bl.blasst_check() == 0


def test_paged_offsets_past_32_bits(bl):
    """A pool of more than 2^31 elements, its last pages in use, some of them named twice."""
    import torch
    g = gen(15)
    page, hkv, d = 64, 8, 128
    total = (1 << 31) // (page * hkv * d) + 9
    kp = torch.empty(total, page, hkv, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    table = torch.tensor([[total - 1, 0, total - 2, total - 1], [total - 3, total - 2, -1, -1]], dtype=torch.int32, device="cuda")
    lens = [230, 100]
    for i in sorted(set(table.flatten().tolist()) - {-1}):
        kp[i] = rand(g, page, hkv, d, dtype="bfloat16")
        vp[i] = rand(g, page, hkv, d, dtype="bfloat16")
    q = rand(g, 2, 16, d, dtype="bfloat16")
    got = bl.attention_paged(q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), R.cu([1, 1]))
    k, v = (torch.cat([t[table[s].long().clamp(min=0)].flatten(0, 1)[:n] for s, n in enumerate(lens)]) for t in (kp, vp))
    R.check_packed(got, q, k, v, [1, 1], lens, True)
    new = rand(g, 2, hkv, d, dtype="bfloat16")
    bl.paged_append(q, new, new, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), R.cu([1, 1]))
    assert torch.equal(kp[total - 1, 229 - 192], new[0]) and torch.equal(vp[total - 2, 99 - 64], new[1])
    assert bl.blasst_check() == 0


# ------------------------------------------------ streams, graphs, together
def test_streams_and_own_workspaces(bl):
    import torch
    lens = [900, 30, 1]
    q, k, v, g = qkv(16, lens, lens, 4, 2, 64, "bfloat16")
    dout = rand(g, sum(lens), 4, 64, dtype="bfloat16")
    cu = R.cu(lens)
    o, lse = bl.attention_packed(q, k, v, cu)
    grads = bl.attention_packed_backward(q, k, v, o, lse, dout, cu)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    results = []
    for i, s in enumerate(side):
        if i == 0:
            with torch.cuda.stream(s):
                r = bl.attention_packed(q, k, v, cu)
                results.append((r, bl.attention_packed_backward(q, k, v, o, lse, dout, cu)))
        else:  # a stream object, a raw handle; the second with workspaces of its own
            at = s if i == 1 else s.cuda_stream
            ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
                  (bl.blasst_seq_workspace_bytes(64), bl.blasst_packed_bwd_workspace_bytes(931, 4, 2))] if i == 2 else [None, None]
            r = bl.attention_packed(q, k, v, cu, workspace=ws[0], stream=at)
            results.append((r, bl.attention_packed_backward(q, k, v, o, lse, dout, cu, workspace=ws[1], stream=at)))
    torch.cuda.synchronize()
    for r, gr in results:
        assert torch.equal(r[0], o) and torch.equal(r[1], lse)
        assert all(torch.equal(a, b) for a, b in zip(gr, grads))
    assert bl.blasst_check() == 0


def test_inputs_freed_behind_a_call_on_another_stream(bl):
    """A tensor that the caller drops after a call on a stream of its choice is not
    given to anyone else before the kernel has read it."""
    import torch
    side = torch.cuda.Stream()
    freq, _ = bl.rope_frequencies(128)
    x = rand(gen(29), 1000, 8, 128, dtype="bfloat16")
    want = bl.rotary(x, freq)
    mine = x.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    y = bl.rotary(mine, freq, stream=side)
    del mine
    others = [torch.full_like(x, 7.0) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(y, want) and len(others) == 4


def test_captured_steps_follow_the_lengths(bl):
    """A decode step captured once and replayed with longer sequences and other
    pages; a captured training step replayed with other inputs."""
    import torch
    g = gen(17)
    hq, hkv, d, page, n = 8, 2, 64, 16, 3
    width = 20
    kp = torch.full((n * width, page, hkv, d), math.nan, dtype=torch.float16, device="cuda")
    vp = kp.clone()
    table = torch.randperm(n * width, generator=g, device="cuda").int().view(n, width)
    start = [5, 100, 31]
    lens = torch.tensor(start, dtype=torch.int32, device="cuda")
    freq, _ = bl.rope_frequencies(d)
    cu = R.cu([1] * n)
    keys = [[[], []] for _ in range(n)]
    for s, m in enumerate(start):  # what is cached before
        kv = [rand(g, m, hkv, d, dtype="float16") for _ in range(2)]
        j = torch.arange(m, device="cuda")
        for i, pool in enumerate((kp, vp)):
            pool[table[s].long()[j // page], j % page] = kv[i]
            keys[s][i].append(kv[i])
    q, k, v = (torch.zeros(n, h, d, dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv))

    def step():
        lens.add_(1)
        turned = bl.paged_append(q, k, v, kp, vp, table, lens, cu, inv_freq=freq)
        return turned, bl.attention_paged(turned, kp, vp, table, lens, cu)

    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        kp0, vp0, lens0 = kp.clone(), vp.clone(), lens.clone()
        step()
        kp.copy_(kp0), vp.copy_(vp0), lens.copy_(lens0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=warm):
        turned, out = step()
    lens.copy_(lens0), kp.copy_(kp0), vp.copy_(vp0)
    for i in range(4):
        for t in (q, k, v):
            t.copy_(rand(g, *t.shape, dtype="float16"))
        if i == 2:  # a page moves
            a, b = int(table[1, 2]), int(table[0, 15])
            kp[b], vp[b] = kp[a].clone(), vp[a].clone()
            table[1, 2], table[0, 15] = b, a
        graph.replay()
        torch.cuda.synchronize()
        for s in range(n):
            pos = torch.tensor([start[s] + i], device="cuda")
            keys[s][0].append(bl.rotary(k[s:s + 1], freq, pos))
            keys[s][1].append(v[s:s + 1].clone())
        kl = [m + i + 1 for m in start]
        kk, vv = (torch.cat([t for s in keys for t in s[j]]) for j in range(2))
        R.check_packed(out, turned, kk, vv, [1] * n, kl, True, what=f"step {i}")
    # training
    L = [40, 200]
    x = [torch.zeros(240, h, d, dtype=torch.float16, device="cuda") for h in (4, 2, 2, 4)]
    ends = R.cu(L)

    def train():
        o, lse = bl.attention_packed(x[0], x[1], x[2], ends)
        return o, lse, bl.attention_packed_backward(x[0], x[1], x[2], o, lse, x[3], ends)

    with torch.cuda.stream(warm):
        train()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=warm):
        o, lse, got = train()
    for lens2 in ([40, 200], [201, 39]):
        for t in x:
            t.copy_(rand(g, *t.shape, dtype="float16"))
        ends.copy_(R.cu(lens2))
        graph.replay()
        torch.cuda.synchronize()
        R.check_packed((o, lse), *x[:3], lens2, lens2, True)
        R.check_grads(got, *x[:3], o, lse, x[3], lens2, lens2, True)
    assert bl.blasst_check() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_prompts_in_chunks_equal_packed_prompts(bl, dtype):
    """The operators together: prompts that enter the cache in chunks and single
    tokens, each attending to what is cached, against one packed call over the
    whole turned prompts."""
    import torch
    g = gen(18)
    hq, hkv, d, page, lens = 8, 2, 128, 32, [300, 77, 131]
    freq, m = bl.rope_frequencies(d, scaling="blend", factor=4.0, original_len=64)
    q, k, v = (rand(g, sum(lens), h, d, dtype=dtype) for h in (hq, hkv, hkv))
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    tq, tk = bl.rotary(q, freq, pos, mscale=m), bl.rotary(k, freq, pos, mscale=m)
    whole = bl.attention_packed(tq, tk, v, R.cu(lens))
    R.check_packed(whole, tq, tk, v, lens, lens, True)
    need = [-(-n // page) for n in lens]
    kp = torch.full((sum(need), page, hkv, d), math.nan, dtype=q.dtype, device="cuda")
    vp = kp.clone()
    table = torch.full((3, max(need)), -1, dtype=torch.int32, device="cuda")
    order, at = torch.randperm(sum(need), generator=g, device="cuda").int(), 0
    for s, c in enumerate(need):
        table[s, :c] = order[at:at + c]
        at += c
    done = [0, 0, 0]
    starts = [a for a, _ in R.spans(lens)]
    o, lse = torch.empty_like(q), torch.empty(sum(lens), hq, device="cuda")
    for chunk in ([256, 50, 0], [1, 1, 130], [40, 1, 1], [3, 25, 0]):
        idx = torch.cat([torch.arange(starts[s] + done[s], starts[s] + done[s] + c, device="cuda") for s, c in enumerate(chunk)])
        done = [a + c for a, c in zip(done, chunk)]
        cu, now = R.cu(chunk), torch.tensor(done, dtype=torch.int32, device="cuda")
        turned = bl.paged_append(q[idx], k[idx], v[idx], kp, vp, table, now, cu, inv_freq=freq, mscale=m)
        assert torch.equal(turned, tq[idx])
        o[idx], lse[idx] = bl.attention_paged(turned, kp, vp, table, now, cu)
    assert done == lens
    R.check_packed((o, lse), tq, tk, v, lens, lens, True)
    assert bl.blasst_check() == 0


def test_training_step_through_rotary(bl):
    """rotary -> packed attention and back: gradients of the projections' outputs
    against 64-bit autograd of the same formula."""
    import torch
    g = gen(19)
    lens, hq, hkv, d = [120, 40], 4, 2, 64
    freq, _ = bl.rope_frequencies(32)
    q, k, v = (rand(g, 160, h, d, dtype="bfloat16") for h in (hq, hkv, hkv))
    dout = rand(g, 160, hq, d, dtype="bfloat16")
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    cu = R.cu(lens)
    tq, tk = bl.rotary(q, freq, pos, interleaved=True), bl.rotary(k, freq, pos, interleaved=True)
    o, lse = bl.attention_packed(tq, tk, v, cu)
    dq, dk, dv = bl.attention_packed_backward(tq, tk, v, o, lse, dout, cu)
    got = [bl.rotary_backward(dq, freq, pos, interleaved=True), bl.rotary_backward(dk, freq, pos, interleaved=True), dv]
    leaf = [t.double().requires_grad_() for t in (q, k, v)]
    a, c = pos.double()[:, None] * freq, None

    def turn(x):
        c, s = a.cos()[:, None], a.sin()[:, None]
        p, r = x[..., 0:32:2], x[..., 1:32:2]
        return torch.cat([torch.stack([p * c - r * s, p * s + r * c], -1).flatten(-2), x[..., 32:]], -1)

    loss = 0.0
    for x, y in R.spans(lens):
        qq, kk = turn(leaf[0])[x:y].transpose(0, 1), turn(leaf[1])[x:y].repeat_interleave(2, 1).transpose(0, 1)
        s = (qq @ kk.transpose(1, 2) / math.sqrt(d)).masked_fill(
            torch.ones(y - x, y - x, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        loss = loss + (s.softmax(-1) @ leaf[2][x:y].repeat_interleave(2, 1).transpose(0, 1) * dout[x:y].double().transpose(0, 1)).sum()
    loss.backward()
    # turned inputs, P or dS, the gradient before and behind the turn: four roundings of random sign in
    # a row, norm-wise at most 4 u of the sums of their terms; against the gradient's norm twice that
    for t, x in zip(got, leaf):
        assert float((t.double() - x.grad).norm()) <= 8 * 2.0 ** -8 * float(x.grad.norm())
    assert bl.blasst_check() == 0
