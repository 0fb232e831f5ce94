"""Host-side checks of the operators over sequences of different lengths: the C
ABI refuses bad arguments before it touches a device, the frequency tables, the
binding's refusals."""
import ctypes as C
import math
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def struct_of(name):
    """The ctypes form of an argument struct, read from the header."""
    src = open(os.path.join(ROOT, "include", "blasst.h")).read()
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), src, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = []
    for line in filter(None, (x.strip() for x in body.split(";"))):
        if "*" in line:
            fields.append((line.split("*")[-1].strip(), C.c_void_p))
            continue
        kind = next(t for t in ("long long", "size_t", "int", "float") if line.startswith(t))
        ctype = {"long long": C.c_longlong, "size_t": C.c_size_t, "int": C.c_int, "float": C.c_float}[kind]
        fields += [(n.strip(), ctype) for n in line[len(kind):].split(",")]
    return type(name, (C.Structure,), {"_fields_": fields})


@pytest.fixture(scope="module")
def lib():
    from dynamic_block_sparse_tiled_b200 import build
    build.build()
    import dynamic_block_sparse_tiled_b200 as bl
    return bl.load_library()


def call(lib, entry, base, **kw):
    args = {**base, **kw}
    t = struct_of(entry.replace("_fwd", "") + "_args")
    known = {f[0] for f in t._fields_}
    assert set(args) <= known, set(args) - known
    return getattr(lib, entry)(C.byref(t(**args)))


ROTARY = dict(x=0x10000, y=0x20000, positions=None, freq=0x30000, B=1, L=4, H=2, d=64, rot=64, x_sb=512,
              x_sl=128, x_sh=64, y_sb=512, y_sl=128, y_sh=64, scale=1.0)
APPEND = dict(q=0x10000, q_out=0x10000, k=0x20000, v=0x30000, k_pages=0x40000, v_pages=0x50000,
              page_table=0x60000, kv_lens=0x70000, cu_q=0x80000, freq=0x90000, n_seq=2, T=4, Hq=4, Hkv=2,
              d=64, rot=64, n_pages=4, page_size=16, table_width=2, table_stride=2, q_st=256, q_sh=64,
              qo_st=256, qo_sh=64, k_st=128, k_sh=64, v_st=128, v_sh=64, kp_sp=2048, kp_st=128, kp_sh=64,
              vp_sp=2048, vp_st=128, vp_sh=64, scale=1.0)
PACKED = dict(q=0x10000, k=0x20000, v=0x30000, o=0x40000, lse=0x50000, cu_q=0x60000, cu_k=0x60000, n_seq=2,
              Tq=8, Tk=8, Hq=4, Hkv=2, d=64, q_st=256, q_sh=64, k_st=128, k_sh=64, v_st=128, v_sh=64,
              causal=1, workspace=0x70000, workspace_bytes=1 << 30)
BACKWARD = dict(PACKED, dout=0x80000, dq=0x90000, dk=0xA0000, dv=0xB0000, o_st=256, o_sh=64, do_st=256,
                do_sh=64)
PAGED = dict(q=0x10000, k_pages=0x40000, v_pages=0x50000, o=0x20000, lse=0x30000, page_table=0x60000,
             kv_lens=0x70000, cu_q=0x80000, n_seq=2, Tq=4, Hq=4, Hkv=2, d=64, n_pages=4, page_size=16,
             table_width=2, table_stride=2, q_st=256, q_sh=64, kp_sp=2048, kp_st=128, kp_sh=64, vp_sp=2048,
             vp_st=128, vp_sh=64, causal=1, workspace=0x90000, workspace_bytes=1 << 30)


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(freq=None), -1), (dict(dtype=3), -2), (dict(B=-1), -1),
    (dict(d=0), -1), (dict(rot=0), -1), (dict(rot=63), -1), (dict(rot=66), -1), (dict(d=1025, rot=2), -2),
    (dict(scale=0.0), -1), (dict(scale=math.inf), -1), (dict(scale=math.nan), -1), (dict(x=0x10001), -1),
    (dict(freq=0x30004), -1), (dict(positions=0x40004, pos64=1), -1), (dict(positions=0x40002), -1),
    (dict(y=0x10000, y_sl=64), -1),  # in place with other strides
    (dict(L=0), 0), (dict(H=0), 0),
])
def test_rotary_refusals(lib, bad, code):
    assert call(lib, "blasst_rotary", ROTARY, **bad) == code


@pytest.mark.parametrize("bad,code", [
    *[({n: None}, -1) for n in ("k", "v", "k_pages", "v_pages", "page_table", "kv_lens", "cu_q", "q", "q_out")],
    (dict(dtype=3), -2), (dict(n_seq=-1), -1), (dict(T=-1), -1), (dict(Hkv=0), -1), (dict(Hq=0), -1),
    (dict(n_pages=0), -1), (dict(page_size=0), -1), (dict(table_stride=1), -1), (dict(rot=0), -1),
    (dict(freq=None), -1), (dict(rot=66), -1), (dict(scale=-1.0), -1), (dict(d=1026, rot=2), -2),
    (dict(k=0x20001), -1), (dict(kv_lens=0x70002), -1), (dict(qo_st=512), -1), (dict(T=0), 0), (dict(n_seq=0), 0),
])
def test_append_refusals(lib, bad, code):
    assert call(lib, "blasst_append", APPEND, **bad) == code


COMMON = [(dict(n_seq=-1), -1), (dict(Hq=3), -1), (dict(Hkv=0), -1), (dict(d=96), -2), (dict(d=256), -2),
          (dict(Hq=258, Hkv=2), -2), (dict(dtype=1), -2), (dict(dtype=9), -2), (dict(scale=math.nan), -1),
          (dict(q=0x10008), -1), (dict(lse=0x50004), -1), (dict(cu_q=0x60002), -1), (dict(q_st=0), -1),
          (dict(q_sh=-64), -1), (dict(q_st=260), -1), (dict(workspace=None), -5), (dict(workspace=0x70008), -5)]


@pytest.mark.parametrize("bad,code", COMMON + [
    *[({n: None}, -1) for n in ("q", "k", "v", "o", "lse", "cu_q", "cu_k")],
    (dict(Tq=-1), -1), (dict(Tk=-1), -1), (dict(k_st=4), -1), (dict(v_sh=0), -1), (dict(Tq=0), 0), (dict(n_seq=0), 0),
])
def test_packed_refusals(lib, bad, code):
    assert call(lib, "blasst_packed_fwd", PACKED, **bad) == code


@pytest.mark.parametrize("bad,code", COMMON + [
    *[({n: None}, -1) for n in ("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv", "cu_q", "cu_k")],
    (dict(o_st=0), -1), (dict(do_st=0), -1), (dict(do_sh=12), -1), (dict(dk=0xA0008), -1),
    (dict(workspace_bytes=287), -5), (dict(n_seq=0), 0), (dict(Tq=0, Tk=0), 0),
])
def test_packed_backward_refusals(lib, bad, code):
    assert call(lib, "blasst_packed_bwd", BACKWARD, **bad) == code


@pytest.mark.parametrize("bad,code", COMMON + [
    *[({n: None}, -1) for n in ("q", "k_pages", "v_pages", "o", "lse", "page_table", "kv_lens", "cu_q")],
    (dict(page_size=20), -2), (dict(page_size=4), -2), (dict(page_size=0), -1), (dict(n_pages=0), -1),
    (dict(table_width=3), -1), (dict(kp_sp=0), -1), (dict(vp_sh=63), -1), (dict(kv_lens=0x70001), -1),
    (dict(Tq=0), 0), (dict(n_seq=0), 0),
])
def test_paged_refusals(lib, bad, code):
    assert call(lib, "blasst_paged_fwd", PAGED, **bad) == code


def test_null_arguments(lib):
    for entry in ("blasst_rotary", "blasst_append", "blasst_packed_fwd", "blasst_packed_bwd", "blasst_paged_fwd"):
        assert getattr(lib, entry)(None) == -1


def test_workspaces(lib):
    import dynamic_block_sparse_tiled_b200 as bl
    assert bl.blasst_packed_bwd_workspace_bytes(8, 4, 2) == 2 * 16 + 8 * 4 * 8
    for bad in ((-1, 4, 2), (8, 0, 2), (8, 4, 0)):
        assert bl.blasst_packed_bwd_workspace_bytes(*bad) == 0
    assert bl.blasst_seq_workspace_bytes(96) == 0
    assert bl.blasst_status_string(bl.BLASST_EINDEX).startswith("BLASST_EINDEX")


def test_binding_refuses_tensors_off_the_gpu():
    import torch
    import dynamic_block_sparse_tiled_b200 as bl
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    f, _ = bl.rope_frequencies(64, device="cpu")
    pool = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 2, dtype=torch.int32)
    lse = torch.zeros(3, 2)
    for run in (lambda: bl.rotary(x, f), lambda: bl.rotary_backward(x, f), lambda: bl.attention_packed(x, x, x, cu),
                lambda: bl.attention_packed_backward(x, x, x, x, lse, x, cu),
                lambda: bl.attention_paged(x, pool, pool, table, cu[:1], cu),
                lambda: bl.paged_append(x, x, x, pool, pool, table, cu[:1], cu)):
        with pytest.raises(ValueError, match="CUDA device"):
            run()


def test_rope_frequencies():
    import torch
    import dynamic_block_sparse_tiled_b200 as bl
    i = torch.arange(32, dtype=torch.float64)
    base = 10000.0 ** (-2 * i / 64)
    f = lambda **kw: bl.rope_frequencies(64, device="cpu", **kw)  # noqa: E731
    plain, m = f()
    assert torch.equal(plain, base) and m == 1.0
    assert torch.allclose(f(scaling="linear", factor=4.0)[0], base / 4, rtol=1e-15)
    ntk = f(scaling="ntk", factor=4.0)[0]
    # the fastest pair is kept, the slowest is slowed by the factor
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], base[-1] / 4, rel_tol=1e-12)
    blend, m = f(scaling="blend", factor=4.0, original_len=2048)
    assert math.isclose(m, 0.1 * math.log(4.0) + 1.0)
    turns = 2048 * base / (2 * math.pi)
    kept, slowed = blend == base, torch.isclose(blend, base / 4, rtol=1e-14)
    # (the straight line runs between whole pair indices: one pair of slack each side)
    assert bool(kept[turns > 32 * 1.4].all()) and bool(slowed[turns < 1 / 1.4].all())
    assert bool((blend <= base).all()) and bool((blend >= base / 4 * (1 - 1e-14)).all())
    bands, m = f(scaling="bands", factor=8.0, original_len=8192)
    turns = 8192 * base / (2 * math.pi)
    assert m == 1.0 and bool((bands == base)[turns >= 4].all())
    assert bool(torch.isclose(bands, base / 8, rtol=1e-14)[turns <= 1].all())


@pytest.mark.parametrize("kw", [dict(rot=63), dict(rot=0), dict(base=1.0), dict(factor=0.0), dict(scaling="what"),
                                dict(rot=2, scaling="ntk", factor=2.0), dict(scaling="blend", factor=2.0),
                                dict(scaling="bands", original_len=64, low=4.0, high=2.0)])
def test_rope_frequencies_refusals(kw):
    import dynamic_block_sparse_tiled_b200 as bl
    with pytest.raises(ValueError):
        bl.rope_frequencies(kw.pop("rot", 64), device="cpu", **kw)
