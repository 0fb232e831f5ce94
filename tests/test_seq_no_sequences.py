"""Tokens of no sequence at all (an idle step of a padded batch): nothing is read or
written, nothing refused."""
import pytest

import test_seq_host as H
from test_seq_host import lib  # noqa: F401


@pytest.mark.parametrize("entry,base", [("blasst_append", H.APPEND), ("blasst_paged_fwd", H.PAGED)])
def test_c_abi(lib, entry, base):  # noqa: F811
    none = dict(page_table=None, kv_lens=None)
    assert H.call(lib, entry, base, n_seq=0, **none) == 0
    assert H.call(lib, entry, base, n_seq=-1, **none) == -1
    for name in none:
        assert H.call(lib, entry, base, **{name: None}) == -1


@pytest.mark.gpu
def test_binding():
    import torch
    import dynamic_block_sparse_tiled_b200 as bl
    x = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    pool = torch.full((2, 16, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    cu, lens, table = (torch.zeros(*n, dtype=torch.int32, device="cuda") for n in ((1,), (0,), (0, 2)))
    o, lse = bl.attention_paged(x, pool, pool, table, lens, cu)
    assert o.shape == x.shape and lse.shape == (3, 2)
    q = torch.full_like(x, 5.0)
    assert bool((bl.paged_append(x, x, x, pool, pool, table, lens, cu, q_out=q) == 5).all())
    assert bool((pool == 7).all()) and bl.blasst_check() == 0
