"""PagedParams of a caller's own geometry object, with the fields that it had to have
before there were sinks and 8-bit caches (no GPU)."""
import types

import pytest

from attention_swa_forward_gb300 import build as B
from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import PagedGeometry


@pytest.mark.parametrize("n_kv", [0, 2])
def test_sinks_and_the_cache_type_may_be_absent(n_kv):
    B.build()
    g = PagedGeometry(B=2, N=4, N_kv=n_kv, D=64, cu_seqlens_q=[3, 8], num_pages=8, page_size=16, max_pages=4)
    fields = {n: x for n, x in vars(g).items() if n not in ("sink_tokens", "cache_dtype")}
    own = types.SimpleNamespace(T_q=8, **fields)
    p, q = swa.PagedParams(own), swa.PagedParams(g)
    assert (p.c.sink_tokens, p.c.cache_dtype) == (0, 0) and p.kv_shape == q.kv_shape == (8, n_kv or 4, 64)
    assert swa.swa_paged_forward_workspace_size(p) == swa.swa_paged_forward_workspace_size(q)
