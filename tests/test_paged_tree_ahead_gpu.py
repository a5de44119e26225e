"""Trees of drafted tokens under a window that begins ahead of its token (a negative
pre_tokens): the chunk's own keys go by the tree alone, the context is what the
window's formula gives (the sinks).  Against the 64-bit definition
(tests/paged_more_ref.py derives the tolerances)."""
import pytest

from tests.test_paged_more_gpu import check, geometry

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["", "e4m3"])
@pytest.mark.parametrize("sinks", [0, 5])
@pytest.mark.parametrize("pre,nxt", [(-1, 1), (-3, 20), (-5, 5), (-200, 300)])
@pytest.mark.parametrize("q_lens,kv_lens,kw", [
    ([5, 1, 4], [100, 60, 4], dict(N=4, N_kv=1, D=64)),             # few rows
    ([4], [1500], dict(N=4, N_kv=1, D=64, dtype="fp16")),           # a bound for several splits
    ([61, 20], [300, 20], dict(N=8, N_kv=2, D=128)),                # row tiles
    ([140, 3], [400, 90], dict(N=2, N_kv=1, D=72)),                 # both, past a key tile
])
def test_a_tree_whose_window_begins_ahead(q_lens, kv_lens, kw, pre, nxt, sinks, cache):
    geom = geometry(q_lens, kv_lens, 16, sparse_mode=4, pre_tokens=pre, next_tokens=nxt, sink_tokens=sinks, cache_dtype=cache,
                    **kw)
    check(geom, kv_lens, 11, tree=True)
