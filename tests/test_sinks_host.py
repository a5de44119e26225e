"""Windows with sinks on the CPU: the exported schedule against brute force, the workspace, and refusals."""
import ctypes

import numpy as np
import pytest

from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import Geometry
from tests.sinks_ref import visible

T = 128


def geometries():
    for S_q, S_kv, pre, nxt, sinks in ((1000, 1000, 100, 0, 4), (2000, 2000, 130, 0, 300), (900, 300, 50, 0, 5),
                                       (300, 900, 50, 20, 129), (700, 700, 300, -200, 260), (1, 1, 0, 0, 1),
                                       (1500, 1500, 0, 0, 10 ** 9), (640, 640, -100, 150, 30)):
        for N, N_kv in ((1, 1), (4, 2)):
            yield Geometry("BNSD", 2, N, 64, S_q=S_q, S_kv=S_kv, N_kv=N_kv, sparse_mode=4, pre_tokens=pre,
                           next_tokens=nxt, sink_tokens=sinks)
    lens = [5, 700, 0, 130, 1, 2000]
    ends = np.cumsum(lens).tolist()
    yield Geometry("TND", 6, 2, 64, cu_seqlens_q=ends, cu_seqlens_kv=ends, sparse_mode=4, pre_tokens=64,
                   next_tokens=0, sink_tokens=6)


def touched(seen):
    """[query tiles, key tiles]: does any pair of the two see each other?"""
    q, k = seen.shape
    pad = np.zeros((-(-q // T) * T, -(-k // T) * T), dtype=bool)
    pad[:q, :k] = seen
    return pad.reshape(-(-q // T), T, -(-k // T), T).any(axis=(1, 3))


@pytest.mark.parametrize("g", list(geometries()), ids=lambda g: f"{g.layout}-{g.S_q}-{g.S_kv}-{g.pre_tokens}-{g.sink_tokens}-{g.N}")
def test_schedule_covers_every_visible_pair(g):
    p = swa.Params(g)
    for pass_, heads in ((0, g.N), (1, g.n_kv), (2, g.N)):
        rows = swa.swa_debug_schedule(p, pass_)
        for b, (n_q, n_kv) in enumerate(g.seq_lens()):
            if n_q == 0 or n_kv == 0:
                continue
            need = touched(visible(g, n_q, n_kv).numpy())
            for h in range(heads):
                mine = rows[(rows[:, 1] == b) & (rows[:, 2] == h)]
                got = np.zeros_like(need)
                for _, _, _, tile, first, count in mine:
                    if pass_ == 0:
                        assert not got[tile, first:first + count].any()  # no tile twice
                        got[tile, first:first + count] = True
                    elif pass_ == 1:
                        got[first:first + count, tile] = True
                    else:
                        got[2 * tile:2 * tile + 2, first:first + count] = True
                assert not (need & ~got).any(), (pass_, b, h)
                if pass_ != 2:
                    # no more than the run from the first to the last touched tile, and the sinks
                    extra = got & ~need
                    bound = need.shape[0] * 2 + need.shape[1] * 2
                    assert extra.sum() <= bound


def test_workspace_holds_the_pieces_and_no_more_than_a_few_per_sm():
    base = dict(S_q=32768, S_kv=32768, N_kv=4, scale=0.1, sparse_mode=4, next_tokens=0)
    size = lambda **kw: swa.swa_backward_workspace_size(swa.Params(Geometry("BNSD", 1, 16, 128, **{**base, **kw})))
    plain = size(pre_tokens=4096)
    assert size(pre_tokens=4096, sink_tokens=0) == plain
    with_sinks = size(pre_tokens=4096, sink_tokens=4) - plain
    assert 0 < with_sinks <= 1000 * 131072 and with_sinks % 131072 == 0
    assert size(pre_tokens=4096, sink_tokens=32768) - plain <= 1000 * 131072
    assert size(pre_tokens=0, sink_tokens=32768) - plain <= 1000 * 131072
    assert size(pre_tokens=4096, sink_tokens=4, sparse_mode=0) == plain


def test_refusals():
    g = Geometry("BNSD", 1, 1, 64, S_q=10, S_kv=10, sparse_mode=4, pre_tokens=3, next_tokens=0, sink_tokens=-1)
    with pytest.raises(swa.SwaError) as e:
        swa.swa_forward_workspace_size(swa.Params(g))
    assert e.value.status == swa.SWA_ERR_PARAM_INVALID and "sink_tokens" in str(e.value)
    d = swa.SwaParams()
    swa.lib().swa_params_default(ctypes.byref(d))
    assert d.sink_tokens == 0


def test_the_oracle_refuses_sinks():
    from oracle import swa_oracle as orc

    with pytest.raises(ValueError, match="sinks"):
        orc._Call(orc.Problem("BNSD", 1, 1, 8, S_q=4, S_kv=4, sink_tokens=1))


def test_a_long_run_of_sinks_behind_few_queries():
    """Sinks in every key tile: only the tiles that have many steps are cut."""
    n = 1 << 20
    g = Geometry("TND", 1, 1, 8, cu_seqlens_q=[60000], cu_seqlens_kv=[n], sparse_mode=4, pre_tokens=100, next_tokens=0,
                 sink_tokens=n)
    rows = swa.swa_debug_schedule(swa.Params(g), 1)
    tiles, count = np.unique(rows[:, 3], return_counts=True)
    assert np.array_equal(tiles, np.arange(n // T)) and (np.diff(count) <= 0).all() and count[0] == 2 and count[-1] == 1
    size = lambda sinks: swa.swa_backward_workspace_size(swa.Params(Geometry(**{**g.as_dict(), "sink_tokens": sinks})))
    assert size(n) - size(0) <= 2 * 304 * 65536
