"""The paged operators where the order of things inside a call, or of calls and
kernels behind one another, carries the result: units of a persistent CTA, the
grids of a mixed batch, calls directly behind the ones that write what they read."""
import pytest
import torch

from attention_swa_forward_gb300 import swa
from tests.paged_ref import DT, assert_within, attention_ref, draw_cache
from tests.test_paged_gpu import geometry

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# More row tiles than SMs, each warp of which has rows past its tile's last:
# a CTA goes from one tile to the next with part of its warps' lanes storing.
RAGGED = {
    "rows_22": ([150] * 8, [150, 400, 151, 300, 0, 220, 33, 600], dict(N=40, N_kv=40, D=128)),
    "rows_1": ([129] * 8, [129, 200, 500, 129, 140, 0, 900, 131], dict(N=44, N_kv=44, D=64, dtype="fp16")),
    "groups_of_3": ([47, 85, 44, 130, 200], [300, 85, 700, 130, 1200], dict(N=96, N_kv=32, D=72)),
    "groups_of_24": ([6, 11, 16, 41, 77, 101, 9, 64] * 3, [60, 11, 500, 900, 77, 0, 30, 2000] * 3,
                     dict(N=96, N_kv=4, D=128, dtype="fp16")),
    "last_round_split": ([1390], [4500], dict(N=16, N_kv=1, D=96)),
}


@pytest.mark.parametrize("name", list(RAGGED))
def test_tiles_whose_warps_are_partly_empty(name):
    q_lens, kv_lens, kw = RAGGED[name]
    geom = geometry(q_lens, kv_lens, 32, sparse_mode=4, next_tokens=0, **kw)
    ks, vs, kp, vp, table, lens = draw_cache(geom, kv_lens, 7, "seen")
    q = torch.randn(geom.T_q, geom.N, geom.D, generator=torch.Generator().manual_seed(8)).to(DT[geom.dtype])
    d = [t.to(DEV) for t in (q, kp, vp, table, lens)]
    ws = swa.paged_forward_workspace(geom, DEV)
    first = swa.paged_forward(geom, *d, workspace=ws)
    swa.check_paged_forward(geom, ws)
    ref, err = attention_ref(geom, q, ks, vs, kv_lens)
    for what, x, r, e in zip(("out", "softmax_max", "softmax_sum"), first, ref, err):
        assert_within(x, r, e, (name, what))
    for _ in range(20):
        again = swa.paged_forward(geom, *d, workspace=ws)
        for a, b in zip(first, again):
            assert torch.equal(a, b)
