"""The paged operators where the order of things inside a call, or of calls and
kernels behind one another, carries the result: units of a persistent CTA, the
grids of a mixed batch, calls directly behind the ones that write what they read."""
import pytest
import torch

from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import PagedGeometry, RopeGeometry
from tests.paged_ref import DT, assert_within, attention_ref, draw_cache, rope_ref
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


# ------------------------------------------------- mixed batches of serving --
def batch(live, long, seed, N=4, N_kv=2, D=64, spread=40, **kw):
    """`live` sequences of which the first few have chunks (`long`), the others one
    to three tokens, in an order of their own; some without any in between."""
    g = torch.Generator().manual_seed(seed)
    num = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    q = list(long) + [num(1, 3) for _ in range(live - len(long))] + [0] * 5
    q = [q[i] for i in torch.randperm(len(q), generator=g).tolist()]
    kv = [n + num(0, spread) if n else num(0, 20) for n in q]
    kv[q.index(long[0])] += kw.pop("longest", 0)
    columns = kw.pop("columns", 0)
    geom = geometry(q, kv, 16, N=N, N_kv=N_kv, D=D, sparse_mode=4, next_tokens=0, **kw)
    geom.max_pages = max(columns, geom.max_pages)
    return geom, kv


# ragged batches past the small table (16 sequences) and at the large one's end
# (512), with tiles and few-row items in one call: few tiles, which are split and
# joined; between half the SMs and all; more than SMs, a last round split among
# them; a longer bound on the lengths, so that few-row items are split as well
MIXED = {
    "40_tiles_split": lambda: batch(40, [130, 70], 1, longest=900),
    "40_few_rows_in_clusters": lambda: batch(40, [100], 2, longest=9000, N=2, N_kv=1, D=32),
    "40_few_rows_joined": lambda: batch(40, [100], 2, spread=3000, N=2, N_kv=1, D=32, columns=10000),
    "17_tiles_of_a_round": lambda: batch(17, [300, 120, 90], 3, N=24, N_kv=24, D=72, dtype="fp16"),
    "40_more_tiles_than_SMs": lambda: batch(40, [400, 300, 200, 33], 4, N=32, N_kv=32, D=40, cache_layout="TND"),
    "40_last_round_split": lambda: batch(40, [1250], 5, N=16, N_kv=1, D=32, longest=3400),
    "512_tiles_split": lambda: batch(512, [90, 50, 40], 6, spread=20, N=2, N_kv=1, D=32),
    "512_many_tiles": lambda: batch(512, [260] * 8, 7, spread=20, N=16, N_kv=16, D=16, dtype="fp16"),
    "513_two_tables": lambda: batch(513, [90, 50, 40], 8, spread=20, N=2, N_kv=1, D=32),
}


class Serving:
    """Chunks whose q, k and v are rotated, appended and attended, one call
    directly behind the other on one stream, all on buffers that are reused."""

    def __init__(self, geom, kv, seed):
        self.geom, self.kv, self.p = geom, kv, swa.PagedParams(geom)
        self.rope = swa.RopeParams(RopeGeometry("TND", 1, geom.T_q, geom.N, geom.D, N_kv=geom.n_kv, dtype=geom.dtype))
        g = self.g = torch.Generator().manual_seed(seed)
        ks, vs, kp, vp, table, lens = draw_cache(geom, kv, seed, "all", poison=0.0)
        self.hist = ks, vs
        self.kp, self.vp, self.table, self.lens = (t.to(DEV) for t in (kp, vp, table, lens))
        T, dt = geom.T_q, DT[geom.dtype]
        self.q, self.rq, self.out = (torch.empty(T, geom.N, geom.D, dtype=dt, device=DEV) for _ in range(3))
        self.k, self.v = (torch.empty(T, geom.n_kv, geom.D, dtype=dt, device=DEV) for _ in range(2))
        self.sm, self.ss = (torch.empty(T, geom.N, device=DEV) for _ in range(2))
        self.wa, self.wf = swa.paged_append_workspace(self.p, DEV), swa.paged_forward_workspace(self.p, DEV)

    def feed(self):
        """New tokens of the same chunks."""
        self.new = [torch.randn(t.shape, generator=self.g).to(t.dtype) for t in (self.q, self.k, self.v)]
        for t, x in zip((self.q, self.k, self.v), self.new):
            t.copy_(x, non_blocking=False)

    def step(self):
        swa.paged_append(self.p, self.k, self.v, self.kp, self.vp, self.table, self.lens, rope=self.rope, q=self.q,
                         q_out=self.rq, workspace=self.wa)
        swa.paged_forward(self.p, self.rq, self.kp, self.vp, self.table, self.lens, self.out, self.sm, self.ss,
                          workspace=self.wf)

    def check(self, what):
        torch.cuda.synchronize()
        swa.check_paged_append(self.p, self.wa)
        swa.check_paged_forward(self.p, self.wf)
        lens = self.geom.q_lens()
        pos = torch.tensor([[n - m + i for n, m in zip(self.kv, lens) for i in range(m)]], dtype=torch.int32)
        # the rotated rows as stored (their own rounding is tested elsewhere)
        rq = self.rq.cpu()
        assert_within(rq, *rope_ref(self.rope.geom, self.new[0], pos), (what, "q"))
        rk, _ = swa.rope(RopeGeometry("TND", 1, self.geom.T_q, self.geom.n_kv, self.geom.D, dtype=self.geom.dtype),
                         self.k, None, pos.to(DEV))
        rk, at = rk.cpu(), 0
        for b, (n, m) in enumerate(zip(self.kv, lens)):
            if m:
                self.hist[0][b][n - m:], self.hist[1][b][n - m:] = rk[at:at + m], self.new[2][at:at + m]
            at += m
        ref, err = attention_ref(self.geom, rq, *self.hist, self.kv)
        for name, x, r, e in zip(("out", "softmax_max", "softmax_sum"), (self.out, self.sm, self.ss), ref, err):
            assert_within(x, r, e, (what, name))
        return [t.clone() for t in (self.out, self.sm, self.ss)]


@pytest.mark.parametrize("name", list(MIXED))
def test_mixed_batches_directly_behind_their_append(name):
    geom, kv = MIXED[name]()
    s = Serving(geom, kv, 13)
    for turn in range(2):
        s.feed()
        torch.cuda.synchronize()
        s.step()
        first = s.check((name, turn))
        # the same step again and again, each behind the last on one workspace
        res = []
        for _ in range(12):
            for t in (s.rq, s.out, s.sm, s.ss):
                t.fill_(7.0)
            s.step()
            res.append([t.clone() for t in (s.out, s.sm, s.ss)])
        for again in res:
            for a, b in zip(first, again):
                assert torch.equal(a, b), name


@pytest.mark.parametrize("name", ["40_tiles_split", "40_few_rows_joined", "40_more_tiles_than_SMs", "512_many_tiles"])
def test_captured_mixed_batch_replays_on_new_tokens(name):
    geom, kv = MIXED[name]()
    s = Serving(geom, kv, 17)
    s.feed()
    s.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
        s.step()  # the same again, behind the first's last grid
    for turn in range(3):
        s.feed()
        torch.cuda.synchronize()
        graph.replay()
        first = s.check((name, turn))
        for _ in range(5):
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, (s.out, s.sm, s.ss)):
            assert torch.equal(a, b), name


def test_new_queries_behind_old_ones_in_the_same_buffer():
    """Each call's q is rotated into the buffer that the call before read, with
    nothing else between: the few-row kernel beside the tiles must see it."""
    geom, kv = batch(40, [64, 40], 9, N=8, N_kv=1, D=128)
    s = Serving(geom, kv, 19)
    feeds, want = [], []
    for _ in range(6):
        s.feed()
        s.step()
        want.append(s.check("serial"))
        feeds.append([t.clone() for t in (s.q, s.k, s.v)])
    torch.cuda.synchronize()
    outs = [[torch.empty_like(t) for t in (s.out, s.sm, s.ss)] for _ in feeds]
    for (q, k, v), o in zip(feeds, outs):
        swa.paged_append(s.p, k, v, s.kp, s.vp, s.table, s.lens, rope=s.rope, q=q, q_out=s.rq, workspace=s.wa)
        swa.paged_forward(s.p, s.rq, s.kp, s.vp, s.table, s.lens, *o, workspace=s.wf)
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
