"""Pages, queries and results in orders of memory other than the dense one: the
dense call's bits."""
import pytest
import torch

from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import RopeGeometry
from tests.paged_ref import DT, draw_cache
from tests.test_paged_gpu import geometry

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# few rows; row tiles with the heads of q packed; both
CHUNKS = {"tokens": ([1, 2, 1], [33, 500, 17]), "chunk": ([90], [200]), "mixed": ([140, 1, 3], [140, 260, 50])}
ORDERS = [(0, 1, 2), (0, 2, 1), (1, 0, 2), (1, 2, 0), (2, 0, 1), (2, 1, 0)]  # outermost first


def in_order(t, order, pad=0):
    """t [a, b, c, D] with its first three dimensions laid out in `order`, and `pad` rows between the outermost."""
    shape = [t.shape[i] for i in order]
    store = torch.full((shape[0], shape[1] * shape[2] + pad, t.shape[3]), float("nan"), dtype=t.dtype, device=DEV)
    inner = store[:, :shape[1] * shape[2]].unflatten(1, shape[1:])
    view = inner.permute(*[order.index(i) for i in range(3)], 3)
    view.copy_(t)
    return view, store


@pytest.mark.parametrize("layout", ["BNSD", "TND"])
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("name", list(CHUNKS))
def test_pages_in_any_order(name, order, layout):
    q_lens, kv_lens = CHUNKS[name]
    geom = geometry(q_lens, kv_lens, 48, N=6, N_kv=3, D=72, sparse_mode=4, next_tokens=0, cache_layout=layout)
    _, _, kp, vp, table, lens = draw_cache(geom, kv_lens, 5, "seen")
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(geom.T_q, n, 72, generator=g).bfloat16().to(DEV) for n in (6, 3, 3))
    kp, vp, table, lens = (t.to(DEV) for t in (kp, vp, table, lens))
    ks, k_store = in_order(kp, order)
    # V with a gap behind each outermost entry that keeps each stride a multiple of the next
    vs, v_store = in_order(vp, order, pad=vp.shape[order[2]])
    dense = swa.paged_forward(geom, q, kp, vp, table, lens)
    got = swa.paged_forward(geom, q, ks, vs, table, lens)
    for a, b in zip(dense, got):
        assert torch.equal(a, b)
    # the append to them
    ws = swa.paged_append_workspace(geom, DEV)
    swa.paged_append(geom, k, v, kp, vp, table, lens, workspace=ws)
    swa.check_paged_append(geom, ws)
    swa.paged_append(geom, k, v, ks, vs, table, lens, workspace=ws)
    swa.check_paged_append(geom, ws)
    same = lambda a, b: torch.equal(torch.nan_to_num(a, nan=7.0), torch.nan_to_num(b, nan=7.0))
    assert same(ks, kp) and same(vs, vp)
    assert torch.isnan(v_store[:, -vp.shape[order[2]]:]).all()  # the gaps are untouched


@pytest.mark.parametrize("name", list(CHUNKS))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_queries_with_gaps(name, dtype):
    """Heads apart, rows apart, heads outermost, a row stride that is no multiple
    of the head's: with and without a tensor map for q."""
    q_lens, kv_lens = CHUNKS[name]
    N, D = 6, 64
    geom = geometry(q_lens, kv_lens, 16, N=N, N_kv=2, D=D, sparse_mode=4, next_tokens=0, dtype=dtype)
    _, _, kp, vp, table, lens = (t.to(DEV) if torch.is_tensor(t) else t for t in draw_cache(geom, kv_lens, 5, "seen"))
    T = geom.T_q
    q = torch.randn(T, N, D, generator=torch.Generator().manual_seed(6)).to(DT[dtype]).to(DEV)
    dense = swa.paged_forward(geom, q, kp, vp, table, lens)
    rope = RopeGeometry("TND", 1, T, N, D, N_kv=2, dtype=dtype)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    turned, _ = swa.rope(rope, q, None, pos)
    for row, head in ((N * (D + 8), D + 8), (N * D + 8, D), (2 * N * D, D), (D, T * D), (D + 8, T * (D + 8) + 16),
                      (3 * N * D, 3 * D), (N * D * 8, 8 * D)):
        size = (T - 1) * row + (N - 1) * head + D
        store = torch.full((size + 8,), float("nan"), dtype=q.dtype, device=DEV)
        view = store.as_strided((T, N, D), (row, head, 1))
        view.copy_(q)
        for a, b in zip(dense, swa.paged_forward(geom, view, kp, vp, table, lens)):
            assert torch.equal(a, b), (row, head)
        before = store.clone()
        out, _ = swa.rope(rope, view, None, pos, q_out=view)  # in place
        assert torch.equal(view, turned), (row, head)
        view.copy_(q)
        assert torch.equal(torch.nan_to_num(store, nan=7.0), torch.nan_to_num(before, nan=7.0))  # nothing between


def test_append_rotates_queries_in_place():
    q_lens, kv_lens = CHUNKS["mixed"]
    geom = geometry(q_lens, kv_lens, 16, N=6, N_kv=3, D=72)
    _, _, kp, vp, table, lens = (t.to(DEV) if torch.is_tensor(t) else t for t in draw_cache(geom, kv_lens, 5))
    g = torch.Generator().manual_seed(6)
    fused = torch.randn(geom.T_q, 12, 72, generator=g).bfloat16().to(DEV)  # q, k and v of one projection
    rope = RopeGeometry("TND", 1, geom.T_q, 6, 72, N_kv=3, rotary_dim=40)
    pages = [t.clone() for t in (kp, vp)]
    want = swa.paged_append(geom, fused[:, 6:9], fused[:, 9:], kp, vp, table, lens, rope=rope, q=fused[:, :6])
    keep = fused[:, 6:].clone()
    got = swa.paged_append(geom, fused[:, 6:9], fused[:, 9:], *pages, table, lens, rope=rope, q=fused[:, :6],
                           q_out=fused[:, :6])
    assert got.data_ptr() == fused.data_ptr() and torch.equal(got, want) and torch.equal(fused[:, 6:], keep)
    for a, b in zip(pages, (kp, vp)):
        assert torch.equal(torch.nan_to_num(a, nan=7.0), torch.nan_to_num(b, nan=7.0))
