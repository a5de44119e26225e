"""The paged cache on the GPU against 64-bit references (tests/paged_ref.py
states the tolerances): attention of chunks from single tokens up, over pages
in any order, with windows, empty rows, poisoned unused slots, freed pages,
strides and bad tables; the append; and the two together against swa_forward."""
import pytest
import torch

from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import Geometry, PagedGeometry, RopeGeometry
from tests.paged_ref import DT, U, assert_within, attention_ref, draw_cache, rope_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = 2147483647


def geometry(q_lens, kv_lens, page=16, extra_pages=3, **kw):
    cu, e = [], 0
    for n in q_lens:
        e += n
        cu.append(e)
    kw.setdefault("scale", kw["D"] ** -0.5)
    need = sum(-(-n // page) for n in kv_lens)
    return PagedGeometry(B=len(q_lens), cu_seqlens_q=cu, num_pages=need + extra_pages, page_size=page,
                         max_pages=max(1, max(-(-n // page) for n in kv_lens)) + 1, **kw)


def run(geom, q, k_pages, v_pages, table, kv_lens, **kw):
    ws = swa.paged_forward_workspace(geom, DEV)
    ws.fill_(0xA5)
    res = swa.paged_forward(geom, q.to(DEV), k_pages.to(DEV), v_pages.to(DEV), table.to(DEV), kv_lens.to(DEV),
                            workspace=ws, **kw)
    swa.check_paged_forward(geom, ws)
    return res


def check(geom, kv_lens, seed, keys="seen"):
    ks, vs, kp, vp, table, lens = draw_cache(geom, kv_lens, seed, keys)
    q = torch.randn(geom.T_q, geom.N, geom.D, generator=torch.Generator().manual_seed(seed + 1)).to(DT[geom.dtype])
    ref, err = attention_ref(geom, q, ks, vs, kv_lens)
    got = run(geom, q, kp, vp, table, lens)
    for what, x, r, e in zip(("out", "softmax_max", "softmax_sum"), got, ref, err):
        assert_within(x, r, e, (geom, what))


# (q_lens, kv_lens, page, settings)
CASES = {
    "token_1": ([1], [1], 16, dict(N=1, D=64)),
    "token_17": ([1], [17], 16, dict(N=4, N_kv=1, D=128)),
    "tokens_ragged": ([1] * 6, [1, 15, 16, 63, 64, 257], 16, dict(N=8, N_kv=2, D=128, sparse_mode=4, next_tokens=0)),
    "tokens_window": ([1] * 5, [3, 40, 130, 500, 1111], 32, dict(N=4, N_kv=4, D=64, sparse_mode=4, pre_tokens=100,
                                                                next_tokens=0, cache_layout="TND", dtype="fp16")),
    "token_long_split": ([1], [9000], 64, dict(N=8, N_kv=1, D=128)),
    "four_tokens_split": ([4, 4], [5000, 77], 48, dict(N=8, N_kv=2, D=96, sparse_mode=4, next_tokens=0)),
    "group_5": ([3, 1], [70, 333], 16, dict(N=10, N_kv=2, D=40, sparse_mode=4, next_tokens=0, dtype="fp16")),
    "group_16": ([1, 1], [129, 640], 128, dict(N=16, N_kv=1, D=72)),
    "group_24": ([2, 1], [129, 300], 16, dict(N=24, N_kv=1, D=64, sparse_mode=4, next_tokens=0)),
    "chunk_mixed": ([37, 1, 0, 130, 1], [37, 200, 0, 400, 1], 16, dict(N=4, N_kv=2, D=128, sparse_mode=4,
                                                                      next_tokens=0)),
    "chunk_window": ([200, 65], [500, 65], 48, dict(N=3, N_kv=3, D=104, sparse_mode=4, pre_tokens=33, next_tokens=0,
                                                    cache_layout="TND")),
    "chunk_no_mask": ([150], [300], 256, dict(N=2, N_kv=1, D=120, dtype="fp16")),
    "chunk_both_edges": ([129, 7], [260, 7], 16, dict(N=2, N_kv=2, D=64, sparse_mode=4, pre_tokens=20,
                                                      next_tokens=15)),
    "rows_without_keys": ([20, 3], [40, 3], 16, dict(N=2, N_kv=1, D=64, sparse_mode=4, pre_tokens=30,
                                                     next_tokens=-5)),
    "window_ahead": ([40], [60], 16, dict(N=2, N_kv=1, D=32, sparse_mode=4, pre_tokens=-3, next_tokens=9)),
    "length_below_chunk": ([30, 5, 2], [10, 0, 2], 16, dict(N=4, N_kv=2, D=64, sparse_mode=4, pre_tokens=50,
                                                            next_tokens=25)),
    "length_below_chunk_no_mask": ([30, 5], [10, 0], 16, dict(N=4, N_kv=2, D=64)),
    "skipped_tail": ([1, 300, 0, 0], [50, 300, 90, 0], 32, dict(N=4, N_kv=1, D=80, sparse_mode=4, next_tokens=0)),
    "scale_negative": ([1, 140], [77, 140], 16, dict(N=4, N_kv=2, D=64, scale=-0.1, sparse_mode=4, next_tokens=0)),
    "scale_zero": ([1, 20], [77, 20], 16, dict(N=4, N_kv=2, D=64, scale=0.0)),
    "d8": ([1, 140], [40, 140], 16, dict(N=2, N_kv=1, D=8, sparse_mode=4, next_tokens=0)),
    "mqa_48": ([3], [200], 16, dict(N=48, N_kv=1, D=64, sparse_mode=4, next_tokens=0)),
    "mqa_256": ([2], [150], 16, dict(N=256, N_kv=1, D=32, sparse_mode=4, next_tokens=0)),
    "one_page": ([1], [10], 16, dict(N=1, D=64, extra_pages=0)),
    "one_page_chunk": ([10], [14], 16, dict(N=4, N_kv=1, D=64, extra_pages=0, sparse_mode=4, next_tokens=0)),
    "one_long_among_many": ([1] * 40, [20000] + [30] * 39, 64, dict(N=4, N_kv=4, D=16)),
    "page_144": ([1, 150], [1000, 700], 144, dict(N=4, N_kv=2, D=64, sparse_mode=4, next_tokens=0,
                                                  cache_layout="TND")),
    # more row tiles than SMs: a CTA walks several, some without keys
    "many_tiles": ([200, 40, 0, 130, 300, 17], [200, 0, 5, 400, 310, 900], 48,
                   dict(N=48, N_kv=48, D=64, sparse_mode=4, pre_tokens=150, next_tokens=0)),
    "many_tiles_fp16": ([700, 33, 129], [700, 20, 600], 16,
                        dict(N=40, N_kv=8, D=128, dtype="fp16", sparse_mode=4, next_tokens=0, cache_layout="TND")),
    "many_tiles_equal": ([70] * 6, [70, 0, 300, 71, 129, 200], 32, dict(N=32, N_kv=32, D=40)),
    "chunk_split": ([160], [4000], 64, dict(N=2, N_kv=1, D=128, sparse_mode=4, next_tokens=0)),
    # a last round of few row tiles, which are split over their keys
    "last_round_split": ([1300], [4700], 48, dict(N=16, N_kv=1, D=32, sparse_mode=4, next_tokens=0)),
    "last_round_split_ragged": ([33, 1, 1200, 60, 0], [40, 900, 5000, 3, 0], 32,
                                dict(N=16, N_kv=2, D=40, dtype="fp16", sparse_mode=4, pre_tokens=3500, next_tokens=0,
                                     cache_layout="TND")),
    "last_round_split_equal": ([200] * 4, [3200, 190, 2500, 2300], 16, dict(N=40, N_kv=40, D=16)),
}


@pytest.mark.parametrize("name", list(CASES))
def test_attention_matches_the_definition(name):
    q_lens, kv_lens, page, kw = CASES[name]
    cu = geometry(q_lens, kv_lens, page, **kw)
    if name == "skipped_tail":
        cu.cu_seqlens_q = [1, 301, 0, 0]
    check(cu, kv_lens, 11)


def test_many_sequences_of_unequal_chunks():
    """More sequences than one launch's table holds."""
    g = torch.Generator().manual_seed(5)
    q_lens = torch.randint(0, 4, (1100,), generator=g).tolist()
    kv_lens = [n + int(x) for n, x in zip(q_lens, torch.randint(0, 30, (1100,), generator=g))]
    kv_lens[7], q_lens[7] = 900, 40
    check(geometry(q_lens, kv_lens, 16, N=2, N_kv=1, D=16, sparse_mode=4, next_tokens=0), kv_lens, 3)


def test_max_kv_len_changes_the_split_only():
    kv_lens = [3000, 20]
    base = dict(q_lens=[1, 1], kv_lens=kv_lens, page=16, N=4, N_kv=2, D=64)
    for most in (3000, 3008, 0):
        check(geometry(**base, max_kv_len=most), kv_lens, 21)


def test_strided_queries_and_pages():
    """q as a slice of a fused projection; K and V interleaved in one cache."""
    kv_lens, q_lens = [50, 333], [3, 150]
    for layout in ("BNSD", "TND"):
        geom = geometry(q_lens, kv_lens, 32, N=4, N_kv=2, D=72, sparse_mode=4, next_tokens=0, cache_layout=layout)
        ks, vs, kp, vp, table, lens = draw_cache(geom, kv_lens, 2, "seen")
        q = torch.randn(geom.T_q, 4, 72).to(torch.bfloat16)
        ref = run(geom, q, kp, vp, table, lens)
        fused = torch.cat((q, torch.full((geom.T_q, 4, 72), float("nan"), dtype=q.dtype)), dim=1).to(DEV)
        both = torch.stack((kp, vp), dim=1).to(DEV)
        wide = torch.full((2, geom.max_pages + 5), -7, dtype=torch.int32)
        wide[:, :geom.max_pages] = table
        out = swa.paged_forward(geom, fused[:, :4], both[:, 0], both[:, 1], wide.to(DEV)[:, :geom.max_pages],
                                lens.to(DEV))
        for a, b in zip(ref, out):
            assert torch.equal(a, b)
        # heads outermost
        heads_first = q.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
        out = run(geom, heads_first, kp, vp, table, lens)
        for a, b in zip(ref, out):
            assert torch.equal(a, b)


def test_statistics_may_be_left_out():
    geom = geometry([1, 140], [100, 140], 16, N=4, N_kv=2, D=64, sparse_mode=4, next_tokens=0)
    ks, vs, kp, vp, table, lens = draw_cache(geom, [100, 140], 2)
    q = torch.randn(geom.T_q, 4, 64).to(torch.bfloat16)
    ref = run(geom, q, kp, vp, table, lens)[0]
    p, ws, out = swa.PagedParams(geom), swa.paged_forward_workspace(geom, DEV), torch.empty_like(ref)
    d = [t.to(DEV) for t in (q, kp, vp, table, lens)]
    st = swa.lib().swa_paged_forward(p.ref(), d[0].data_ptr(), None, d[1].data_ptr(), None, d[2].data_ptr(), None,
                                     d[3].data_ptr(), 0, d[4].data_ptr(), out.data_ptr(), None, None, ws.data_ptr(),
                                     ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == swa.SWA_OK, swa.swa_last_error()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


def test_a_workspace_in_pieces_is_refused():
    """Its bytes must lie behind one another."""
    geom = geometry([1, 40], [5, 60], 16, N=2, N_kv=1, D=64)
    _, _, kp, vp, table, lens = (x.to(DEV) if torch.is_tensor(x) else x for x in draw_cache(geom, [5, 60], 3))
    q = torch.zeros(geom.T_q, 2, 64, dtype=torch.bfloat16, device=DEV)
    need = swa.swa_paged_forward_workspace_size(swa.PagedParams(geom))
    whole = torch.empty(2 * need, dtype=torch.uint8, device=DEV)
    for ws in (whole[::2], whole[:1].expand(need), whole[:need].cpu()):
        with pytest.raises(ValueError):
            swa.paged_forward(geom, q, kp, vp, table, lens, workspace=ws)
        with pytest.raises(ValueError):
            swa.paged_append(geom, q[:, :1], q[:, :1], kp, vp, table, lens, workspace=ws)


def test_rows_behind_the_outputs_are_left_alone():
    geom = geometry([1, 0, 130], [40, 0, 200], 16, N=4, N_kv=2, D=64, sparse_mode=4, next_tokens=0)
    _, _, kp, vp, table, lens = draw_cache(geom, [40, 0, 200], 2)
    q = torch.randn(geom.T_q, 4, 64).to(torch.bfloat16)
    T = geom.T_q
    out = torch.full((T + 9, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    sm, ss = (torch.full((T + 9, 4), 7.0, device=DEV) for _ in range(2))
    run(geom, q, kp, vp, table, lens, out=out[:T], softmax_max=sm[:T], softmax_sum=ss[:T])
    assert (out[T:] == 7).all() and (sm[T:] == 7).all() and (ss[T:] == 7).all()


def status_of(fn, *a):
    with pytest.raises(swa.SwaError) as e:
        fn(*a)
    return e.value.status


@pytest.mark.parametrize("what,value", [("page", -1), ("page", 10 ** 9), ("length", -3), ("length", 10 ** 6)])
@pytest.mark.parametrize("q_lens", [[1, 1], [150, 1]])
def test_bad_tables_are_reported_and_not_followed(what, value, q_lens):
    kv_lens = [200, 90]
    geom = geometry(q_lens, kv_lens, 16, N=4, N_kv=2, D=64, sparse_mode=4, next_tokens=0)
    ks, vs, kp, vp, table, lens = draw_cache(geom, kv_lens, 2)
    q = torch.randn(geom.T_q, 4, 64).to(torch.bfloat16)
    good = run(geom, q, kp, vp, table, lens)
    if what == "page":
        table[0, 3] = value
    else:
        lens[0] = value
    ws = swa.paged_forward_workspace(geom, DEV)
    d = [t.to(DEV) for t in (q, kp, vp, table, lens)]
    got = swa.paged_forward(geom, *d, workspace=ws)
    assert status_of(swa.check_paged_forward, geom, ws) == swa.SWA_ERR_PAGE
    n = q_lens[0]
    assert torch.equal(got[0][n:], good[0][n:])  # the other sequence is unharmed
    assert torch.isfinite(got[0]).all()
    if what == "length":
        assert (got[0][:n] == 0).all() and torch.isneginf(got[1][:n]).all() and (got[2][:n] == 0).all()
    # the next good call with the workspace reports nothing
    swa.paged_forward(geom, d[0], d[1], d[2], *(t.to(DEV) for t in draw_cache(geom, kv_lens, 2)[4:]), workspace=ws)
    swa.check_paged_forward(geom, ws)


def test_captured_decoding_step_replays_with_grown_lengths():
    """Append and attention of one token, captured once, replayed as the
    sequences grow and their tables change."""
    kv0 = [5, 40, 129, 0]
    geom = PagedGeometry(B=4, N=4, N_kv=2, D=64, cu_seqlens_q=[1, 2, 3, 4], num_pages=64, page_size=16, max_pages=14,
                         scale=0.125, sparse_mode=4, pre_tokens=90, next_tokens=0)
    p = swa.PagedParams(geom)
    kp, vp = (torch.full(geom.page_shape(), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.randperm(64)[:56].view(4, 14).to(torch.int32).to(DEV)
    lens = torch.tensor(kv0, dtype=torch.int32, device=DEV)
    k, v = (torch.randn(4, 2, 64, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(4, 4, 64, device=DEV).to(torch.bfloat16)
    hist = [[(torch.randn(2, 64).to(torch.bfloat16), torch.randn(2, 64).to(torch.bfloat16)) for _ in range(n)]
            for n in kv0]
    for b, h in enumerate(hist):
        for j, (a, c) in enumerate(h):
            kp[table[b, j // 16].item(), :, j % 16], vp[table[b, j // 16].item(), :, j % 16] = a.to(DEV), c.to(DEV)
    wa, wf = swa.paged_append_workspace(p, DEV), swa.paged_forward_workspace(p, DEV)
    out, sm, ss = torch.empty_like(q), *(torch.empty(4, 4, device=DEV) for _ in range(2))

    def step():
        swa.paged_append(p, k, v, kp, vp, table, lens, workspace=wa)
        swa.paged_forward(p, q, kp, vp, table, lens, out, sm, ss, workspace=wf)

    keep = kp.clone(), vp.clone(), lens.clone()
    step()
    torch.cuda.synchronize()
    for t, z in zip((kp, vp, lens), keep):
        t.copy_(z)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lens.add_(1)
        step()
    for turn in range(3):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape).to(torch.bfloat16))
        if turn == 1:  # the window left page 0 of sequence 2 behind: freed
            table[2, 0] = -1
        g.replay()
        torch.cuda.synchronize()
        swa.check_paged_append(p, wa)
        swa.check_paged_forward(p, wf)
        for b in range(4):
            hist[b].append((k[b].cpu(), v[b].cpu()))
        n = [len(h) for h in hist]
        ref, err = attention_ref(geom, q.cpu(), [torch.stack([a for a, _ in h]) for h in hist],
                                 [torch.stack([c for _, c in h]) for h in hist], n)
        for x, r, e in zip((out, sm, ss), ref, err):
            assert_within(x, r, e, ("replay", turn))


# ------------------------------------------------------------------ append --
@pytest.mark.parametrize("rope", [None, "default positions", "three axes"])
@pytest.mark.parametrize("layout,dtype,D,page", [("BNSD", "bf16", 128, 16), ("TND", "fp16", 72, 48)])
def test_append_writes_the_chunk_and_nothing_else(rope, layout, dtype, D, page):
    q_lens, kv_lens = [1, 40, 0, 7, 3], [17, 40, 5, 100, 1]  # (the last: two tokens before its start)
    geom = geometry(q_lens, kv_lens, page, N=6, N_kv=3, D=D, dtype=dtype, cache_layout=layout)
    ks, vs, kp, vp, table, lens = draw_cache(geom, kv_lens, 4)
    T = geom.T_q
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(T, 3, D, generator=g).to(DT[dtype]) for _ in range(2))
    q = torch.randn(T, 6, D, generator=g).to(DT[dtype])
    rg = pos = None
    row_pos = [n - m + i for n, m in zip(kv_lens, q_lens) for i in range(m)]
    row_seq = [b for b, m in enumerate(q_lens) for i in range(m)]
    if rope == "default positions":
        rg = RopeGeometry("TND", 1, T, 6, D, N_kv=3, dtype=dtype)
        at = torch.tensor([[max(x, 0) for x in row_pos]], dtype=torch.int32)
    elif rope:
        rg = RopeGeometry("TND", 1, T, 6, D, N_kv=3, dtype=dtype, sections=[D // 4, 2, D // 4 - 2], rotary_dim=D)
        at = pos = torch.randint(0, 3000, (3, T), generator=g, dtype=torch.int32)
    dk, dv = kp.to(DEV), vp.to(DEV)
    ws = swa.paged_append_workspace(geom, DEV)
    ws.fill_(0x5A)
    q_out = swa.paged_append(geom, k.to(DEV), v.to(DEV), dk, dv, table.to(DEV), lens.to(DEV), rope=rg,
                             positions=None if pos is None else pos.to(DEV), q=q.to(DEV) if rg else None, workspace=ws)
    swa.check_paged_append(geom, ws)
    want_k, err = (k.double(), torch.zeros(k.shape, dtype=torch.float64)) if rg is None else rope_ref(rg, k, at)
    if rg is None:
        assert q_out is None
    else:
        assert_within(q_out, *rope_ref(rg, q, at), "q")
    ref_k, ref_v, ek = kp.double(), vp.double(), torch.zeros(kp.shape, dtype=torch.float64)
    for t, (b, p) in enumerate(zip(row_seq, row_pos)):
        if p < 0:
            continue
        where = (int(table[b, p // page]), slice(None), p % page) if layout == "BNSD" else \
            (int(table[b, p // page]), p % page)
        ref_k[where], ref_v[where], ek[where] = want_k[t], v[t].double(), err[t]
    assert_within(dk, ref_k, ek, "k pages")
    assert_within(dv, ref_v, torch.zeros(()), "v pages")


def test_append_bad_tables_are_reported_and_not_written():
    q_lens, kv_lens = [20, 5], [100, 50]
    geom = geometry(q_lens, kv_lens, 16, N=2, N_kv=2, D=64)
    _, _, kp, vp, table, lens = draw_cache(geom, kv_lens, 4, poison=3.0)
    k, v = (torch.randn(25, 2, 64).to(torch.bfloat16).to(DEV) for _ in range(2))
    ws = swa.paged_append_workspace(geom, DEV)
    bad = table.clone()
    bad[1, 50 // 16 - 1:] = 10 ** 8
    dk, dv = kp.to(DEV), vp.to(DEV)
    swa.paged_append(geom, k, v, dk, dv, bad.to(DEV), lens.to(DEV), workspace=ws)
    assert status_of(swa.check_paged_append, geom, ws) == swa.SWA_ERR_PAGE
    mine = set(table[1, 50 // 16 - 1:].tolist()) - {-1}
    for pg in mine:
        assert torch.equal(dk[pg].cpu(), kp[pg]) and torch.equal(dv[pg].cpu(), vp[pg])
    lens2 = lens.clone()
    lens2[0] = 10 ** 6
    swa.paged_append(geom, k, v, dk, dv, table.to(DEV), lens2.to(DEV), workspace=ws)
    assert status_of(swa.check_paged_append, geom, ws) == swa.SWA_ERR_PAGE
    # pages before the chunk are not looked at
    ok = table.clone()
    ok[0, :80 // 16] = -1
    swa.paged_append(geom, k, v, dk, dv, ok.to(DEV), lens.to(DEV), workspace=ws)
    swa.check_paged_append(geom, ws)


def test_append_many_sequences_and_strides():
    """More sequences than a launch's table holds; k and v as slices of a fused projection."""
    g = torch.Generator().manual_seed(5)
    q_lens = torch.randint(0, 4, (1100,), generator=g).tolist()
    kv_lens = [n + int(x) for n, x in zip(q_lens, torch.randint(0, 30, (1100,), generator=g))]
    geom = geometry(q_lens, kv_lens, 16, N=2, N_kv=2, D=16)
    ks, vs, kp, vp, table, lens = draw_cache(geom, kv_lens, 4, poison=0.0)
    fused = torch.randn(geom.T_q, 4, 16, generator=g).to(torch.bfloat16).to(DEV)
    dk, dv = kp.to(DEV), vp.to(DEV)
    ws = swa.paged_append_workspace(geom, DEV)
    swa.paged_append(geom, fused[:, :2], fused[:, 2:], dk, dv, table.to(DEV), lens.to(DEV), workspace=ws)
    swa.check_paged_append(geom, ws)
    f, row = fused.cpu(), 0
    for b, (n, m) in enumerate(zip(kv_lens, q_lens)):
        for i in range(m):
            p = n - m + i
            kp[int(table[b, p // 16]), :, p % 16], vp[int(table[b, p // 16]), :, p % 16] = f[row, :2], f[row, 2:]
            row += 1
    assert torch.equal(dk.cpu(), kp) and torch.equal(dv.cpu(), vp)


# ------------------------------------------------------------ used together --
def test_prompt_in_chunks_then_tokens_equals_the_dense_forward():
    """Rotate and append a prompt chunk by chunk, attend over the pages, then
    go on token by token: every row agrees with swa_forward on the whole
    rotated sequence under the same window, within both paths' rounding."""
    S, N, N_kv, D, pre = 700, 8, 2, 128, 250
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(S, n, D, generator=g).to(torch.bfloat16).to(DEV) for n in (N, N_kv, N_kv))
    pos = torch.arange(S, dtype=torch.int32, device=DEV)[None]
    rq, rk = swa.rope(RopeGeometry("TND", 1, S, N, D, N_kv=N_kv), q, k, pos)
    dense = Geometry("TND", 1, N, D, cu_seqlens_q=[S], cu_seqlens_kv=[S], N_kv=N_kv, scale=D ** -0.5, sparse_mode=4,
                     pre_tokens=pre, next_tokens=0)
    want = swa.forward(dense, rq, rk, v)
    kp, vp = (torch.full((20, N_kv, 48, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.randperm(20, generator=g)[None, :15].to(torch.int32).to(DEV)
    at = 0
    for m in (300, 150, 240, 1, 1, 1, 4, 3):
        geom = PagedGeometry(B=1, N=N, N_kv=N_kv, D=D, cu_seqlens_q=[m], num_pages=20, page_size=48, max_pages=15,
                             scale=D ** -0.5, sparse_mode=4, pre_tokens=pre, next_tokens=0)
        lens = torch.tensor([at + m], dtype=torch.int32, device=DEV)
        c = slice(at, at + m)
        rot = swa.paged_append(geom, k[c], v[c], kp, vp, table, lens, rope=RopeGeometry("TND", 1, m, N, D, N_kv=N_kv),
                               q=q[c])
        assert torch.equal(rot, rq[c])
        out, sm, ss = swa.paged_forward(geom, rot, kp, vp, table, lens)
        # both paths are within (u + 2 e) of the weighted mean of |v| and a
        # stored output's u, and their scores within e (tests/paged_ref.py)
        size = (rq[c].float().abs().transpose(0, 1) @ rk.float().abs().repeat_interleave(N // N_kv, 1).permute(1, 2, 0))
        e = D * 2.0 ** -23 * size.max() * D ** -0.5 + 2.0 ** -22 * (size.max() * D ** -0.5 + 1)
        assert (out.float() - want[0][c].float()).abs().max() <= 2 * (2 * U["bf16"] + 2 * e) * v.float().abs().max()
        assert (sm - want[1][c]).abs().max() <= 2 * e
        assert ((ss / want[2][c]) - 1).abs().max() <= 2 * (2 * e + S * 2.0 ** -24)
        at += m
    assert at == S


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    """Every parameter drawn at once."""
    g = torch.Generator().manual_seed(100 + seed)
    pick = lambda *x: x[int(torch.randint(0, len(x), (1,), generator=g))]
    num = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    N_kv = pick(1, 2, 3)
    B = num(1, 6)
    q_lens = [pick(0, 1, 1, 2, num(1, 20), num(1, 200)) for _ in range(B)]
    q_lens[num(0, B - 1)] = num(1, 150)
    kv_lens = [max(0, n + pick(0, 0, num(0, 40), num(0, 900)) - pick(0, 0, 0, num(0, 5))) for n in q_lens]
    kw = dict(N=N_kv * pick(1, 2, 3, 4, 5, 8, 16, 17), N_kv=N_kv, D=8 * num(1, 16), dtype=pick("bf16", "fp16"),
              cache_layout=pick("BNSD", "TND"), sparse_mode=pick(0, 4, 4, 4))
    if kw["sparse_mode"] == 4:
        kw.update(pre_tokens=pick(INF, num(0, 300), num(-3, 20)), next_tokens=pick(0, 0, num(3, 40), INF))
    geom = geometry(q_lens, kv_lens, 16 * pick(1, 2, 3, 5, 8, 9), **kw)
    geom.max_kv_len = pick(0, max(max(kv_lens), 1))
    check(geom, kv_lens, seed)
