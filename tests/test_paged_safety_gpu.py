"""The paged and rotary operators where they could go wrong without a wrong
number in a plain test: the bounds-checked build, a bounded wait that runs
out, calls on two streams at once, offsets past 32 bits, a replayed graph whose
workspace other calls used in between, and a cache shared by two calls."""
import pytest
import torch

from attention_swa_forward_gb300 import build as B
from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import PagedGeometry, RopeGeometry
from tests.paged_ref import DT, assert_within, attention_ref, draw_cache
from tests.test_paged_gpu import CASES, geometry
from tests.test_rope_gpu import CASES as ROPE_CASES
from tests.test_rope_gpu import draw as rope_draw

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def libs():
    B.build()
    B.build(checked=True)
    return swa.lib(), swa.checked_lib()


def problem(name, seed=31):
    q_lens, kv_lens, page, kw = CASES[name]
    geom = geometry(q_lens, kv_lens, page, **kw)
    if name == "skipped_tail":
        geom.cu_seqlens_q = [1, 301, 0, 0]
    cache = draw_cache(geom, kv_lens, seed, "seen")
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(geom.T_q, n, geom.D, generator=g).to(DT[geom.dtype])
               for n in (geom.N, geom.n_kv, geom.n_kv))
    return geom, kv_lens, cache, q, k, v


def forward(geom, cache, q, **kw):
    _, _, kp, vp, table, lens = cache
    ws = swa.paged_forward_workspace(geom, DEV)
    got = swa.paged_forward(geom, *(t.to(DEV) for t in (q, kp, vp, table, lens)), workspace=ws, **kw)
    return got, ws


@pytest.mark.parametrize("name", list(CASES))
def test_checked_build_stays_in_bounds_and_matches(name, libs):
    geom, kv_lens, cache, q, k, v = problem(name)
    res = []
    for library in libs:
        with swa.using(library):
            got, ws = forward(geom, cache, q)
            swa.check_paged_forward(geom, ws)
            # the chunk appended to copies of the pages (a length below the chunk stores part of it)
            _, _, kp, vp, table, lens = cache
            whole = table.clone()
            free = iter(sorted(set(range(geom.num_pages)) - set(table.flatten().tolist())))
            for b, n in enumerate(kv_lens):
                for e in range(max(0, n - geom.q_lens()[b]) // geom.page_size, -(-n // geom.page_size)):
                    if whole[b, e] < 0:
                        whole[b, e] = next(free)
            dk, dv = kp.to(DEV), vp.to(DEV)
            rope = RopeGeometry("TND", 1, geom.T_q, geom.N, geom.D, N_kv=geom.n_kv, dtype=geom.dtype)
            wa = swa.paged_append_workspace(geom, DEV)
            qo = swa.paged_append(geom, k.to(DEV), v.to(DEV), dk, dv, whole.to(DEV), lens.to(DEV), rope=rope,
                                  q=q.to(DEV), workspace=wa)
            swa.check_paged_append(geom, wa)
            res.append([t.cpu().float() for t in (*got, qo, dk, dv)])
    for a, b in zip(*res):
        assert torch.equal(torch.nan_to_num(a, nan=123.0), torch.nan_to_num(b, nan=123.0)), name


@pytest.mark.parametrize("name", sorted(ROPE_CASES))
def test_checked_rotation_matches(name, libs):
    geom = RopeGeometry(**ROPE_CASES[name])
    q, k, pos = (t.to(DEV) for t in rope_draw(geom, 3))
    res = []
    for library in libs:
        with swa.using(library):
            res.append(swa.rope(geom, q, k, pos))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


@pytest.mark.parametrize("name", ["tokens_ragged", "chunk_mixed", "chunk_window"])
def test_shortened_extents_are_reported(name, libs):
    geom, kv_lens, cache, q, k, v = problem(name)
    release, checked = libs
    for library, want in ((checked, swa.SWA_ERR_BOUNDS), (release, swa.SWA_OK)):
        with swa.using(library):
            swa.swa_debug_extent_slack(8)
            try:
                _, ws = forward(geom, cache, q)
                torch.cuda.synchronize()
            finally:
                swa.swa_debug_extent_slack(0)
            p = swa.PagedParams(geom)
            st = swa.lib().swa_paged_forward_status(p.ref(), ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
            assert st == want
            _, ws = forward(geom, cache, q)
            swa.check_paged_forward(geom, ws)


def test_a_wait_that_runs_out_is_reported():
    """Only the tile kernel waits on barriers: a chunk of more than 16 rows."""
    geom, kv_lens, cache, q, _, _ = problem("chunk_window")
    swa.swa_debug_stall(8)
    try:
        _, ws = forward(geom, cache, q)
        with pytest.raises(swa.SwaError) as e:
            swa.check_paged_forward(geom, ws)
    finally:
        swa.swa_debug_stall(0)
    assert e.value.status == swa.SWA_ERR_TIMEOUT
    got, ws = forward(geom, cache, q)
    swa.check_paged_forward(geom, ws)
    ref, err = attention_ref(geom, q, cache[0], cache[1], kv_lens)
    for x, r, b in zip(got, ref, err):
        assert_within(x, r, b, "after a timeout")


def test_two_streams_at_once_match_serial_calls():
    names = ["chunk_mixed", "token_long_split", "tokens_window", "chunk_split"]
    work, serial = [], []
    for n in names:
        geom, _, cache, q, _, _ = problem(n)
        d = [t.to(DEV) for t in (q, *cache[2:])]
        p = swa.PagedParams(geom)
        ws = [swa.paged_forward_workspace(p, DEV) for _ in range(2)]
        serial.append([t.clone() for t in swa.paged_forward(p, *d, workspace=ws[0])])
        work.append((p, d, ws))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, (p, d, ws) in enumerate(work):
            for s in range(2):
                got[s].append((i, swa.paged_forward(p, *d, workspace=ws[s], stream=streams[s])))
    torch.cuda.synchronize()
    for s in range(2):
        for i, res in got[s]:
            for a, b in zip(res, serial[i]):
                assert torch.equal(a, b)


def test_page_offsets_past_32_bits():
    """Pages 2^31 elements apart (the cache spans more than 2^32 elements)."""
    P, N, N_kv, D = 32, 4, 2, 64
    need = 2 * (1 << 31) + N_kv * P * D
    if torch.cuda.mem_get_info()[0] < 2 * 2 * need + (1 << 30):
        pytest.skip("needs 18 GB of device memory")
    store = [torch.empty(need, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    far = [s.as_strided((3, N_kv, P, D), (1 << 31, P * D, D, 1)) for s in store]
    for q_lens in ([1, 1], [40, 20]):
        geom = PagedGeometry(B=2, N=N, N_kv=N_kv, D=D, cu_seqlens_q=[q_lens[0], sum(q_lens)], num_pages=3, page_size=P,
                             max_pages=2, scale=0.125, sparse_mode=4, next_tokens=0)
        g = torch.Generator().manual_seed(3)
        kv_lens = [60, 25]
        table = torch.tensor([[2, 0], [1, -1]], dtype=torch.int32)
        ks, vs = ([torch.randn(n, N_kv, D, generator=g).bfloat16() for n in kv_lens] for _ in range(2))
        q = torch.randn(geom.T_q, N, D, generator=g).bfloat16()
        for f in far:
            f.fill_(float("nan"))
        # write it all through the append, then read it
        whole = PagedGeometry(B=2, N=N, N_kv=N_kv, D=D, cu_seqlens_q=[60, 85], num_pages=3, page_size=P, max_pages=2)
        lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
        wa = swa.paged_append_workspace(whole, DEV)
        swa.paged_append(whole, torch.cat(ks).to(DEV), torch.cat(vs).to(DEV), *far, table.to(DEV), lens, workspace=wa)
        swa.check_paged_append(whole, wa)
        ws = swa.paged_forward_workspace(geom, DEV)
        got = swa.paged_forward(geom, q.to(DEV), *far, table.to(DEV), lens, workspace=ws)
        swa.check_paged_forward(geom, ws)
        ref, err = attention_ref(geom, q, ks, vs, kv_lens)
        for x, r, b in zip(got, ref, err):
            assert_within(x, r, b, ("far pages", q_lens))


def test_replay_after_other_calls_used_the_workspace():
    """A graph and eager calls share a workspace one after the other."""
    geom, _, cache, q, _, _ = problem("token_long_split")
    p = swa.PagedParams(geom)
    d = [t.to(DEV) for t in (q, *cache[2:])]
    other, _, oc, oq, _, _ = problem("chunk_split")
    size = max(swa.swa_paged_forward_workspace_size(x) for x in (p, swa.PagedParams(other)))
    ws = torch.full((size,), 0x77, dtype=torch.uint8, device=DEV)
    out = [torch.empty_like(d[0]), *(torch.empty(geom.T_q, geom.N, device=DEV) for _ in range(2))]
    want = [t.clone() for t in swa.paged_forward(p, *d, *out, workspace=ws)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        swa.paged_forward(p, *d, *out, workspace=ws)
    for _ in range(3):
        swa.paged_forward(other, *(t.to(DEV) for t in (oq, *oc[2:])), workspace=ws)
        for t in out:
            t.fill_(7.0)
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    swa.check_paged_forward(p, ws)


def test_a_page_shared_by_two_sequences():
    """A prefix page named by two block tables (read only) serves both."""
    geom = geometry([1, 40], [100, 132], 16, N=4, N_kv=2, D=64, sparse_mode=4, next_tokens=0)
    ks, vs, kp, vp, table, lens = draw_cache(geom, [100, 132], 3)
    for e in range(4):
        table[1, e] = table[0, e]
    ks[1][:64], vs[1][:64] = ks[0][:64], vs[0][:64]
    q = torch.randn(41, 4, 64, generator=torch.Generator().manual_seed(2)).bfloat16()
    got, ws = forward(geom, (None, None, kp, vp, table, lens), q)
    swa.check_paged_forward(geom, ws)
    ref, err = attention_ref(geom, q, ks, vs, [100, 132])
    for x, r, b in zip(got, ref, err):
        assert_within(x, r, b, "shared prefix")


@pytest.mark.parametrize("name", ["token_long_split", "tokens_ragged", "chunk_split", "chunk_mixed", "many_tiles",
                                  "many_tiles_fp16", "last_round_split_ragged"])
def test_same_bits_from_run_to_run(name):
    geom, _, cache, q, _, _ = problem(name)
    first, _ = forward(geom, cache, q)
    for _ in range(3):
        again, _ = forward(geom, cache, q)
        for a, b in zip(first, again):
            assert torch.equal(a, b)


def test_a_bad_length_among_many_tiles_harms_no_other():
    geom, kv_lens, cache, q, _, _ = problem("many_tiles")
    good, _ = forward(geom, cache, q)
    lens = cache[5].clone()
    lens[3] = -1
    got, ws = forward(geom, (*cache[:5], lens), q)
    with pytest.raises(swa.SwaError) as e:
        swa.check_paged_forward(geom, ws)
    assert e.value.status == swa.SWA_ERR_PAGE
    a, b = 240, 370  # the fourth sequence's rows
    assert (got[0][a:b] == 0).all() and torch.isneginf(got[1][a:b]).all()
    for x, y in zip(got, good):
        assert torch.equal(x[:a], y[:a]) and torch.equal(x[b:], y[b:])


@pytest.mark.parametrize("q_lens", [[1, 1], [150, 1]])
def test_a_page_number_just_past_the_last(q_lens):
    geom = geometry(q_lens, [200, 90], 16, N=4, N_kv=2, D=64, sparse_mode=4, next_tokens=0)
    _, _, kp, vp, table, lens = draw_cache(geom, [200, 90], 2)
    table[1, 2] = geom.num_pages
    q = torch.randn(geom.T_q, 4, 64).bfloat16()
    got, ws = forward(geom, (None, None, kp, vp, table, lens), q)
    with pytest.raises(swa.SwaError) as e:
        swa.check_paged_forward(geom, ws)
    assert e.value.status == swa.SWA_ERR_PAGE
    assert torch.isfinite(got[0]).all()
