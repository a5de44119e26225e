"""Sinks, trees of drafted tokens and the 8-bit cache in paged attention, alone and
together, against 64-bit references (tests/paged_more_ref.py); the append to an
8-bit cache and what is read back of it, bit for bit; and a run of them together."""
import pytest
import torch

from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import Geometry, PagedGeometry, RopeGeometry
from tests.paged_more_ref import (LEAST, attention_ref, decode, draw_cache, draw_tree, encode, pack, tree_of)
from tests.paged_ref import DT, assert_within, rope_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def geometry(q_lens, kv_lens, page=16, extra_pages=3, **kw):
    ends = [sum(q_lens[:i + 1]) for i in range(len(q_lens))]
    kw.setdefault("scale", kw["D"] ** -0.5)
    return PagedGeometry(B=len(q_lens), cu_seqlens_q=ends, num_pages=sum(-(-n // page) for n in kv_lens) + extra_pages,
                         page_size=page, max_pages=max(1, max(-(-n // page) for n in kv_lens)) + 1, **kw)


def make(geom, kv_lens, seed, tree=False, words_more=0, spread=0, loud=1.0):
    """Everything a call needs, on the CPU."""
    trees = None
    if tree:
        trees = [tree_of(draw_tree(m, seed + 7 * b)) for b, m in enumerate(geom.q_lens())]
    ks, vs, pages, exps, table, lens = draw_cache(geom, kv_lens, seed, trees, spread)
    q = (torch.randn(geom.T_q, geom.N, geom.D, generator=torch.Generator().manual_seed(seed + 1)) * loud).to(DT[geom.dtype])
    kw = {}
    if geom.cache_dtype:
        kw.update(k_exponents=exps[0], v_exponents=exps[1])
    if tree:
        words = -(-max(geom.q_lens()) // 32) + words_more
        kw["tree"] = torch.cat([pack(see, words) for see, _ in trees if len(see)])
        kw["depth"] = torch.tensor([d for _, depth in trees for d in depth], dtype=torch.int32)
    return dict(ks=ks, vs=vs, pages=pages, table=table, lens=lens, q=q, kw=kw, trees=trees)


def run(geom, p, **more):
    ws = swa.paged_forward_workspace(geom, DEV)
    ws.fill_(0xA5)
    dev = {n: t.to(DEV) for n, t in p["kw"].items()}
    res = swa.paged_forward(geom, p["q"].to(DEV), *[t.to(DEV) for t in p["pages"]], p["table"].to(DEV),
                            p["lens"].to(DEV), workspace=ws, **dev, **more)
    swa.check_paged_forward(geom, ws)
    return res


def check(geom, kv_lens, seed, tree=False, **kw):
    p = make(geom, kv_lens, seed, tree, **kw)
    ref, err = attention_ref(geom, p["q"], p["ks"], p["vs"], kv_lens, p["trees"])
    for what, x, r, e in zip(("out", "softmax_max", "softmax_sum"), run(geom, p), ref, err):
        assert_within(x, r, e, (geom, what))


# (q_lens, kv_lens, page, tree, settings)
W = dict(sparse_mode=4, next_tokens=0)
CASES = {
    # ------------------------------------------------------------- sinks
    "sinks_token": ([1], [500], 16, False, dict(N=4, N_kv=1, D=64, pre_tokens=50, sink_tokens=4, **W)),
    "sinks_tokens_ragged": ([1] * 7, [1, 3, 4, 17, 64, 257, 1000], 16, False,
                            dict(N=8, N_kv=2, D=128, pre_tokens=30, sink_tokens=5, **W)),
    "sinks_fill_groups": ([1, 2], [700, 333], 32, False, dict(N=4, N_kv=2, D=96, pre_tokens=100, sink_tokens=64, **W)),
    "sinks_meet_window": ([1, 1, 1], [100, 120, 140], 16, False, dict(N=2, N_kv=2, D=64, pre_tokens=60, sink_tokens=50, **W)),
    "sinks_same_group": ([1, 1], [60, 61], 16, False, dict(N=2, N_kv=1, D=64, pre_tokens=51, sink_tokens=5, **W)),
    "sinks_past_length": ([1, 1], [30, 200], 16, False, dict(N=2, N_kv=1, D=64, pre_tokens=3, sink_tokens=100000, **W)),
    "sinks_split": ([1], [9000], 64, False, dict(N=8, N_kv=1, D=128, pre_tokens=5000, sink_tokens=200, **W)),
    "sinks_clustered": ([2], [1500], 16, False, dict(N=4, N_kv=4, D=64, pre_tokens=1000, sink_tokens=33, dtype="fp16", **W)),
    "sinks_no_window": ([1, 20], [40, 90], 16, False, dict(N=2, N_kv=1, D=64, sink_tokens=9)),
    "sinks_ahead": ([3, 30], [50, 200], 16, False, dict(N=2, N_kv=1, D=64, pre_tokens=-3, next_tokens=9, sink_tokens=6,
                                                      sparse_mode=4)),
    "sinks_not_reached": ([20, 3], [40, 3], 16, False, dict(N=2, N_kv=1, D=64, pre_tokens=30, next_tokens=-25, sink_tokens=12,
                                                          sparse_mode=4)),
    "sinks_chunk": ([200, 65], [900, 65], 48, False, dict(N=3, N_kv=3, D=104, pre_tokens=33, sink_tokens=4, cache_layout="TND",
                                                         **W)),
    "sinks_chunk_wide": ([150], [2000], 16, False, dict(N=4, N_kv=1, D=128, pre_tokens=256, sink_tokens=300, **W)),
    "sinks_chunk_meets": ([140], [400], 64, False, dict(N=2, N_kv=2, D=64, pre_tokens=130, sink_tokens=200, dtype="fp16", **W)),
    "sinks_chunk_split": ([160], [4000], 64, False, dict(N=2, N_kv=1, D=128, pre_tokens=2500, sink_tokens=130, **W)),
    "sinks_mixed": ([37, 1, 0, 130, 1], [370, 200, 0, 900, 1], 16, False, dict(N=4, N_kv=2, D=128, pre_tokens=64, sink_tokens=17,
                                                                             **W)),
    "sinks_many_tiles": ([700, 33, 129], [2700, 20, 600], 16, False, dict(N=40, N_kv=8, D=64, pre_tokens=300, sink_tokens=4, **W)),
    "sinks_below_chunk": ([30, 5, 2], [10, 0, 2], 16, False, dict(N=4, N_kv=2, D=64, pre_tokens=5, next_tokens=25, sink_tokens=3,
                                                                sparse_mode=4)),
    # ------------------------------------------------------------- trees
    "tree_of_one": ([1, 1], [1, 90], 16, True, dict(N=4, N_kv=1, D=64)),
    "tree_small": ([4, 3, 2], [100, 3, 51], 16, True, dict(N=4, N_kv=1, D=128)),
    "tree_window": ([8, 5], [400, 60], 32, True, dict(N=4, N_kv=4, D=64, pre_tokens=40, dtype="fp16", **W)),
    "tree_window_shorter_than_depth": ([16], [80], 16, True, dict(N=1, D=64, pre_tokens=2, **W)),
    "tree_window_zero": ([12], [80], 16, True, dict(N=1, D=64, pre_tokens=0, **W)),
    "tree_sinks": ([7, 16], [300, 700], 16, True, dict(N=2, N_kv=2, D=128, pre_tokens=50, sink_tokens=4, **W)),
    "tree_61": ([61], [1000], 64, True, dict(N=8, N_kv=2, D=128)),
    "tree_past_a_word": ([33, 32, 31], [50, 32, 200], 16, True, dict(N=16, N_kv=1, D=40, pre_tokens=64, **W)),
    "tree_past_a_tile": ([200, 140], [900, 140], 48, True, dict(N=2, N_kv=1, D=96, pre_tokens=300, sink_tokens=20,
                                                               cache_layout="TND", **W)),
    "tree_unaligned": ([50], [117], 16, True, dict(N=4, N_kv=2, D=64, dtype="fp16")),
    "tree_split": ([61], [6000], 64, True, dict(N=4, N_kv=1, D=128)),
    "tree_few_split": ([4], [9000], 64, True, dict(N=4, N_kv=1, D=64, pre_tokens=8000, **W)),
    "tree_mixed": ([30, 1, 0, 3, 70], [300, 40, 5, 90, 70], 16, True, dict(N=8, N_kv=2, D=64, pre_tokens=64, sink_tokens=3, **W)),
    "tree_below_chunk": ([20, 9, 4], [10, 0, 4], 16, True, dict(N=4, N_kv=2, D=64, pre_tokens=30, **W)),
    "tree_many": ([5] * 40, [20 + 13 * i for i in range(40)], 16, True, dict(N=8, N_kv=8, D=64, pre_tokens=200, **W)),
    # --------------------------------------------------------- 8-bit cache
    "e4m3_token": ([1], [17], 16, False, dict(N=4, N_kv=1, D=128)),
    "e4m3_tokens_ragged": ([1] * 6, [1, 15, 16, 63, 64, 257], 16, False, dict(N=8, N_kv=2, D=128, **W)),
    "e4m3_tokens_fp16": ([1] * 5, [3, 40, 130, 500, 1111], 32, False, dict(N=4, N_kv=4, D=64, pre_tokens=100, dtype="fp16",
                                                                          cache_layout="TND", **W)),
    "e4m3_d8": ([1, 140], [40, 140], 16, False, dict(N=2, N_kv=1, D=8, **W)),
    "e4m3_d24": ([2, 30], [90, 140], 16, False, dict(N=2, N_kv=2, D=24, dtype="fp16")),
    "e4m3_d72": ([3, 100], [500, 300], 48, False, dict(N=4, N_kv=2, D=72, **W)),
    "e4m3_d80_tnd": ([3, 100], [500, 300], 48, False, dict(N=4, N_kv=2, D=80, cache_layout="TND", **W)),
    "e4m3_d104_fp16": ([1, 77], [333, 200], 16, False, dict(N=3, N_kv=3, D=104, dtype="fp16", cache_layout="TND", **W)),
    "e4m3_d40": ([1, 33], [77, 99], 16, False, dict(N=5, N_kv=1, D=40, **W)),
    "e4m3_split": ([1], [9000], 64, False, dict(N=8, N_kv=1, D=128)),
    "e4m3_clustered": ([2], [1500], 16, False, dict(N=4, N_kv=4, D=64, dtype="fp16")),
    "e4m3_chunk": ([130, 300], [400, 310], 64, False, dict(N=4, N_kv=2, D=128, **W)),
    "e4m3_chunk_fp16": ([150], [300], 256, False, dict(N=2, N_kv=1, D=64, dtype="fp16")),
    "e4m3_chunk_window": ([200, 65], [700, 65], 48, False, dict(N=3, N_kv=3, D=96, pre_tokens=33, cache_layout="TND", **W)),
    "e4m3_chunk_split": ([160], [4000], 64, False, dict(N=2, N_kv=1, D=128, **W)),
    "e4m3_many_tiles": ([700, 33, 129], [700, 20, 600], 16, False, dict(N=40, N_kv=8, D=128, dtype="fp16", **W)),
    "e4m3_last_round_split": ([1300], [4700], 48, False, dict(N=16, N_kv=1, D=32, **W)),
    "e4m3_mixed": ([37, 1, 0, 130, 1], [37, 200, 0, 400, 1], 16, False, dict(N=4, N_kv=2, D=128, **W)),
    "e4m3_sinks": ([1, 3, 100], [400, 500, 900], 16, False, dict(N=4, N_kv=2, D=128, pre_tokens=60, sink_tokens=5, **W)),
    "e4m3_tree": ([4, 61, 20], [300, 500, 20], 16, True, dict(N=4, N_kv=2, D=64)),
    "e4m3_tree_sinks": ([4, 61], [300, 800], 32, True, dict(N=8, N_kv=1, D=128, pre_tokens=100, sink_tokens=130, dtype="fp16",
                                                          **W)),
    "e4m3_scale_negative": ([1, 140], [77, 140], 16, False, dict(N=4, N_kv=2, D=64, scale=-0.1, **W)),
    "e4m3_rows_without_keys": ([20, 3], [40, 3], 16, False, dict(N=2, N_kv=1, D=64, sparse_mode=4, pre_tokens=30,
                                                               next_tokens=-5)),
    "e4m3_short_units": ([16 * 9] * 8, [144, 150, 200, 256, 300, 400, 144, 145], 16, False, dict(N=16, N_kv=16, D=64, pre_tokens=3,
                                                                                             **W)),
    "e4m3_short_units_d72": ([144] * 8, [144, 150, 200, 256, 300, 400, 144, 145], 16, False,
                             dict(N=16, N_kv=16, D=72, pre_tokens=3, **W)),
    "e4m3_below_chunk": ([20, 3, 1, 1], [10, 0, 0, 1], 16, False, dict(N=4, N_kv=2, D=64, pre_tokens=5, next_tokens=25,
                                                                     sink_tokens=3, sparse_mode=4)),
    "e4m3_sixteen_rows": ([2, 1, 2], [900, 33, 16], 16, False, dict(N=8, N_kv=1, D=64, pre_tokens=300, sink_tokens=20, **W)),
    "e4m3_sixteen_rows_d120": ([4, 3], [250, 77], 48, False, dict(N=8, N_kv=2, D=120, dtype="fp16", **W)),
    "e4m3_mqa_48": ([3], [200], 16, False, dict(N=48, N_kv=1, D=64, **W)),
}


@pytest.mark.parametrize("name", list(CASES))
def test_attention_matches_the_definition(name):
    q_lens, kv_lens, page, tree, kw = CASES[name]
    check(geometry(q_lens, kv_lens, page, **kw), kv_lens, 11, tree)


@pytest.mark.parametrize("dtype,spread,loud", [("bf16", 25, 1.0), ("bf16", 60, 1.0), ("fp16", 12, 1.0), ("bf16", 6, 1e-20),
                                               ("bf16", 6, 30.0)])
@pytest.mark.parametrize("q_lens,kv_lens,D", [([1, 2], [700, 90], 128), ([140, 40], [700, 90], 128), ([1], [3000], 64),
                                              ([90], [300], 72), ([3], [300], 40)])
def test_rows_of_very_different_size_in_the_8_bit_cache(dtype, spread, loud, q_lens, kv_lens, D):
    """Exponents far apart within a tile and from tile to tile, rows of zeros, queries of any size."""
    geom = geometry(q_lens, kv_lens, 16, N=4, N_kv=2, D=D, dtype=dtype, cache_dtype="e4m3",
                    scale=D ** -0.5 * (1e20 if loud < 1e-9 else 1.0), **W)
    check(geom, kv_lens, 17, spread=spread, loud=loud)


@pytest.mark.parametrize("q_len", [1, 150])
def test_a_key_without_values_may_have_all_the_weight(q_len):
    """A first key that every query prefers, with a row of zeros for its values, among keys with large ones."""
    n = 500
    geom = geometry([q_len], [n], 16, N=2, N_kv=1, D=64, cache_dtype="e4m3", **W)
    p = make(geom, [n], 8)
    k, v = p["ks"][0].clone(), p["vs"][0].clone()
    k[0] = 0.6
    p["q"] = (p["q"].float().abs() + 1.0).to(p["q"].dtype)
    v[0] = 0.0
    v[-3:] *= 64.0
    for x, t in enumerate((k, v)):
        codes, e = encode(t, "bf16")
        for j in range(n):
            page, slot = int(p["table"][0, j // 16]), j % 16
            p["pages"][x].view(torch.uint8)[page, :, slot] = codes[j].view(torch.uint8)
            p["kw"][("k_exponents", "v_exponents")[x]][page, :, slot] = e[j]
        p["ks" if x == 0 else "vs"] = [decode(codes, e)]
    ref, err = attention_ref(geom, p["q"], p["ks"], p["vs"], [n])
    assert (ref[2] < 6.0).all()  # (a good part of the weight is on it)
    for what, x, r, e in zip(("out", "softmax_max", "softmax_sum"), run(geom, p), ref, err):
        assert_within(x, r, e, what)


def test_more_sequences_than_a_table_holds():
    g = torch.Generator().manual_seed(5)
    q_lens = torch.randint(0, 4, (1100,), generator=g).tolist()
    kv_lens = [n + int(x) for n, x in zip(q_lens, torch.randint(0, 30, (1100,), generator=g))]
    kv_lens[7], q_lens[7] = 900, 40
    for tree, cache in ((True, ""), (False, "e4m3")):
        check(geometry(q_lens, kv_lens, 16, N=2, N_kv=1, D=16, pre_tokens=20, sink_tokens=3, cache_dtype=cache, **W),
              kv_lens, 3, tree)


def test_a_tree_that_is_a_line_is_the_causal_chunk():
    """Bit for bit: the same keys in the same order."""
    for q_lens, kv_lens, kw in (([4, 4], [90, 70], dict(N=4, N_kv=1, D=64)),
                                ([100], [350], dict(N=4, N_kv=2, D=128, pre_tokens=4000, sink_tokens=1))):
        geom = geometry(q_lens, kv_lens, 16, sparse_mode=4, next_tokens=0, **kw)
        p = make(geom, kv_lens, 5)
        ref = run(geom, p)
        lines = [torch.tril(torch.ones(m, m, dtype=torch.bool)) for m in q_lens]
        p["kw"]["tree"] = torch.cat([pack(x, -(-max(q_lens) // 32)) for x in lines])
        for depth in (None, torch.tensor([i for m in q_lens for i in range(m)], dtype=torch.int32)):
            if depth is not None:
                p["kw"]["depth"] = depth
            for a, b in zip(ref, run(geom, p)):
                assert torch.equal(a, b)


def test_rows_that_see_nothing_and_depths_outside():
    """An empty row of the tree still sees its context; with no context, nothing."""
    geom = geometry([6, 6, 60], [6, 40, 60], 16, N=2, N_kv=1, D=64)
    p = make(geom, [6, 40, 60], 2, True)
    trees = []
    for b, m in enumerate((6, 6, 60)):
        see = torch.rand(m, m, generator=torch.Generator().manual_seed(b)) < 0.4  # any rows at all, later tokens too
        see[0], see[m // 2] = False, False
        trees.append((see, [0] * m))
    p["trees"] = trees
    p["kw"]["tree"] = torch.cat([pack(see, 2) for see, _ in trees])
    p["kw"]["depth"] = torch.zeros(72, dtype=torch.int32)
    ref, err = attention_ref(geom, p["q"], p["ks"], p["vs"], [6, 40, 60], trees)
    for x, r, e in zip(run(geom, p), ref, err):
        assert_within(x, r, e, "any tree")
    assert torch.isinf(ref[1][0]).all() and torch.isinf(ref[1][12 + 30]).all()
    # depths are held within the chunk
    geom = geometry([5], [50], 16, N=2, N_kv=1, D=64, pre_tokens=10, **W)
    p = make(geom, [50], 3, True)
    see = p["trees"][0][0]
    p["kw"]["depth"] = torch.tensor([-7, 2 ** 31 - 1, -2 ** 31, 3, 9], dtype=torch.int32)
    ref, err = attention_ref(geom, p["q"], p["ks"], p["vs"], [50], [(see, [0, 4, 0, 3, 4])])
    for x, r, e in zip(run(geom, p), ref, err):
        assert_within(x, r, e, "depths")


def test_strides():
    """Pages of K and V side by side with gaps, a tree with longer rows, q as a slice."""
    for cache in ("", "e4m3"):
        for layout in ("BNSD", "TND"):
            kv_lens = [50, 333]
            geom = geometry([3, 60], kv_lens, 32, N=4, N_kv=2, D=72, pre_tokens=90, sink_tokens=3, cache_layout=layout,
                            cache_dtype=cache, **W)
            p = make(geom, kv_lens, 2, True)
            ref = run(geom, p)
            as_bytes = (lambda t: t.view(torch.uint8)) if cache else (lambda t: t)
            both = torch.stack([as_bytes(t) for t in p["pages"]], dim=1).to(DEV)
            wide = torch.cat((both, both), dim=-1)[..., :72]
            dt = p["pages"][0].dtype
            pages = [wide[:, x].view(dt) if not cache else wide[:, x].view(torch.float8_e4m3fn) for x in range(2)]
            fused = torch.cat((p["q"], p["q"]), dim=1).to(DEV)
            kw = {n: t.to(DEV) for n, t in p["kw"].items()}
            kw["tree"] = torch.cat((kw["tree"], torch.full((63, 3), -1, dtype=torch.int32, device=DEV)), dim=1)
            for tree in (kw["tree"], kw["tree"][:, :2]):
                kw["tree"] = tree
                out = swa.paged_forward(geom, fused[:, :4], *pages, p["table"].to(DEV), p["lens"].to(DEV), **kw)
                for a, b in zip(ref, out):
                    assert torch.equal(a, b)


# ------------------------------------------------------------ 8-bit cache --
def empty_cache(geom):
    pages = [torch.full(geom.page_shape(), 0x55, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
    exps = [torch.full(geom.exponent_shape(), 0x55, dtype=torch.int8, device=DEV) for _ in range(2)]
    return pages, exps


def chunk_pages(geom, kv_lens, seed):
    order = torch.randperm(geom.num_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((geom.B, geom.max_pages), -1, dtype=torch.int32)
    for b, n in enumerate(kv_lens):
        for e in range(-(-n // geom.page_size)):
            table[b, e] = order.pop()
    return table.to(DEV), torch.tensor(kv_lens, dtype=torch.int32, device=DEV)


APPENDS = {
    "bf16": ([1, 5, 0, 40], [30, 5, 7, 100], 16, dict(N=2, D=128)),
    "fp16_tnd": ([3, 70], [90, 70], 48, dict(N=4, N_kv=4, D=96, dtype="fp16", cache_layout="TND")),
    "d8": ([7], [9], 16, dict(N=3, D=8)),
    "d24": ([7, 2], [9, 2], 16, dict(N=3, D=24, dtype="fp16")),
    "d40_tnd": ([17, 2], [90, 2], 16, dict(N=5, D=40, cache_layout="TND")),
    "d72": ([17, 2], [90, 2], 16, dict(N=2, D=72)),
    "d120": ([9, 9, 9], [9, 10, 11], 32, dict(N=1, D=120)),
    "equal_tokens": ([1] * 64, list(range(1, 65)), 16, dict(N=8, D=64)),
    "many": ([300, 1200], [300, 5000], 64, dict(N=2, D=128, dtype="fp16")),
    "below_chunk": ([9, 4], [5, 0], 16, dict(N=2, D=64)),
}


@pytest.mark.parametrize("name", list(APPENDS))
def test_append_quantises_by_the_rule_and_reads_back(name):
    """Codes, exponents and the values read back are exact; other slots are left alone."""
    q_lens, kv_lens, page, kw = APPENDS[name]
    geom = geometry(q_lens, kv_lens, page, cache_dtype="e4m3", **kw)
    g = torch.Generator().manual_seed(3)
    rows = [torch.randn(geom.T_q, geom.n_kv, geom.D, generator=g) for _ in range(2)]
    # rows of every size, with what rounds to either side, subnormal codes, zeros, and the largest values
    sizes = torch.pow(2.0, torch.randint(-24, 14, (geom.T_q, geom.n_kv, 1), generator=g).float())
    rows = [(r * sizes).to(DT[geom.dtype]) for r in rows]
    rows[0][0] = 0
    rows[0][-1, 0, :4] = torch.tensor([65504.0, -65504.0, 1.0, 2.0 ** -14]).to(DT[geom.dtype])
    rows[1][0, 0, :3] = torch.tensor([448.0, 0.4375, 2.0 ** -9]).to(DT[geom.dtype])
    table, lens = chunk_pages(geom, kv_lens, 1)
    pages, exps = empty_cache(geom)
    ws = swa.paged_append_workspace(geom, DEV)
    ws.fill_(0xA5)
    dev = [r.to(DEV) for r in rows]
    swa.paged_append(geom, *dev, *pages, table, lens, workspace=ws, k_exponents=exps[0], v_exponents=exps[1])
    swa.check_paged_append(geom, ws)
    want_pages, want_exps = [t.cpu() for t in empty_cache(geom)[0]], [t.cpu() for t in empty_cache(geom)[1]]
    values = [torch.zeros(geom.T_q, geom.n_kv, geom.D, dtype=torch.float64) for _ in range(2)]
    t = 0
    for b, (n, m) in enumerate(zip(kv_lens, q_lens)):
        for i in range(m):
            j = n - m + i
            for x in range(2):
                codes, e = encode(rows[x][t], geom.dtype)
                if j >= 0:
                    p, slot = int(table[b, j // page]), j % page
                    at = (p, slice(None), slot) if geom.cache_layout == "BNSD" else (p, slot)
                    want_pages[x].view(torch.uint8)[at] = codes.view(torch.uint8)
                    want_exps[x][p, :, slot] = e
                    values[x][t] = decode(codes, e)
            t += 1
    for x in range(2):
        # (a zero keeps its sign in a code)
        assert torch.equal(pages[x].cpu().view(torch.uint8), want_pages[x].view(torch.uint8)), x
        assert torch.equal(exps[x].cpu(), want_exps[x]), x
    ws.fill_(0xA5)
    back = swa.paged_gather(geom, *pages, table, lens, workspace=ws, k_exponents=exps[0], v_exponents=exps[1])
    swa.check_paged_append(geom, ws)
    for x in range(2):
        assert torch.equal(back[x].cpu().double(), values[x]), x
        # half a step of a code, 2^-4 of the value, or of the smallest code
        e = encode(rows[x], geom.dtype)[1].double()[..., None]
        far = rows[x].double().abs().clamp(max=57344.0)
        off = (values[x] - rows[x].double().clamp(-57344, 57344)).abs()
        stored = (values[x] != 0).any(-1, keepdim=True)
        assert (off <= torch.maximum(2.0 ** -4 * far, 2.0 ** (e - 10)))[stored.expand_as(off)].all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("cache", ["", "e4m3"])
def test_gather_of_whole_sequences_with_strides(dtype, cache):
    kv_lens = [100, 1, 0, 333]
    geom = geometry(kv_lens, kv_lens, 16, N=3, D=40, dtype=dtype, cache_dtype=cache)
    p = make(geom, kv_lens, 4)
    kw = {n: t.to(DEV) for n, t in p["kw"].items()}
    both = torch.full((geom.T_q, 6, 40), 7.0, dtype=DT[dtype], device=DEV)
    k, v = swa.paged_gather(geom, *[t.to(DEV) for t in p["pages"]], p["table"].to(DEV), p["lens"].to(DEV), k=both[:, 0:3],
                            v=both[:, 3:6], **kw)
    assert torch.equal(k.cpu().double(), torch.cat(p["ks"])) and torch.equal(v.cpu().double(), torch.cat(p["vs"]))


@pytest.mark.parametrize("rotary", [0, 48, 64])
@pytest.mark.parametrize("fused", [False, True])
def test_append_of_heads_first_rows(rotary, fused):
    """K, V and Q whose tokens are nearer than their heads: the same codes as of packed rows."""
    q_lens, kv_lens, N, N_kv, D = [5, 37, 1], [9, 60, 1], 6, 3, 64
    geom = geometry(q_lens, kv_lens, 16, N=N, N_kv=N_kv, D=D, cache_dtype="e4m3")
    rope = RopeGeometry("TND", 1, geom.T_q, N, D, N_kv=N_kv, rotary_dim=rotary) if rotary else None
    if fused and not rotary:
        return
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn(n, geom.T_q, D, generator=g).bfloat16().to(DEV) for n in (N, N_kv, N_kv))
    table, lens = chunk_pages(geom, kv_lens, 2)
    results = []
    for first in (lambda t: t.transpose(0, 1), lambda t: t.transpose(0, 1).contiguous()):
        pages, exps = empty_cache(geom)
        kw = dict(k_exponents=exps[0], v_exponents=exps[1], rope=rope)
        if fused:
            kw["q"] = first(q)
        out = swa.paged_append(geom, first(k), first(v), *pages, table, lens, **kw)
        results.append([t.view(torch.uint8) for t in pages] + exps + ([out] if fused else []))
    for x, y in zip(*results):
        assert torch.equal(x, y)


def test_offsets_past_32_bits():
    """Codes behind 2^32: append, gather and both kernels give what they give near the start."""
    q_lens, kv_lens, N_kv, D, P = [1, 70], [300, 200], 8, 128, 256
    geom = geometry(q_lens, kv_lens, P, N=16, N_kv=N_kv, D=D, cache_dtype="e4m3", **W)
    whole = geometry(kv_lens, kv_lens, P, N=16, N_kv=N_kv, D=D, cache_dtype="e4m3")
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(whole.T_q, N_kv, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    q = torch.randn(geom.T_q, 16, D, generator=g).bfloat16().to(DEV)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
    results = []
    for num_pages, first in ((8, 0), (17000, 16990)):  # 4.46 GB of codes each
        geom.num_pages = whole.num_pages = num_pages
        table = torch.full((2, geom.max_pages), -1, dtype=torch.int32)
        table[0, :2], table[1, 0] = torch.tensor([first + 3, first]), first + 2
        table = table.to(DEV)
        pages = [torch.empty(geom.page_shape(), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
        exps = [torch.empty(geom.exponent_shape(), dtype=torch.int8, device=DEV) for _ in range(2)]
        kw = dict(k_exponents=exps[0], v_exponents=exps[1])
        swa.paged_append(whole, k, v, *pages, table, lens, **kw)
        results.append([*swa.paged_gather(whole, *pages, table, lens, **kw), *swa.paged_forward(geom, q, *pages, table, lens, **kw)])
        del pages, exps
    for x, y in zip(*results):
        assert torch.equal(x, y)


def test_special_values():
    """NaN rows come back as NaN and reach the queries that see them; infinities saturate."""
    for dtype in ("bf16", "fp16"):
        geom = geometry([4], [40], 16, N=1, D=64, dtype=dtype, cache_dtype="e4m3")
        rows = [torch.randn(4, 1, 64).to(DT[dtype]) for _ in range(2)]
        rows[0][1, 0, 5] = float("nan")
        rows[1][2, 0, 7], rows[1][2, 0, 8] = float("inf"), -float("inf")
        table, lens = chunk_pages(geom, [40], 1)
        pages, exps = empty_cache(geom)
        kw = dict(k_exponents=exps[0], v_exponents=exps[1])
        swa.paged_append(geom, *[r.to(DEV) for r in rows], *pages, table, lens, **kw)
        k, v = swa.paged_gather(geom, *pages, table, lens, **kw)
        assert torch.isnan(k[1]).all() and not torch.isnan(k[[0, 2, 3]]).any()
        assert v[2, 0, 7] == 57344.0 and v[2, 0, 8] == -57344.0 and not torch.isnan(v).any()
        for q_len in (1, 40):  # both kernels: the chunk's 40 tokens now the whole sequence
            whole = geometry([q_len], [40], 16, N=1, D=64, dtype=dtype, cache_dtype="e4m3", sparse_mode=4, next_tokens=0,
                             pre_tokens=50)
            swa.paged_append(geometry([36], [36], 16, N=1, D=64, dtype=dtype, cache_dtype="e4m3", extra_pages=3),
                             *[torch.randn(36, 1, 64).to(DT[dtype]).to(DEV) for _ in range(2)], *pages, table, lens - 4, **kw)
            out = swa.paged_forward(whole, torch.randn(q_len, 1, 64).to(DT[dtype]).to(DEV), *pages, table, lens, **kw)[0]
            assert torch.isnan(out[-1]).all()
            if q_len == 40:  # (a NaN that one query of a chunk sees may reach its others)
                assert torch.isnan(out[37:]).all()


def test_rotation_on_the_way_into_the_8_bit_cache():
    """K rotated in fp32 and rounded once to a code; q rotated as without the cache."""
    for dtype, D, R, il in (("bf16", 128, 128, False), ("fp16", 96, 48, True), ("bf16", 72, 72, False), ("fp16", 64, 32, False)):
        q_lens, kv_lens = [20, 1, 33], [50, 9, 33]
        geom = geometry(q_lens, kv_lens, 16, N=4, N_kv=2, D=D, dtype=dtype, cache_dtype="e4m3")
        rope = RopeGeometry("TND", 1, geom.T_q, 4, D, N_kv=2, rotary_dim=R, interleaved=il, dtype=dtype)
        g = torch.Generator().manual_seed(6)
        k, v = (torch.randn(geom.T_q, 2, D, generator=g).to(DT[dtype]) for _ in range(2))
        q = torch.randn(geom.T_q, 4, D, generator=g).to(DT[dtype])
        table, lens = chunk_pages(geom, kv_lens, 1)
        pages, exps = empty_cache(geom)
        kw = dict(k_exponents=exps[0], v_exponents=exps[1])
        q_out = swa.paged_append(geom, k.to(DEV), v.to(DEV), *pages, table, lens, rope=rope, q=q.to(DEV), **kw)
        pos = torch.cat([torch.arange(n - m, n) for n, m in zip(kv_lens, q_lens)]).to(torch.int32)[None]
        kb, vb = swa.paged_gather(geom, *pages, table, lens, **kw)
        assert torch.equal(q_out, swa.rope(rope, q.to(DEV), None, pos.to(DEV))[0])
        y, _ = rope_ref(rope, k, pos)
        err = 2.0 ** -21 * 2 * k.double().abs().amax(-1, keepdim=True)  # of the rotation in fp32 (tests/paged_ref.py)
        e = encode(y, dtype)[1].double()[..., None]
        # half a step of a code, whichever exponent the row got of two next to a border
        assert_within(kb, y, err + torch.maximum(2.0 ** -4 * (y.abs() + err), 2.0 ** (e - 9)), "rotated k")
        assert torch.equal(vb.cpu().double(), decode(*encode(v, dtype)))


def test_16_bit_gather_returns_what_append_stored():
    geom = geometry([30, 2, 500], [90, 2, 700], 16, N=2, D=72, cache_layout="TND")
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(geom.T_q, 2, 72, generator=g).bfloat16().to(DEV) for _ in range(2))
    table, lens = chunk_pages(geom, [90, 2, 700], 1)
    pages = [torch.zeros(geom.page_shape(), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    swa.paged_append(geom, k, v, *pages, table, lens)
    kb, vb = swa.paged_gather(geom, *pages, table, lens)
    assert torch.equal(k, kb) and torch.equal(v, vb)


# --------------------------------------------------------------- together --
@pytest.mark.parametrize("cache", ["", "e4m3"])
def test_serving_a_conversation(cache):
    """A prompt, drafted trees of which a path is accepted, and single tokens, under a
    window with sinks: the accepted tokens' results are those of the dense forward
    over the whole sequence (16-bit cache) or over the values that the cache holds."""
    N, N_kv, D, pre, sinks, total = 4, 2, 64, 40, 4, 260
    g = torch.Generator().manual_seed(1)
    x = [torch.randn(total, n, D, generator=g).bfloat16().to(DEV) for n in (N, N_kv, N_kv)]
    rope = lambda n: RopeGeometry("TND", 1, n, N, D, N_kv=N_kv)
    kw = dict(num_pages=20, page_size=16, max_pages=18, N=N, N_kv=N_kv, D=D, scale=0.125, sparse_mode=4, pre_tokens=pre,
              next_tokens=0, sink_tokens=sinks, cache_dtype=cache)
    plan = lambda m: PagedGeometry(B=1, cu_seqlens_q=[m], **kw)
    dt = torch.float8_e4m3fn if cache else torch.bfloat16
    pages = [torch.zeros(plan(1).page_shape(), device=DEV).to(dt) for _ in range(2)]
    exps = dict(k_exponents=None, v_exponents=None)
    if cache:
        exps = {n: torch.zeros(plan(1).exponent_shape(), dtype=torch.int8, device=DEV) for n in exps}
    table = torch.randperm(20, generator=g)[None, :18].to(torch.int32).to(DEV)
    got, at = [], 0

    def step(rows, kept, tree=None, depth=None):
        """Append and attend with these rows of x at the end; keep the results of `kept` of them."""
        nonlocal at
        m = len(rows)
        lens = torch.tensor([at + m], dtype=torch.int32, device=DEV)
        q, k, v = (t[rows].contiguous() for t in x)
        pos = at + (torch.arange(m) if depth is None else depth)
        q = swa.paged_append(plan(m), k, v, *pages, table, lens, rope=rope(m), positions=pos.to(torch.int32)[None].to(DEV),
                             q=q, **exps)
        more = {} if tree is None else dict(tree=tree.to(DEV), depth=depth.to(torch.int32).to(DEV))
        out = swa.paged_forward(plan(m), q, *pages, table, lens, **exps, **more)[0]
        got.append(out[kept])
        if tree is not None:  # the accepted path once more, in its order
            lens = torch.tensor([at + len(kept)], dtype=torch.int32, device=DEV)
            path = [rows[i] for i in kept]
            k, v = (t[path].contiguous() for t in x[1:])
            pos = (at + torch.arange(len(kept))).to(torch.int32)[None].to(DEV)
            swa.paged_append(plan(len(kept)), k, v, *pages, table, lens, rope=rope(len(kept)), positions=pos, **exps)
        at += len(kept)

    step(list(range(100)), list(range(100)))
    r = torch.Generator().manual_seed(2)
    while at < total - 30:
        m = int(torch.randint(3, 20, (1,), generator=r))
        parents = draw_tree(m, at)
        see, depth = tree_of(parents)
        leaf = int(torch.randint(0, m, (1,), generator=r))
        path = see[leaf].nonzero()[:, 0].tolist()
        rows = [total - 1 - i % 20 for i in range(m)]  # rejected drafts: other tokens' rows
        for place, i in enumerate(path):
            rows[i] = at + place
        step(rows, path, pack(see, 1), torch.tensor(depth))
        step([at], [0])
    lens = torch.tensor([at], dtype=torch.int32, device=DEV)
    k, v = swa.paged_gather(PagedGeometry(B=1, cu_seqlens_q=[at], **kw), *pages, table, lens, **exps)
    pos = torch.arange(at, dtype=torch.int32, device=DEV)[None]
    rq, rk = swa.rope(rope(at), x[0][:at].contiguous(), x[1][:at].contiguous(), pos)
    if not cache:
        assert torch.equal(k, rk) and torch.equal(v, x[2][:at])
    dense = swa.forward(Geometry("TND", 1, N, D, N_kv=N_kv, cu_seqlens_q=[at], cu_seqlens_kv=[at], scale=0.125, sparse_mode=4,
                                 pre_tokens=pre, next_tokens=0, sink_tokens=sinks), rq, k, v)[0]
    out = torch.cat(got).float()
    # two evaluations, each within the roundings of P and of the result (2^-8 each) of |values| that reach 4.5
    assert (out - dense.float()).abs().max() <= 2 * 2 * 2.0 ** -8 * v.float().abs().max()
    assert (out - dense.float()).norm() <= 6e-3 * dense.float().norm()


# ----------------------------------------------------------------- safety --
def test_unpacked_pages_in_passes():
    """Bounds on the lengths whose 16-bit pages do not fit the workspace at once: some sequences after the others."""
    q_lens, kv_lens = [40, 30, 1, 50, 33], [300, 90, 40, 200, 33]
    geom = geometry(q_lens, kv_lens, 16, N=8, N_kv=8, D=128, cache_dtype="e4m3", sparse_mode=4, next_tokens=0)
    geom.max_pages = 131072 // 16
    assert swa.swa_paged_forward_workspace_size(swa.PagedParams(geom)) < (1 << 30) + (64 << 20)
    check(geom, kv_lens, 9)
    check(geometry(q_lens, kv_lens, 16, N=8, N_kv=8, D=128, cache_dtype="e4m3", max_kv_len=300, **W), kv_lens, 9)


def test_the_largest_bound_on_the_lengths():
    """2^28 keys: runs of keys so long that a grid holds them."""
    geom = geometry([2], [500], 65536, N=1, D=16, cache_dtype="e4m3")
    geom.max_pages = (1 << 28) // 65536
    check(geom, [500], 12)


def guarded(call):
    """Status that `call` raises, or None."""
    try:
        call()
    except swa.SwaError as e:
        return e.status
    return None


@pytest.mark.parametrize("name", ["sinks_mixed", "tree_mixed", "e4m3_mixed", "e4m3_tree_sinks", "e4m3_d72", "e4m3_sinks",
                                  "tree_past_a_tile", "e4m3_split", "e4m3_chunk_split"])
def test_bounds_checked_build_gives_the_same_bits(name):
    q_lens, kv_lens, page, tree, kw = CASES[name]
    if name.startswith("e4m3"):
        kw = dict(kw, cache_dtype="e4m3")
    geom = geometry(q_lens, kv_lens, page, **kw)
    p = make(geom, kv_lens, 11, tree)
    ref = run(geom, p)
    with swa.using(swa.checked_lib()):
        got = run(geom, p)  # (raises where an access was skipped)
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cache", ["", "e4m3"])
@pytest.mark.parametrize("q_len", [1, 4, 60])
def test_bad_pages_and_lengths_are_reported_and_not_followed(cache, q_len):
    kv_lens = [200, 100]
    kw = dict(N=4, N_kv=2, D=64, pre_tokens=60, sink_tokens=20, cache_dtype=cache, **W)
    geom = geometry([q_len, q_len], kv_lens, 16, **kw)
    p = make(geom, kv_lens, 3)
    good = run(geom, p)
    for entry, bad in ((0, -1), (0, geom.num_pages), (11, 2 ** 31 - 1), (12, -2 ** 31)):
        table = p["table"].clone()
        table[0, entry] = bad
        ws = swa.paged_forward_workspace(geom, DEV)
        ws.fill_(0xA5)
        dev = {n: t.to(DEV) for n, t in p["kw"].items()}
        out = swa.paged_forward(geom, p["q"].to(DEV), *[t.to(DEV) for t in p["pages"]], table.to(DEV), p["lens"].to(DEV),
                                workspace=ws, **dev)
        assert guarded(lambda: swa.check_paged_forward(geom, ws)) == swa.SWA_ERR_PAGE
        for a, b in zip(out, good):
            assert torch.equal(a[q_len:], b[q_len:])
        # a page that is not followed reads as zeros
        ks, vs = [t.clone() for t in p["ks"]], [t.clone() for t in p["vs"]]
        ks[0][16 * entry:16 * entry + 16], vs[0][16 * entry:16 * entry + 16] = 0, 0
        ref, err = attention_ref(geom, p["q"], ks, vs, kv_lens)
        for x, r, e in zip(out, ref, err):
            assert_within(x, r, e, (entry, bad))
    for bad in (-1, geom.max_pages * 16 + 1):
        lens = p["lens"].clone()
        lens[0] = bad
        ws = swa.paged_forward_workspace(geom, DEV)
        dev = {n: t.to(DEV) for n, t in p["kw"].items()}
        out = swa.paged_forward(geom, p["q"].to(DEV), *[t.to(DEV) for t in p["pages"]], p["table"].to(DEV), lens.to(DEV),
                                workspace=ws, **dev)
        assert guarded(lambda: swa.check_paged_forward(geom, ws)) == swa.SWA_ERR_PAGE
        assert (out[0][:q_len] == 0).all() and torch.isinf(out[1][:q_len]).all() and (out[2][:q_len] == 0).all()
        for a, b in zip(out, good):
            assert torch.equal(a[q_len:], b[q_len:])


def test_bad_pages_in_append_and_gather():
    geom = geometry([20, 3], [90, 40], 16, N=2, D=64, cache_dtype="e4m3")
    rows = [torch.randn(23, 2, 64, generator=torch.Generator().manual_seed(x)).bfloat16().to(DEV) for x in range(2)]
    table, lens = chunk_pages(geom, [90, 40], 1)
    for bad_table, bad_lens in (((0, 5, geom.num_pages), None), ((1, 2, -1), None), (None, (0, -3)), (None, (1, 10 ** 9))):
        t, n = table.clone(), lens.clone()
        if bad_table:
            t[bad_table[0], bad_table[1]] = bad_table[2]
        if bad_lens:
            n[bad_lens[0]] = bad_lens[1]
        pages, exps = empty_cache(geom)
        kw = dict(k_exponents=exps[0], v_exponents=exps[1])
        ws = swa.paged_append_workspace(geom, DEV)
        swa.paged_append(geom, *rows, *pages, t, n, workspace=ws, **kw)
        assert guarded(lambda: swa.check_paged_append(geom, ws)) == swa.SWA_ERR_PAGE
        k, v = swa.paged_gather(geom, *pages, t, n, workspace=ws, **kw)
        assert guarded(lambda: swa.check_paged_append(geom, ws)) == swa.SWA_ERR_PAGE
        # what was stored comes back; the rest is zeros
        for x, got in zip(rows, (k, v)):
            want = decode(*encode(x.cpu(), "bf16"))
            got = got.cpu().double()
            hit = (got == want).all(-1).all(-1)
            assert (got[~hit] == 0).all() and hit.any() and not hit.all()


@pytest.mark.parametrize("cache,tree,q_len", [("", True, 61), ("", False, 1), ("e4m3", False, 1), ("e4m3", True, 61),
                                              ("e4m3", False, 4)])
def test_replayed_graph_follows_new_lengths_trees_and_pages(cache, tree, q_len):
    """A captured step replays with new lengths, tables, trees, depths and exponents in place, on another stream; two
    captured steps with workspaces of their own run after one another; the bits are the eager ones."""
    kv = [[300, 90], [500, 61], [70, 444]]
    base = dict(N=8, N_kv=2, D=64, pre_tokens=100, sink_tokens=5, cache_dtype=cache, **W)
    most = geometry([q_len] * 2, [500, 500], 16, max_kv_len=500, **base)
    problems = []
    for x, lens in enumerate(kv):
        geom = geometry([q_len] * 2, [max(n, q_len) for n in lens], 16, **base)
        geom.num_pages, geom.max_pages, geom.max_kv_len = most.num_pages, most.max_pages, most.max_kv_len
        problems.append(make(geom, [max(n, q_len) for n in lens], 20 + x, tree))
    fixed = {n: t.to(DEV) for n, t in problems[0]["kw"].items()}
    fixed.update(q=problems[0]["q"].to(DEV), k=problems[0]["pages"][0].to(DEV), v=problems[0]["pages"][1].to(DEV),
                 table=problems[0]["table"].to(DEV), lens=problems[0]["lens"].to(DEV))
    plan = swa.PagedParams(most)
    extra = {n: fixed[n] for n in problems[0]["kw"]}

    def call(ws):
        return swa.paged_forward(plan, fixed["q"], fixed["k"], fixed["v"], fixed["table"], fixed["lens"], workspace=ws, **extra)

    spaces = [swa.paged_forward_workspace(plan, DEV) for _ in range(3)]
    call(spaces[0])
    torch.cuda.synchronize()
    graphs = []
    for ws in spaces[1:]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = call(ws)
        graphs.append((graph, res, ws))
    side = torch.cuda.Stream()
    for p in problems:
        as_bytes = lambda t: t.view(torch.uint8) if cache else t
        for n, t in (("q", p["q"]), ("table", p["table"]), ("lens", p["lens"]), *p["kw"].items()):
            fixed[n].copy_(t.to(DEV))
        for n, t in zip("kv", p["pages"]):
            as_bytes(fixed[n]).copy_(as_bytes(t).to(DEV))
        ref = call(spaces[0])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for graph, _, _ in graphs:
                graph.replay()
        torch.cuda.synchronize()
        for _, res, ws in graphs:
            swa.check_paged_forward(plan, ws)
            for a, b in zip(ref, res):
                assert torch.equal(a, b)


def test_another_stream():
    geom = geometry([61, 1], [500, 300], 16, N=8, N_kv=2, D=64, cache_dtype="e4m3", **W)
    p = make(geom, [500, 300], 4)
    ref = run(geom, p)
    dev = dict(q=p["q"].to(DEV), table=p["table"].to(DEV), lens=p["lens"].to(DEV), **{n: t.to(DEV) for n, t in p["kw"].items()})
    pages = [t.to(DEV) for t in p["pages"]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = swa.paged_forward(geom, dev["q"], *pages, dev["table"], dev["lens"], k_exponents=dev["k_exponents"],
                            v_exponents=dev["v_exponents"], stream=side)
    k, v = swa.paged_gather(geom, *pages, dev["table"], dev["lens"], k_exponents=dev["k_exponents"],
                            v_exponents=dev["v_exponents"], stream=side)
    side.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    assert torch.equal(k[-1].cpu().double(), p["ks"][1][-1])


def test_two_threads_at_once():
    """Calls of two threads, each with its stream and workspace, give the bits of calls one after the other."""
    import threading
    work = []
    for seed, (q_lens, kv_lens, tree) in enumerate((([61, 1, 4], [900, 700, 300], True), ([150, 1], [400, 2000], False))):
        geom = geometry(q_lens, kv_lens, 16, N=8, N_kv=2, D=128, pre_tokens=200, sink_tokens=4, cache_dtype="e4m3", **W)
        p = make(geom, kv_lens, seed + 3, tree)
        work.append((geom, p, run(geom, p)))
    torch.cuda.synchronize()
    got = [[], []]

    def many(i):
        geom, p, _ = work[i]
        dev = {n: t.to(DEV) for n, t in p["kw"].items()}
        args = [t.to(DEV) for t in (p["q"], *p["pages"], p["table"], p["lens"])]
        ws = swa.paged_forward_workspace(geom, DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                got[i].append(swa.paged_forward(geom, *args, workspace=ws, **dev))
        side.synchronize()

    threads = [threading.Thread(target=many, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 20
        for res in got[i]:
            for x, y in zip(work[i][2], res):
                assert torch.equal(x, y)


def test_python_refusals():
    geom = geometry([3, 40], [50, 90], 16, N=4, N_kv=2, D=64, cache_dtype="e4m3")
    p = make(geom, [50, 90], 4, True)
    a = dict(q=p["q"], k_pages=p["pages"][0], v_pages=p["pages"][1], block_table=p["table"], kv_lens=p["lens"], **p["kw"])
    a = {n: t.to(DEV) for n, t in a.items()}
    swa.paged_forward(geom, **a)
    wrong = {
        "k_pages": [a["k_pages"].view(torch.uint8), a["k_pages"].view(torch.int8), a["k_pages"][:-1]],
        "v_pages": [a["v_pages"].float().bfloat16()],
        "k_exponents": [a["k_exponents"].view(torch.uint8), a["k_exponents"][:-1], a["k_exponents"].transpose(1, 2),
                        a["k_exponents"].cpu(), 3],
        "v_exponents": [a["v_exponents"].int(), a["v_exponents"][..., :-1]],
        "tree": [a["tree"].long(), a["tree"][:-1], a["tree"][:, :1], a["tree"].flatten(), a["tree"].t().contiguous().t(),
                 a["tree"].cpu(), "tree"],
        "depth": [a["depth"].long(), a["depth"][:-1], a["depth"][:, None], a["depth"].cpu(), a["depth"].repeat(2)[::2]],
    }
    for name, values in wrong.items():
        for value in values:
            with pytest.raises(ValueError, match="k_exponents|v_exponents|tree|depth|k_pages|v_pages"):
                swa.paged_forward(geom, **{**a, name: value})
    for name in ("k_exponents", "v_exponents"):
        with pytest.raises(swa.SwaError) as e:
            swa.paged_forward(geom, **{**a, name: None})
        assert e.value.status == swa.SWA_ERR_PARAM_NULLPTR
    with pytest.raises(swa.SwaError):
        swa.paged_forward(geom, **{**a, "tree": None})  # a depth without a tree
    kv = [torch.zeros(43, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    cache = {n: a[n] for n in ("k_pages", "v_pages", "block_table", "kv_lens")}
    exps = {n: a[n] for n in ("k_exponents", "v_exponents")}
    for value in (kv[0][:-1], kv[0].half(), kv[0].cpu(), kv[0][..., :-1]):
        with pytest.raises(ValueError):
            swa.paged_gather(geom, **cache, k=value, v=kv[1], **exps)
        with pytest.raises(ValueError):
            swa.paged_append(geom, value, kv[1], **cache, **exps)
    with pytest.raises(swa.SwaError):
        swa.paged_gather(geom, **cache)
    with pytest.raises(swa.SwaError):
        swa.paged_append(geom, *kv, **cache)
    torch.cuda.synchronize()
