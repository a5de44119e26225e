"""Windows with sinks in the dense forward and backward against a 64-bit
reference (tests/sinks_ref.py derives the bounds), and equivalent problems."""
import pytest
import torch

from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import Geometry, draw
from tests.paged_ref import assert_within
from tests.sinks_ref import reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAMES = ("out", "softmax_max", "softmax_sum", "dq", "dk", "dv")


def bnsd(B, N, S, D, S_kv=None, **kw):
    kw.setdefault("scale", D ** -0.5)
    return Geometry("BNSD", B, N, D, S_q=S, S_kv=S if S_kv is None else S_kv, sparse_mode=4, **kw)


def tnd(q, kv, N, D, **kw):
    kw.setdefault("scale", D ** -0.5)
    ends = lambda x: [sum(x[:i + 1]) for i in range(len(x))]
    return Geometry("TND", len(q), N, D, cu_seqlens_q=ends(q), cu_seqlens_kv=ends(kv), sparse_mode=4, **kw)


def step(g, inp, mask=None):
    dev = [t.to(DEV) for t in (inp.q, inp.k, inp.v, inp.dy)]
    mask = None if mask is None else mask.to(DEV)
    ws = torch.full((swa.swa_backward_workspace_size(swa.Params(g)),), 0xA5, dtype=torch.uint8, device=DEV)
    out, smax, ssum = swa.forward(g, *dev[:3], mask)
    grads = swa.backward(g, *dev, out, smax, ssum, mask, workspace=ws)
    swa.check_workspace(ws)
    return (out, smax, ssum, *grads)


CASES = {
    "one_sink": bnsd(1, 1, 300, 64, pre_tokens=40, next_tokens=0, sink_tokens=1),
    "four_sinks": bnsd(2, 2, 700, 128, pre_tokens=100, next_tokens=0, sink_tokens=4),
    "a_whole_tile": bnsd(1, 2, 900, 128, pre_tokens=64, next_tokens=0, sink_tokens=128),
    "past_a_tile": bnsd(1, 2, 900, 96, pre_tokens=30, next_tokens=0, sink_tokens=131, dtype="fp16"),
    "three_tiles": bnsd(1, 4, 1300, 64, N_kv=2, pre_tokens=130, next_tokens=0, sink_tokens=300),
    "sinks_reach_the_window": bnsd(1, 1, 600, 72, pre_tokens=200, next_tokens=0, sink_tokens=250),
    "more_sinks_than_keys": bnsd(1, 2, 400, 128, pre_tokens=10, next_tokens=0, sink_tokens=100000),
    "window_of_one": bnsd(1, 2, 520, 64, pre_tokens=0, next_tokens=0, sink_tokens=3),
    "keys_ahead": bnsd(1, 2, 520, 128, pre_tokens=20, next_tokens=33, sink_tokens=7),
    "sinks_not_yet_reached": bnsd(1, 1, 400, 64, pre_tokens=300, next_tokens=-60, sink_tokens=50),
    "window_ahead": bnsd(1, 1, 400, 64, pre_tokens=-5, next_tokens=20, sink_tokens=9),
    "more_queries_than_keys": bnsd(1, 2, 800, 64, S_kv=200, pre_tokens=50, next_tokens=0, sink_tokens=5),
    "more_keys_than_queries": bnsd(1, 2, 200, 128, S_kv=900, pre_tokens=50, next_tokens=0, sink_tokens=5),
    "grouped": bnsd(1, 12, 640, 128, N_kv=3, pre_tokens=90, next_tokens=0, sink_tokens=20),
    "mqa_pieces": bnsd(1, 8, 1500, 64, N_kv=1, pre_tokens=70, next_tokens=0, sink_tokens=140, dtype="fp16"),
    "d8": bnsd(1, 1, 300, 8, pre_tokens=20, next_tokens=0, sink_tokens=2),
    "d40_many_heads": bnsd(2, 40, 512, 40, pre_tokens=60, next_tokens=0, sink_tokens=5),
    "scale_negative": bnsd(1, 1, 300, 64, pre_tokens=50, next_tokens=0, sink_tokens=4, scale=-0.2),
    "fp32": bnsd(1, 2, 400, 64, pre_tokens=50, next_tokens=0, sink_tokens=4, dtype="fp32"),
    "dropout": bnsd(1, 2, 500, 128, pre_tokens=60, next_tokens=0, sink_tokens=4, keep_prob=0.75, dropout_gen=1,
                    dropout_seed=77),
    "dropout_d64": bnsd(1, 4, 700, 64, N_kv=2, pre_tokens=60, next_tokens=0, sink_tokens=129, keep_prob=0.75,
                        dropout_gen=1, dropout_seed=78),
    "dropout_mask": bnsd(1, 2, 500, 64, pre_tokens=60, next_tokens=0, sink_tokens=4, keep_prob=0.75),
    "ragged": tnd([1, 0, 300, 129, 700], [1, 0, 300, 129, 700], 4, 128, N_kv=2, pre_tokens=64, next_tokens=0,
                  sink_tokens=4),
    "ragged_unequal": tnd([50, 600, 0, 7], [400, 60, 9, 0], 2, 64, pre_tokens=30, next_tokens=0, sink_tokens=10,
                          dtype="fp16"),
    "ragged_many": tnd([40 + 7 * i for i in range(20)], [40 + 7 * i for i in range(20)], 2, 96, pre_tokens=16,
                       next_tokens=0, sink_tokens=6),
}


def check(g, seed):
    inp = draw(g, seed)
    if g.dtype == "fp32":  # the products take bf16 copies: values that those hold
        for n in ("q", "k", "v", "dy"):
            setattr(inp, n, getattr(inp, n).bfloat16().float())
    mask = inp.drop_mask
    if g.dropout_gen:
        bits = swa.dropout_mask(g, DEV)
        got = step(g, inp)
    else:
        bits = mask
        got = step(g, inp, mask)
    res, err = reference(g, inp.q, inp.k, inp.v, inp.dy, bits)
    if g.dtype == "fp32":
        # out goes through bf16 once more on its way into D
        extra = 2.0 ** -8 * (inp.dy.double().abs() * res[0].abs()).sum(-1).amax()
        err[3] += extra * g.scale * inp.k.double().abs().amax()
        err[4] += extra * g.scale * inp.q.double().abs().amax() * g.S_q
    for n, x, r, e in zip(NAMES, got, res, err):
        assert_within(x, r, e, (g, n))


@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_backward_match_the_definition(name):
    check(CASES[name], 5)


@pytest.mark.parametrize("pairs", [1, 2])
def test_both_forwards_of_small_heads(pairs):
    swa.swa_debug_forward_pairs(pairs)
    try:
        for name in ("three_tiles", "past_a_tile", "more_queries_than_keys", "sinks_not_yet_reached", "d8", "ragged_unequal"):
            check(CASES[name], 6)
    finally:
        swa.swa_debug_forward_pairs(0)


def test_more_sequences_than_a_table_holds():
    lens = [3 + (5 * i) % 90 for i in range(700)]
    lens[3], lens[600] = 500, 800
    check(tnd(lens, lens, 1, 16, pre_tokens=20, next_tokens=0, sink_tokens=5), 8)


def test_no_sinks_gives_the_bits_of_the_plain_window():
    g0 = bnsd(1, 4, 900, 128, N_kv=2, pre_tokens=100, next_tokens=0)
    inp = draw(g0, 3)
    ref = step(g0, inp)
    for sinks in (0, 1):  # one sink is seen anyway by a window that reaches everything
        g = bnsd(1, 4, 900, 128, N_kv=2, pre_tokens=100 if sinks == 0 else 5000, next_tokens=0, sink_tokens=sinks)
        want = ref if sinks == 0 else step(bnsd(1, 4, 900, 128, N_kv=2, pre_tokens=5000, next_tokens=0), inp)
        for n, a, b in zip(NAMES, step(g, inp), want):
            assert torch.equal(a, b) or n in ("dk", "dv"), n  # (pieces are summed in another order)
            assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-3), n


def test_same_bits_again_and_in_a_graph():
    g = bnsd(1, 8, 1500, 64, N_kv=1, pre_tokens=70, next_tokens=0, sink_tokens=140)
    inp = draw(g, 9)
    dev = [t.to(DEV) for t in (inp.q, inp.k, inp.v, inp.dy)]
    p = swa.Params(g)
    fws, bws = (torch.empty(n, dtype=torch.uint8, device=DEV) for n in
                (swa.swa_forward_workspace_size(p), swa.swa_backward_workspace_size(p)))

    def call():
        out, sm, ss = swa.forward(g, *dev[:3], workspace=fws)
        return (out, sm, ss, *swa.backward(g, *dev, out, sm, ss, workspace=bws))

    ref = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        res = call()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, res):
            assert torch.equal(a, b)


def test_host_step_with_sinks():
    g = bnsd(1, 4, 700, 64, N_kv=2, pre_tokens=64, next_tokens=0, sink_tokens=9)
    inp = draw(g, 12)
    ref = step(g, inp)
    host = [t.pin_memory() for t in (inp.q, inp.k, inp.v, inp.dy)]
    res = [torch.empty_like(t, device="cpu").pin_memory() for t in ref]
    buf = swa.step_host(g, *host, *res, chunks=2)
    torch.cuda.synchronize()
    swa.check_step_host(g, 2, buf)
    for n, a, b in zip(NAMES, res, ref):
        # (fewer heads at a time may cut a tile with sinks into other pieces)
        same = torch.equal(a, b.cpu())
        assert same or (n in ("dk", "dv") and torch.allclose(a.float(), b.cpu().float(), rtol=2.0 ** -7, atol=1e-3)), n


def test_long_sequence_on_a_few_rows():
    """Past 2^15 keys: selected rows of each result against the definition."""
    S, D, pre, sinks = 40000, 64, 1000, 5
    g = bnsd(1, 2, S, D, N_kv=1, pre_tokens=pre, next_tokens=0, sink_tokens=sinks)
    gen = torch.Generator(DEV).manual_seed(1)
    q, dy = (torch.randn(1, 2, S, D, generator=gen, device=DEV).bfloat16() for _ in range(2))
    k, v = (torch.randn(1, 1, S, D, generator=gen, device=DEV).bfloat16() for _ in range(2))
    out, sm, ss = swa.forward(g, q, k, v)
    dq, dk, dv = swa.backward(g, q, k, v, dy, out, sm, ss)
    kk, vv = k[0, 0].double(), v[0, 0].double()
    sink_dk, sink_dv = (torch.zeros(sinks, D, dtype=torch.float64, device=DEV) for _ in range(2))
    for h in range(2):
        for c in range(0, S, 4000):
            i = torch.arange(c, c + 4000, device=DEV)
            lo = max(0, c - pre)
            keys = torch.cat((torch.arange(min(sinks, lo), device=DEV), torch.arange(lo, c + 4000, device=DEV)))
            seen = (keys <= i[:, None]) & ((keys >= i[:, None] - pre) | (keys < sinks))
            x, y = q[0, h, c:c + 4000].double(), dy[0, h, c:c + 4000].double()
            s = ((x @ kk[keys].T) * g.scale).masked_fill(~seen, -float("inf"))
            p = torch.softmax(s, 1)
            o = p @ vv[keys]
            ds = p * (y @ vv[keys].T - (y * o).sum(1, keepdim=True))
            for a, b in ((out[0, h, c:c + 4000], o), (dq[0, h, c:c + 4000], ds @ kk[keys] * g.scale)):
                # the roundings of P, dS and the results: 2^-8 of a few values each
                assert (a.double() - b).norm() <= 1e-2 * b.norm()
            for row in range(sinks):
                sink_dk[row] += (ds[:, keys == row] * x).sum(0) * g.scale
                sink_dv[row] += (p[:, keys == row] * y).sum(0)
    assert (dk[0, 0, :sinks].double() - sink_dk).norm() <= 1e-2 * sink_dk.norm()
    assert (dv[0, 0, :sinks].double() - sink_dv).norm() <= 1e-2 * sink_dv.norm()


@pytest.mark.parametrize("name", ["past_a_tile", "mqa_pieces", "ragged_unequal", "dropout_d64", "keys_ahead"])
def test_bounds_checked_build_gives_the_same_bits(name):
    g = CASES[name]
    inp = draw(g, 4)
    mask = inp.drop_mask
    ref = step(g, inp, mask)
    with swa.using(swa.checked_lib()):
        got = step(g, inp, mask)
    for n, a, b in zip(NAMES, got, ref):
        assert torch.equal(a, b), n


def test_no_allocation_entry_point():
    g = CASES["grouped"]
    inp = draw(g, 4)
    ref = step(g, inp)
    dev = [t.to(DEV) for t in (inp.q, inp.k, inp.v, inp.dy)]
    grads = [torch.empty_like(t) for t in dev[:3]]
    st = swa.swa_backward_noalloc(swa.Params(g), *[t.data_ptr() for t in dev], *[t.data_ptr() for t in ref[:3]], None,
                                  *[t.data_ptr() for t in grads], torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == swa.SWA_OK
    for n, a, b in zip(NAMES[3:], grads, ref[3:]):
        assert torch.equal(a, b), n
