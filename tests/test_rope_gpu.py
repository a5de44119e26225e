"""Rotary positions on the GPU against the 64-bit definition (tests/paged_ref.py
states the tolerance): layouts, pair forms, axes, partial rotation, element
types, strides, far and negative positions, in place, and the gradient."""
import pytest
import torch

from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import RopeGeometry
from tests.paged_ref import DT, assert_within, rope_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def draw(geom, seed, top=5000, low=-50):
    g = torch.Generator().manual_seed(seed)
    dt = DT[geom.dtype]
    qs = (geom.B, geom.N, geom.S, geom.D) if geom.layout == "BNSD" else (geom.B * geom.S, geom.N, geom.D)
    ks = (geom.B, geom.n_kv, geom.S, geom.D) if geom.layout == "BNSD" else (geom.B * geom.S, geom.n_kv, geom.D)
    q, k = torch.randn(qs, generator=g).to(dt), torch.randn(ks, generator=g).to(dt)
    pos = torch.randint(low, top, (geom.n_axes, geom.B * geom.S), generator=g, dtype=torch.int32)
    return q, k, pos


CASES = {
    "tnd_bf16": dict(layout="TND", B=1, S=37, N=4, N_kv=2, D=128),
    "bnsd_fp16_3axes": dict(layout="BNSD", B=2, S=45, N=6, N_kv=3, D=64, sections=[8, 12, 12], dtype="fp16"),
    "bnsd_fp32_interleaved": dict(layout="BNSD", B=3, S=7, N=2, D=96, interleaved=True, dtype="fp32"),
    "tnd_partial": dict(layout="TND", B=1, S=33, N=5, N_kv=1, D=112, rotary_dim=48),
    "tnd_partial_odd_interleaved": dict(layout="TND", B=2, S=9, N=3, D=88, rotary_dim=40, interleaved=True),
    "d8": dict(layout="TND", B=1, S=5, N=1, D=8, dtype="fp16"),
    "d24_tail": dict(layout="BNSD", B=1, S=19, N=2, D=24, rotary_dim=8),
    "d72_fp32": dict(layout="TND", B=1, S=11, N=3, N_kv=2, D=72, dtype="fp32", sections=[30, 6]),
    "one_row": dict(layout="TND", B=1, S=1, N=32, N_kv=8, D=128),
    "rows_past_a_cta": dict(layout="BNSD", B=2, S=6000, N=2, N_kv=1, D=64, sections=[16, 16]),
    "mqa_many_heads": dict(layout="TND", B=1, S=3, N=256, N_kv=1, D=40),
    "own_frequencies": dict(layout="TND", B=1, S=21, N=2, D=32, inv_freq=[1.0, -0.5, 0.0, 700.25] * 4,
                            pair_axis=[0, 1, 2, 3] * 4),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_forward_and_gradient_match_the_definition(name):
    geom = RopeGeometry(**CASES[name])
    q, k, pos = draw(geom, 5)
    for call, inverse in ((swa.rope, False), (swa.rope_backward, True)):
        got = call(geom, q.to(DEV), k.to(DEV), pos.to(DEV))
        for x, y, what in zip((q, k), got, "qk"):
            ref, err = rope_ref(geom, x, pos, inverse)
            assert_within(y, ref, err, (name, what, inverse))


def test_gradient_against_differences():
    """d/dx sum(w * rope(x)) by central differences: the map is linear, so they
    are exact but for fp32 rounding (2^-22 of the row's size each way)."""
    geom = RopeGeometry("TND", 1, 6, 2, 16, sections=[4, 4], dtype="fp32")
    q, _, pos = draw(geom, 9)
    w = torch.randn(q.shape, generator=torch.Generator().manual_seed(1))
    dq, _ = swa.rope_backward(geom, w.to(DEV), None, pos.to(DEV))
    h = 0.5
    for e in range(0, q.numel(), 7):
        d = torch.zeros(q.numel())
        d[e] = h
        hi, _ = swa.rope(geom, (q + d.view(q.shape)).to(DEV), None, pos.to(DEV))
        lo, _ = swa.rope(geom, (q - d.view(q.shape)).to(DEV), None, pos.to(DEV))
        diff = ((hi - lo).cpu().double() * w.double()).sum() / (2 * h)
        size = (q.abs().amax() + h) * w.abs().amax()
        assert abs(diff - dq.cpu().reshape(-1)[e].double()) <= 16 * 2.0 ** -21 * size


def test_far_positions_keep_their_accuracy():
    geom = RopeGeometry("TND", 1, 64, 2, 128, dtype="fp32")
    q, k, _ = draw(geom, 3)
    g = torch.Generator().manual_seed(4)
    pos = torch.randint(2 ** 31 - 10 ** 6, 2 ** 31 - 1, (1, 64), generator=g, dtype=torch.int64)
    pos[0, ::2] *= -1
    pos[0, 0], pos[0, 1] = -2 ** 31, 2 ** 31 - 1
    pos = pos.to(torch.int32)
    y, _ = swa.rope(geom, q.to(DEV), k.to(DEV), pos.to(DEV))
    ref, err = rope_ref(geom, q, pos)
    # angles up to 2^31 radians: inv_freq (a unit in the last place), 1 / (2 pi), their
    # product and the reference's own product each round by 2^-53, the first
    # by twice that: 6 * 2^-53 * 2^31 radians on |a| + |b|
    slack = 6 * 2.0 ** -22 * 2 * q.abs().amax().double()
    assert_within(y, ref, err + slack, "far")


def test_only_q_or_only_k():
    geom = RopeGeometry("TND", 1, 10, 4, 64, N_kv=2)
    q, k, pos = draw(geom, 6)
    both = swa.rope(geom, q.to(DEV), k.to(DEV), pos.to(DEV))
    a, none = swa.rope(geom, q.to(DEV), None, pos.to(DEV))
    none2, b = swa.rope(geom, None, k.to(DEV), pos.to(DEV))
    assert none is None and none2 is None
    assert torch.equal(a, both[0]) and torch.equal(b, both[1])


@pytest.mark.parametrize("layout", ["BNSD", "TND"])
def test_slices_of_a_projection_and_in_place(layout):
    """q and k as slices of one fused [.., N + 2 N_kv, D] projection, results
    written back in place: the dense result's bits, v untouched."""
    geom = RopeGeometry(layout, 2, 13, 4, 80, N_kv=2, sections=[10, 30], dtype="bf16")
    q, k, pos = draw(geom, 7)
    ref = swa.rope(geom, q.to(DEV), k.to(DEV), pos.to(DEV))
    v = torch.randn(k.shape).to(k.dtype)
    fused = torch.cat((q, k, v), dim=1).to(DEV)
    fq, fk, fv = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    out = swa.rope(geom, fq, fk, pos.to(DEV), fq, fk)
    assert out[0].data_ptr() == fq.data_ptr()
    assert torch.equal(fq, ref[0]) and torch.equal(fk, ref[1]) and torch.equal(fv.cpu(), v)
    # a transposed BNSD view of a [B, S, N, D] tensor, heads innermost
    if layout == "BNSD":
        t = q.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
        assert torch.equal(swa.rope(geom, t, None, pos.to(DEV))[0], ref[0])
    # one gradient row shared by every head (a broadcast input)
    one = q[:, :1].to(DEV)
    assert torch.equal(swa.rope(geom, one.expand(q.shape), None, pos.to(DEV))[0],
                       swa.rope(geom, one.expand(q.shape).contiguous(), None, pos.to(DEV))[0])


def test_forward_then_backward_returns_and_streams():
    geom = RopeGeometry("TND", 1, 500, 8, 128, N_kv=2, sections=[16, 24, 24], dtype="fp32")
    q, k, pos = (t.to(DEV) for t in draw(geom, 8))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y = swa.rope(geom, q, k, pos, stream=st)
    back = swa.rope_backward(geom, *y, pos, stream=st)
    st.synchronize()
    for x, z in zip((q, k), back):
        # two rotations, each within 2^-21 of its pair and 2^-24 stored
        assert (x - z).abs().max() <= 4 * 2.0 ** -21 * x.abs().max() * 2
    with torch.cuda.stream(st):
        y2 = swa.rope(swa.RopeParams(geom), q, k, pos)
    st.synchronize()
    assert torch.equal(y[0], y2[0]) and torch.equal(y[1], y2[1])


def test_captured_rotation_replays():
    geom = RopeGeometry("TND", 1, 64, 4, 64, sections=[16, 16])
    q, k, pos = (t.to(DEV) for t in draw(geom, 2))
    p = swa.RopeParams(geom)
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    swa.rope(p, q, k, pos, yq, yk)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        swa.rope(p, q, k, pos, yq, yk)
        swa.rope_backward(p, yq, yk, pos, yq, yk)
    pos.add_(17)
    want = swa.rope_backward(p, *swa.rope(p, q, k, pos), pos)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(yq, want[0]) and torch.equal(yk, want[1])


def test_positions_of_another_shape_are_refused():
    """[rows, n_axes] holds as many numbers as [n_axes, rows]."""
    geom = RopeGeometry("TND", 1, 12, 2, 64, sections=[16, 16])
    q, k, pos = (t.to(DEV) for t in draw(geom, 2))
    for bad in (pos.T.contiguous(), pos.flatten(), pos.T):
        with pytest.raises(ValueError):
            swa.rope(geom, q, k, bad)
    one = RopeGeometry("TND", 1, 12, 2, 64)
    a = swa.rope(one, q, k, pos[0])
    b = swa.rope(one, q, k, pos[:1])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
