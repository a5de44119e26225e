"""Few query rows over an 8-bit cache whose values differ by many powers of two: a
row's result depends on what the row sees, not on larger values that only other
rows of its chunk see, or that it gives little weight.

Bounds, first order, for a row with weights P_j (sum 1) over n keys of rows v_j with
exponents e_j: a weight is off by 2 e of itself for its score's error e
(tests/paged_more_ref.py), is rounded to fp16 relative to the row's largest
P_j 2^e_j, 2^-11 of itself or 2^-31 of that largest (a code is at most 448, and 448 2^e_j
at most twice the largest of v_j unless e_j is the least), and fp32 sums of n terms,
which the products may truncate, add n 2^-23; storing adds half a step.  Sequences of
more than 16 rows per key/value head: weights rounded to the element type instead, and
in fp16 to 2^-25 of the largest value that the row sees."""
import pytest
import torch

from tests.paged_more_ref import LEAST, attention_ref, seen_of
from tests.paged_ref import U, assert_within
from tests.test_paged_more_gpu import geometry, make, run

pytestmark = pytest.mark.gpu
W = dict(sparse_mode=4, next_tokens=0)


def scale_values(geom, p, kv_lens, shift):
    """V of key j of sequence b times 2^shift(b, j, n, m), by its exponents."""
    for b, (n, m) in enumerate(zip(kv_lens, geom.q_lens())):
        vs = p["vs"][b]
        for j in range(n):
            page = int(p["table"][b, j // geom.page_size])
            if page < 0:
                continue
            at = p["kw"]["v_exponents"][page, :, j % geom.page_size]
            e = (at.int() + shift(b, j, n, m)).clamp(LEAST[geom.dtype], 7)
            vs[j] *= torch.pow(2.0, (e - at.int()).double())[:, None]
            at.copy_(e.to(torch.int8))


def result_bounds(geom, q, ks, vs, kv_lens, trees=None):
    """The bound of `out`, from the keys that each row sees."""
    T, N, D = q.shape
    G, u = N // geom.n_kv, U[geom.dtype]
    eo = torch.zeros(T, N, D, dtype=torch.float64)
    zero = torch.zeros((), dtype=torch.float64)
    row = 0
    for b, (n, m) in enumerate(zip(kv_lens, geom.q_lens())):
        r = slice(row, row + m)
        row += m
        if n == 0 or m == 0:
            continue
        seen = seen_of(geom, n, m, *(trees[b] if trees is not None else ()))
        for h in range(N):
            x, k, v = q[r, h].double(), ks[b][:, h // G], vs[b][:, h // G]
            s = torch.where(seen, (x @ k.T) * geom.scale, torch.full((), -float("inf"), dtype=torch.float64))
            size = torch.where(seen, (x.abs() @ k.abs().T) * abs(geom.scale), zero).amax(1)
            P = torch.nan_to_num(torch.softmax(s, 1))
            e = D * 2.0 ** -23 * size + 2.0 ** -22 * (size + 1)
            e = e + abs(geom.scale) * x.abs().amax(1) * 2.0 ** -39 * k.abs().sum(1).amax()
            top = v.abs().amax(1)
            if m * G <= 16:
                w = 2.0 ** -11
                small = 2.0 ** -31 * (P * torch.maximum(2 * top, torch.full((), 448 * 2.0 ** LEAST[geom.dtype]))).amax(1)
            else:
                w = u
                small = 2.0 ** -25 * torch.where(seen, top, zero).amax(1) if geom.dtype == "fp16" else zero.expand(m)
            err = (P @ v.abs()) * (w + 2 * e + n * 2.0 ** -23)[:, None] + n * small[:, None]
            eo[r, h] = err + u * ((P @ v).abs() + err) + (2.0 ** -25 if geom.dtype == "fp16" else 0.0)
    return eo


def check(geom, p, kv_lens):
    ref, err = attention_ref(geom, p["q"], p["ks"], p["vs"], kv_lens, p["trees"])
    bounds = (result_bounds(geom, p["q"], p["ks"], p["vs"], kv_lens, p["trees"]), *err[1:])
    for what, x, r, e in zip(("out", "softmax_max", "softmax_sum"), run(geom, p), ref, bounds):
        assert_within(x, r, e, (geom, what))


SHAPES = {
    "8_rows": ([4, 3], [90, 333], dict(N=2, N_kv=1, D=128)),
    "16_rows": ([4], [200], dict(N=8, N_kv=2, D=128)),
    "16_rows_d64": ([8, 2], [77, 300], dict(N=2, N_kv=1, D=64)),
    "d72": ([4], [120], dict(N=2, N_kv=1, D=72)),
    "d40_16_rows": ([4], [120], dict(N=4, N_kv=1, D=40)),
    "clustered": ([2], [1500], dict(N=4, N_kv=4, D=64)),
    "split": ([3], [9000], dict(N=4, N_kv=2, D=128)),
    "row_tiles": ([40], [300], dict(N=4, N_kv=2, D=128)),
}


@pytest.mark.parametrize("dtype,quiet,loud", [("bf16", -40, 10), ("bf16", -93, 14), ("bf16", -20, 4), ("fp16", -8, 14)])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_larger_values_of_a_later_token(shape, dtype, quiet, loud):
    """Each chunk's last token has far larger values than all before it."""
    q_lens, kv_lens, kw = SHAPES[shape]
    geom = geometry(q_lens, kv_lens, 16, cache_dtype="e4m3", dtype=dtype, **W, **kw)
    p = make(geom, kv_lens, 21)
    scale_values(geom, p, kv_lens, lambda b, j, n, m: loud if j == n - 1 else quiet)
    check(geom, p, kv_lens)


@pytest.mark.parametrize("shape", ["8_rows", "16_rows", "d72", "row_tiles"])
def test_larger_values_of_a_sibling_in_a_tree(shape):
    q_lens, kv_lens, kw = SHAPES[shape]
    geom = geometry(q_lens, kv_lens, 16, cache_dtype="e4m3", **kw)
    p = make(geom, kv_lens, 22, True)
    scale_values(geom, p, kv_lens, lambda b, j, n, m: (-60, 10, -30)[j % 3] if j >= n - m else -45)
    check(geom, p, kv_lens)


@pytest.mark.parametrize("shape", ["8_rows", "16_rows", "16_rows_d64", "d40_16_rows"])
def test_larger_values_that_left_the_window(shape):
    """The first token of a chunk still sees keys far larger than all that the later ones see."""
    q_lens, kv_lens, kw = SHAPES[shape]
    geom = geometry(q_lens, kv_lens, 16, cache_dtype="e4m3", pre_tokens=40, **W, **kw)
    p = make(geom, kv_lens, 23)
    scale_values(geom, p, kv_lens, lambda b, j, n, m: 12 if j <= n - m - 40 else -40)
    check(geom, p, kv_lens)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("sharp", [1.0, 12.0, 60.0])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_any_values_under_any_weights(shape, sharp, dtype):
    """Exponents all over their range, under weights from nearly equal to one key's alone, rising and falling along the
    sequence."""
    q_lens, kv_lens, kw = SHAPES[shape]
    geom = geometry(q_lens, kv_lens, 16, cache_dtype="e4m3", dtype=dtype, **W, **kw)
    for way in (lambda j, n: (j * 37) % 108, lambda j, n: j * 108 // n, lambda j, n: 107 - j * 108 // n):
        p = make(geom, kv_lens, 24, loud=sharp)
        scale_values(geom, p, kv_lens, lambda b, j, n, m: way(j, n) - 92)
        check(geom, p, kv_lens)


def test_a_weight_on_zeros():
    """Rows of zeros, whose exponent is the least, take nearly all the weight; the rest is far smaller and counts."""
    for sharp in (3.0, 10.0):
        geom = geometry([3], [400], 16, N=2, N_kv=1, D=64, cache_dtype="e4m3", **W)
        p = make(geom, [400], 25, loud=sharp)
        scale_values(geom, p, [400], lambda b, j, n, m: -200)
        heavy = (p["q"][:, 0].double() @ p["ks"][0][:, 0].T).amax(0) > 0
        p["vs"][0][heavy] = 0
        for j in heavy.nonzero()[:, 0].tolist():
            page, slot = int(p["table"][0, j // 16]), j % 16
            p["pages"][1].view(torch.uint8)[page, :, slot] = 0
        check(geom, p, [400])
