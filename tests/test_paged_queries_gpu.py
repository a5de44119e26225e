"""Few query rows over an 8-bit cache at the ends of what a query and the scale may be:
rows of q near the largest bf16 number, rows of zeros or of tiny values under a tiny
scale.  The results are the definition's (tests/paged_more_ref.py), as over a 16-bit cache.

Scores before the scale are fp32 numbers over a 16-bit cache and in row tiles: rows of up
to 7 2^124 = 2^126.8 times keys of up to 4 and more, 64 of them summed, pass 2^128 there.
The few-row kernel over the 8-bit cache brings its queries into range first, and its
scores do not."""
import pytest
import torch

from tests.paged_more_ref import attention_ref
from tests.paged_ref import assert_within
from tests.test_paged_more_gpu import geometry, make, run

pytestmark = pytest.mark.gpu
SHAPES = [([1, 4], [90, 300], dict(N=2, N_kv=1, D=128)), ([4], [200], dict(N=8, N_kv=2, D=64)), ([3], [120], dict(N=2, N_kv=1, D=72)),
          ([1], [3000], dict(N=4, N_kv=2, D=128)), ([40], [300], dict(N=2, N_kv=1, D=64))]


SIZES = [(2.0 ** 112, 2.0 ** -115), (2.0 ** 118, 2.0 ** -120), (2.0 ** 124, 2.0 ** -126), (2.0 ** -90, 1e-20),
         (2.0 ** -120, 2.0 ** -30), (0.0, 1e-20), (0.0, 1e-30), (0.0, -1e-20), (2.0 ** -110, -1e-30)]
CASES = [(size, scale, shape, cache) for size, scale in SIZES for shape in range(len(SHAPES)) for cache in ("", "e4m3")
         if size < 2.0 ** 124 or (cache and shape < 4)]


@pytest.mark.parametrize("size,scale,shape,cache", CASES)
def test_queries_and_scales_of_any_size(size, scale, shape, cache):
    q_lens, kv_lens, kw = SHAPES[shape]
    geom = geometry(q_lens, kv_lens, 16, cache_dtype=cache, sparse_mode=4, next_tokens=0, pre_tokens=100, scale=scale, **kw)
    p = make(geom, kv_lens, 41)
    p["q"] = (p["q"].double().clamp(-7, 7) * size).bfloat16()
    assert torch.isfinite(p["q"]).all()
    ref, err = attention_ref(geom, p["q"], p["ks"], p["vs"], kv_lens)
    for what, x, r, e in zip(("out", "softmax_max", "softmax_sum"), run(geom, p), ref, err):
        assert_within(x, r, e, what)
