"""Exponents of an 8-bit cache that another writer put below the least of the type:
every reader takes them for the least (-15 fp16, -100 bf16)."""
import pytest
import torch

from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import PagedGeometry
from tests.paged_more_ref import LEAST, attention_ref
from tests.paged_ref import assert_within
from tests.test_paged_more_gpu import DEV, geometry, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("q_len,D", [(1, 64), (1, 128), (2, 72), (4, 64), (40, 64)])
def test_exponents_below_the_least(dtype, q_len, D):
    n, least = 150, LEAST[dtype]
    geom = geometry([q_len], [n], 16, N=4, N_kv=2, D=D, dtype=dtype, cache_dtype="e4m3", sparse_mode=4, next_tokens=0,
                    scale=1.0 if dtype == "fp16" else D ** -0.5)
    p = make(geom, [n], 31)
    for x, name in enumerate(("k_exponents", "v_exponents")):
        for j in range(n):
            if (j + x) % 3:
                continue
            e = p["kw"][name][int(p["table"][0, j // 16]), :, j % 16]
            p[("ks", "vs")[x]][0][j] *= torch.pow(2.0, (least - e.int()).double())[:, None]
            e.fill_((least - 5, least - 1, -128)[j % 9 // 3])
    ref, err = attention_ref(geom, p["q"], p["ks"], p["vs"], [n])
    for what, x, r, e in zip(("out", "softmax_max", "softmax_sum"), run(geom, p), ref, err):
        assert_within(x, r, e, what)
    whole = PagedGeometry(**{**geom.__dict__, "cu_seqlens_q": [n]})
    back = swa.paged_gather(whole, *[t.to(DEV) for t in p["pages"]], p["table"].to(DEV), p["lens"].to(DEV),
                            **{n: t.to(DEV) for n, t in p["kw"].items()})
    for got, want in zip(back, (p["ks"][0], p["vs"][0])):
        assert torch.equal(got.cpu().double(), want)
