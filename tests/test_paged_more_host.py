"""Refusals of the calls with sinks, trees and an 8-bit cache, on the CPU: every case returns before any device work."""
import ctypes

import pytest

from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import PagedGeometry

NULL, INVALID, UNSUPPORTED, WORKSPACE = (swa.SWA_ERR_PARAM_NULLPTR, swa.SWA_ERR_PARAM_INVALID, swa.SWA_ERR_UNSUPPORTED,
                                         swa.SWA_ERR_WORKSPACE)
P16 = 1 << 20  # an aligned address that nothing reads


def geom(**kw):
    base = dict(B=2, N=4, N_kv=2, D=64, cu_seqlens_q=[33, 40], num_pages=8, page_size=16, max_pages=4)
    return PagedGeometry(**{**base, **kw})


def test_structs_match_c_layout(tmp_path):
    import os
    import subprocess

    from attention_swa_forward_gb300 import build as B

    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "swa.h"\nint main(void){printf("%zu %zu %zu %zu %zu %zu",'
                   "sizeof(swa_paged_extra_t), offsetof(swa_paged_extra_t, depth), sizeof(swa_paged_params_t),"
                   "offsetof(swa_paged_params_t, sink_tokens), offsetof(swa_paged_params_t, cache_dtype),"
                   "offsetof(swa_params_t, sink_tokens)); return 0;}")
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-I", B.INCLUDE, str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    E, PP = swa.SwaPagedExtra, swa.SwaPagedParams
    assert got == [ctypes.sizeof(E), E.depth.offset, ctypes.sizeof(PP), PP.sink_tokens.offset, PP.cache_dtype.offset,
                   swa.SwaParams.sink_tokens.offset]
    assert os.path.exists(exe)


def forward(g, extra=None, ws=1 << 40, **change):
    p = swa.PagedParams(g)
    x = None
    if extra is not None:
        x = swa.SwaPagedExtra(**extra)
    a = dict(q=P16, qs=None, kp=P16, kps=None, vp=P16, vps=None, extra=None if x is None else ctypes.addressof(x), table=P16,
             stride=0, lens=P16, out=P16, smax=None, ssum=None, ws=P16, n=0, stream=None)
    a.update(change)
    status = swa.lib().swa_paged_forward_ext(p.ref(), *a.values())
    return status, swa.swa_last_error()


# Each differs from a call that gets as far as the workspace check, which refuses it (size 0).
E4 = dict(cache_dtype="e4m3")
X8 = dict(k_exponents=P16, v_exponents=P16)


@pytest.mark.parametrize("want,words,g,extra", [
    (WORKSPACE, "workspace", {}, None),
    (WORKSPACE, "workspace", {}, {}),
    (WORKSPACE, "workspace", dict(sink_tokens=3, sparse_mode=4), {}),
    (WORKSPACE, "workspace", E4, X8),
    (WORKSPACE, "workspace", {}, dict(tree=P16)),
    (WORKSPACE, "workspace", {}, dict(tree=P16, tree_stride=2, depth=P16)),
    (WORKSPACE, "workspace", dict(sparse_mode=4, next_tokens=0), dict(tree=P16)),
    (INVALID, "sink_tokens", dict(sink_tokens=-1), None),
    (NULL, "k_exponents", E4, None),
    (NULL, "v_exponents", E4, dict(k_exponents=P16)),
    (INVALID, "aligned", E4, dict(k_exponents=P16 + 8, v_exponents=P16)),
    (INVALID, "e4m3", {}, X8),
    (INVALID, "tree_stride", {}, dict(tree=P16, tree_stride=1)),
    (INVALID, "tree_stride", {}, dict(tree=P16, tree_stride=-2)),
    (INVALID, "tree", {}, dict(depth=P16)),
    (INVALID, "tree", {}, dict(tree_stride=2)),
    (INVALID, "aligned", {}, dict(tree=P16 + 2)),
    (INVALID, "aligned", {}, dict(tree=P16, depth=P16 + 1)),
    (INVALID, "next_tokens", dict(sparse_mode=4, pre_tokens=9, next_tokens=-1), dict(tree=P16)),
])
def test_forward_refusals(want, words, g, extra):
    status, text = forward(geom(**g), extra)
    assert status == want and words in text, (status, text)


def test_cache_dtype_is_checked():
    p = swa.PagedParams(geom())
    p.c.cache_dtype = 2
    with pytest.raises(swa.SwaError, match="cache_dtype"):
        swa.swa_paged_forward_workspace_size(p)
    with pytest.raises(KeyError):
        swa.PagedParams(geom(cache_dtype="e5m2"))


def test_plain_calls_refuse_an_8_bit_cache():
    p = swa.PagedParams(geom(**E4))
    assert swa.lib().swa_paged_forward(p.ref(), P16, None, P16, None, P16, None, P16, 0, P16, P16, None, None, P16, 0,
                                       None) == NULL
    assert swa.lib().swa_paged_append(p.ref(), P16, None, P16, None, P16, None, P16, None, P16, 0, P16, None, None, None, None,
                                      None, None, P16, 0, None) == NULL


def gather(g, **change):
    p = swa.PagedParams(g)
    a = dict(kp=P16, kps=None, vp=P16, vps=None, ke=None, ve=None, table=P16, stride=0, lens=P16, k=P16, ks=None, v=P16, vs=None,
             ws=P16, n=0, stream=None)
    a.update(change)
    return swa.lib().swa_paged_gather(p.ref(), *a.values()), swa.swa_last_error()


@pytest.mark.parametrize("want,words,g,change", [
    (WORKSPACE, "workspace", {}, {}),
    (WORKSPACE, "workspace", E4, dict(ke=P16, ve=P16)),
    (NULL, "k is", {}, dict(k=None)),
    (NULL, "v is", {}, dict(v=None)),
    (INVALID, "aligned", {}, dict(v=P16 + 2)),
    (NULL, "k_pages", {}, dict(kp=None)),
    (NULL, "block_table", {}, dict(table=None)),
    (NULL, "v_exponents", E4, dict(ke=P16)),
    (INVALID, "e4m3", {}, dict(ke=P16)),
    (INVALID, "overlaps", {}, dict(ks="overlap", n=1 << 30)),
    (WORKSPACE, "workspace", {}, dict(n=1 << 30, ws=P16 + 16)),
    (UNSUPPORTED, "fp32", dict(dtype="fp32"), {}),
])
def test_gather_refusals(want, words, g, change):
    keep = swa.SwaStrides(0, 64, 64)
    change = {n: (ctypes.addressof(keep) if x == "overlap" else x) for n, x in change.items()}
    status, text = gather(geom(**g), **change)
    assert status == want and words in text, (status, text)


def test_workspace_covers_sinks():
    """More keys per row, never fewer splits than they need; none without a window."""
    size = lambda **kw: swa.swa_paged_forward_workspace_size(swa.PagedParams(geom(max_pages=10000, **kw)))
    window = dict(sparse_mode=4, pre_tokens=1000, next_tokens=0)
    assert size(**window, sink_tokens=100000) >= size(**window)
    assert size(sink_tokens=100000) == size()
    assert size(**window, sink_tokens=1 << 60) >= size(**window)


def test_workspace_of_the_longest_bound():
    """Splits of the keys stay what a grid's second dimension holds: 16 rows of 64 sums, a maximum and a sum each."""
    g = PagedGeometry(B=1, N=1, N_kv=1, D=64, cu_seqlens_q=[1], num_pages=1, page_size=65536, max_pages=4096,
                      cache_dtype="e4m3")
    assert swa.swa_paged_forward_workspace_size(swa.PagedParams(g)) <= 65535 * (16 * (64 * 4 + 8) + 4) + 4096
