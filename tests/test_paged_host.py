"""Host-side checks of the rotary and paged-cache operators (no GPU): the
ctypes mirrors match the C structs, the defaults are the documented ones, and
every refusal returns its status before any CUDA work."""
import ctypes
import os
import subprocess

import pytest

from attention_swa_forward_gb300 import build as B
from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import PagedGeometry, RopeGeometry

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced: every case fails its checks first
OK, NULL, BAD, UNSUP, WS = (swa.SWA_OK, swa.SWA_ERR_PARAM_NULLPTR, swa.SWA_ERR_PARAM_INVALID,
                            swa.SWA_ERR_UNSUPPORTED, swa.SWA_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return swa.lib()


def test_ctypes_structs_match_c_layout(tmp_path):
    structs = {"swa_rope_params_t": swa.SwaRopeParams, "swa_paged_params_t": swa.SwaPagedParams,
               "swa_strides_t": swa.SwaStrides, "swa_page_strides_t": swa.SwaPageStrides}
    lines = []
    for c, py in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        lines += [f'printf("%zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "swa.h"\nint main(void){' + "".join(lines) +
                   "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    want = []
    for py in structs.values():
        want.append(ctypes.sizeof(py))
        want += [getattr(py, f).offset for f, _ in py._fields_]
    assert got == want


def test_defaults(lib):
    r, p = swa.SwaRopeParams(), swa.SwaPagedParams()
    lib.swa_rope_params_default(ctypes.byref(r))
    lib.swa_paged_params_default(ctypes.byref(p))
    assert (r.n_axes, r.base, r.N_kv, r.rotary_dim, r.interleaved) == (1, 10000.0, 0, 0, 0)
    assert (p.scale, p.pre_tokens, p.next_tokens, p.sparse_mode, p.max_kv_len) == (1.0, 2147483647, 2147483647, 0, 0)


# ------------------------------------------------------------------ rotary --
ROPE = dict(layout="TND", B=1, S=16, N=4, D=64, N_kv=2)


def rope_status(lib, change=None, fields=None, backward=False, **args):
    p = swa.RopeParams(RopeGeometry(**{**ROPE, **(change or {})}))
    for k, v in (fields or {}).items():
        setattr(p.c, k, v)
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, pos=FAKE, qo=FAKE, qos=None, ko=FAKE, kos=None)
    a.update(args)
    fn = lib.swa_rope_backward if backward else lib.swa_rope_forward
    return fn(p.ref(), *(ctypes.byref(x) if isinstance(x, swa.SwaStrides) else x for x in a.values()), None)


S = swa.SwaStrides


@pytest.mark.parametrize("want,case", [
    (NULL, dict(q=None)), (NULL, dict(q=None, qo=None, k=None, ko=None)), (NULL, dict(pos=None)),
    (NULL, dict(ko=None)), (BAD, dict(q=FAKE + 8)), (BAD, dict(ko=FAKE + 2)), (BAD, dict(pos=FAKE + 2)),
    (BAD, dict(fields=dict(N=0))), (BAD, dict(fields=dict(N=257))), (BAD, dict(fields=dict(N_kv=-1))),
    (BAD, dict(fields=dict(D=0))), (UNSUP, dict(fields=dict(D=136))), (UNSUP, dict(fields=dict(D=60))),
    (BAD, dict(fields=dict(S=0))), (BAD, dict(fields=dict(B=0))), (BAD, dict(fields=dict(B=1 << 20, S=1 << 20))),
    (BAD, dict(fields=dict(layout=2))), (BAD, dict(fields=dict(dtype=3))), (BAD, dict(fields=dict(interleaved=2))),
    (BAD, dict(fields=dict(rotary_dim=72))), (BAD, dict(fields=dict(rotary_dim=-8))),
    (UNSUP, dict(fields=dict(rotary_dim=12))), (BAD, dict(fields=dict(n_axes=0))), (BAD, dict(fields=dict(n_axes=5))),
    (BAD, dict(change=dict(sections=[16, 16]), fields=dict(n_axes=1))),
    (BAD, dict(fields=dict(inv_freq=None, base=0.0))), (BAD, dict(fields=dict(inv_freq=None, base=float("inf")))),
    (BAD, dict(change=dict(inv_freq=[float("nan")] * 32))), (BAD, dict(change=dict(inv_freq=[2.0 ** 21] * 32))),
    (BAD, dict(qs=S(0, 257, 64))), (BAD, dict(ks=S(0, -128, 64))), (BAD, dict(qos=S(0, 0, 64))),
    (BAD, dict(kos=S(0, 128, 8))), (BAD, dict(qs=S(0, 1 << 39, 64))),
    # rows of a result that overlap
    (BAD, dict(qos=S(0, 64, 64))), (BAD, dict(qos=S(0, 248, 64))), (BAD, dict(kos=S(0, 64, 1016))),
    (BAD, dict(change=dict(layout="BNSD", B=2, S=8), qos=S(2040, 64, 512))),
])
@pytest.mark.parametrize("backward", [False, True])
def test_rope_refusals(lib, want, case, backward):
    assert rope_status(lib, backward=backward, **case) == want, swa.swa_last_error()
    assert swa.swa_last_error()


def test_rope_params_in_python():
    with pytest.raises(ValueError):
        swa.RopeParams(RopeGeometry(**ROPE, sections=[10, 10]))
    with pytest.raises(ValueError):
        swa.RopeParams(RopeGeometry(**ROPE, inv_freq=[1.0]))


def test_rope_null_params(lib):
    assert lib.swa_rope_forward(None, FAKE, None, None, None, FAKE, FAKE, None, None, None, None) == NULL
    lib.swa_rope_params_default(None)
    lib.swa_paged_params_default(None)


# ------------------------------------------------------------------- paged --
PAGED = dict(B=3, N=4, D=64, cu_seqlens_q=[1, 1, 9], num_pages=10, page_size=16, max_pages=5, N_kv=2)


def paged(change=None, fields=None):
    p = swa.PagedParams(PagedGeometry(**{**PAGED, **(change or {})}))
    for k, v in (fields or {}).items():
        setattr(p.c, k, v)
    return p


@pytest.mark.parametrize("want,case", [
    (OK, dict()), (OK, dict(fields=dict(page_size=48))), (OK, dict(change=dict(cu_seqlens_q=[1, 9, 0]))),
    (BAD, dict(fields=dict(N=0))), (BAD, dict(fields=dict(N_kv=3))), (BAD, dict(fields=dict(N_kv=8))),
    (UNSUP, dict(fields=dict(D=129))), (BAD, dict(fields=dict(D=-8))), (UNSUP, dict(fields=dict(dtype=2))),
    (BAD, dict(fields=dict(dtype=7))), (BAD, dict(fields=dict(sparse_mode=2))),
    (BAD, dict(fields=dict(sparse_mode=4, pre_tokens=3, next_tokens=-4))),
    (OK, dict(fields=dict(sparse_mode=0, pre_tokens=3, next_tokens=-4))),
    (BAD, dict(fields=dict(scale=float("nan")))), (BAD, dict(fields=dict(scale=1e39))),
    (BAD, dict(fields=dict(cache_layout=5))),
    (BAD, dict(fields=dict(num_pages=0))), (BAD, dict(fields=dict(num_pages=1 << 31))),
    (BAD, dict(fields=dict(page_size=0))), (BAD, dict(fields=dict(page_size=1 << 17))),
    (UNSUP, dict(fields=dict(page_size=24))), (UNSUP, dict(fields=dict(page_size=8))),
    (BAD, dict(fields=dict(max_pages=0))), (BAD, dict(fields=dict(max_kv_len=-1))),
    (BAD, dict(fields=dict(max_kv_len=1 << 29))), (BAD, dict(fields=dict(B=0))), (BAD, dict(fields=dict(T_q=0))),
    (BAD, dict(fields=dict(T_q=8))), (BAD, dict(change=dict(cu_seqlens_q=[3, 2, 9]))),
    (BAD, dict(fields=dict(T_q=(1 << 20) + 1))),
])
def test_paged_parameter_checks(lib, want, case):
    p = paged(**case)
    n = ctypes.c_size_t(0)
    for fn in (lib.swa_paged_forward_workspace_size, lib.swa_paged_append_workspace_size):
        assert fn(p.ref(), ctypes.byref(n)) == want, swa.swa_last_error()
        if want == OK:
            assert n.value >= 256
        assert fn(p.ref(), None) == NULL
        assert fn(None, ctypes.byref(n)) == NULL
    for fn in (lib.swa_paged_forward_status, lib.swa_paged_append_status):
        assert fn(p.ref(), None, None) == (NULL if want == OK else want)


PS = swa.SwaPageStrides


def forward_status(lib, p=None, **args):
    p = p or paged()
    need = swa.swa_paged_forward_workspace_size(p)
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, v=FAKE, vs=None, table=FAKE, ts=0, lens=FAKE, out=FAKE, sm=FAKE, ss=FAKE,
             ws=FAKE, n=need)
    a.update(args)
    return lib.swa_paged_forward(p.ref(), *(ctypes.byref(x) if isinstance(x, ctypes.Structure) else x
                                            for x in a.values()), None)


@pytest.mark.parametrize("want,case", [
    (NULL, dict(q=None)), (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(table=None)),
    (NULL, dict(lens=None)), (NULL, dict(out=None)), (BAD, dict(q=FAKE + 8)), (BAD, dict(v=FAKE + 4)),
    (BAD, dict(out=FAKE + 1)), (BAD, dict(sm=FAKE + 2)), (BAD, dict(table=FAKE + 1)), (BAD, dict(lens=FAKE + 3)),
    (WS, dict(ws=None)), (WS, dict(ws=FAKE + 16)), (WS, dict(n=255)), (BAD, dict(ts=4)), (BAD, dict(ts=-5)),
    (BAD, dict(qs=S(0, 0, 64))), (BAD, dict(qs=S(0, 256, 60))), (BAD, dict(ks=PS(0, 64, 128))),
    (UNSUP, dict(ks=PS(2048 + 8, 1024, 64))), (UNSUP, dict(vs=PS(4096, 512, 64))), 
    (BAD, dict(vs=PS(2048, 1024, 60))), (BAD, dict(ks=PS(2048, 8, 64))), (BAD, dict(ks=PS(1 << 39, 1024, 64))),
])
def test_paged_forward_refusals(lib, want, case):
    assert forward_status(lib, **case) == want, swa.swa_last_error()


def append_status(lib, p=None, rope=None, **args):
    p = p or paged()
    need = swa.swa_paged_append_workspace_size(p)
    r = None
    if rope is not None:
        r = swa.RopeParams(RopeGeometry(**{**dict(layout="TND", B=1, S=9, N=4, D=64, N_kv=2), **rope})).ref()
    a = dict(k=FAKE, ks=None, v=FAKE, vs=None, kp=FAKE, kps=None, vp=FAKE, vps=None, table=FAKE, ts=0, lens=FAKE,
             rope=r, pos=None, q=None, qs=None, qo=None, qos=None, ws=FAKE, n=need)
    a.update(args)
    return lib.swa_paged_append(p.ref(), *(ctypes.byref(x) if isinstance(x, (S, PS)) else x for x in a.values()),
                                None)


@pytest.mark.parametrize("want,case", [
    (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(kp=None)), (NULL, dict(vp=None)),
    (NULL, dict(table=None)), (NULL, dict(lens=None)), (BAD, dict(k=FAKE + 8)), (BAD, dict(vp=FAKE + 8)),
    (WS, dict(ws=None)), (WS, dict(n=256)), (WS, dict(ws=FAKE + 128)),
    (BAD, dict(pos=FAKE)), (BAD, dict(q=FAKE, qo=FAKE)), (NULL, dict(rope={}, q=FAKE)), (NULL, dict(rope={}, qo=FAKE)),
    (BAD, dict(rope={}, q=FAKE + 8, qo=FAKE)), (BAD, dict(rope={}, pos=FAKE + 1)),
    (BAD, dict(rope=dict(S=8))), (BAD, dict(rope=dict(N=8))), (BAD, dict(rope=dict(N_kv=4))), (BAD, dict(rope=dict(D=72))),
    (BAD, dict(rope=dict(dtype="fp16"))), (BAD, dict(rope=dict(layout="BNSD"))),
    (BAD, dict(ks=S(0, 100, 64))), (BAD, dict(rope={}, q=FAKE, qo=FAKE, qos=S(0, 0, 64))),
    (BAD, dict(rope={}, q=FAKE, qo=FAKE, qos=S(0, 192, 64))),
    (BAD, dict(kps=PS(2048, 0, 64))), (BAD, dict(ts=3)),
])
def test_paged_append_refusals(lib, want, case):
    assert append_status(lib, **case) == want, swa.swa_last_error()


def test_python_wrappers_refuse_wrong_tensors():
    """Shapes, types and devices are checked before the library is called."""
    import torch

    g = PagedGeometry(**PAGED)
    q = torch.zeros(9, 4, 64, dtype=torch.bfloat16)
    kv = torch.zeros(9, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(g.page_shape(), dtype=torch.bfloat16)
    table, lens = torch.zeros(3, 5, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for bad in (dict(q=q[:8]), dict(q=q.float()), dict(k=pages[:, :1]), dict(table=table.long()),
                dict(table=table[:1].expand(3, 5)), dict(lens=lens[:2]), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        a = dict(q=q, k=pages, v=pages, table=table, lens=lens)
        a.update(bad)
        with pytest.raises(ValueError):
            swa.paged_forward(g, *a.values())
    for bad in (dict(k=kv[:, :1]), dict(v=kv.half()), dict(kp=pages[1:]), dict(lens=lens.long())):
        a = dict(k=kv, v=kv, kp=pages, vp=pages, table=table, lens=lens)
        a.update(bad)
        with pytest.raises(ValueError):
            swa.paged_append(g, *a.values())
    r = RopeGeometry("TND", 1, 9, 4, 64, N_kv=2)
    pos = torch.zeros(1, 9, dtype=torch.int32)
    for a in ((q, q, pos), (q, kv, pos.long()), (q, kv, pos[:, :8]), (None, None, pos), (q.float(), kv, pos)):
        with pytest.raises(ValueError):
            swa.rope(r, *a)
    with pytest.raises(ValueError):
        swa.PagedParams(PagedGeometry(**{**PAGED, "B": 2}))
