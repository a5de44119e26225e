"""Refusals of the Python calls on tensors that do not fit: the arguments as they
should be are accepted, then one at a time is changed, and the refusal names it
before anything is enqueued.  (Without a GPU the first tensor's device is all
that a call gets to see.)"""
import pytest
import torch

from attention_swa_forward_gb300 import swa
from attention_swa_forward_gb300.workloads import PagedGeometry, RopeGeometry

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, N, N_KV, D, P, PAGES, MAX = 3, 4, 2, 64, 16, 10, 5
T = 9
CU = [1, 1, 9]


def geometry(layout="BNSD"):
    return PagedGeometry(B=B, N=N, N_kv=N_KV, D=D, cu_seqlens_q=CU, num_pages=PAGES, page_size=P, max_pages=MAX,
                         cache_layout=layout)


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def spread(t):
    """The same values with every second element of the last dimension between them."""
    return torch.stack((t, t), dim=-1).flatten(-2)[..., ::2]


# what makes a tensor of any argument unfit
WRONG = {
    "a row less": lambda t: t[:-1],
    "a row more": lambda t: torch.cat((t, t[:1])),
    "one element less in the last dimension": lambda t: t[..., :-1],
    "a dimension more": lambda t: t[None],
    "flattened": lambda t: t.flatten(),
    "another type": lambda t: t.long() if t.dtype == torch.int32 else t.half(),
    "a wider type": lambda t: t.double(),
    "on the host": lambda t: t.cpu(),
    "gaps in the last dimension": spread,
    "not a tensor": lambda t: t.tolist(),
}
DENSE = {"last two dimensions swapped in memory": lambda t: t.transpose(-1, -2).contiguous().transpose(-1, -2)}


def refusals(names, dense=()):
    return [(n, w) for n in names for w in [*WRONG, *(DENSE if n in dense else ())]
            if not (n in ("kv_lens",) and w == "flattened")]


def refused(call, args, name, wrong, **kw):
    bad = dict(args)
    bad[name] = {**WRONG, **DENSE}[wrong](args[name])
    with pytest.raises(ValueError, match="CUDA device" if wrong == "on the host" else rf"\b{name}\b"):
        call(**bad, **kw)
    torch.cuda.synchronize()


def forward_args(layout="BNSD"):
    pages = zeros(*geometry(layout).page_shape())
    return dict(q=zeros(T, N, D), k_pages=pages, v_pages=pages.clone(), block_table=zeros(B, MAX, dtype=torch.int32),
                kv_lens=torch.full((B,), 8, dtype=torch.int32, device=DEV), out=zeros(T, N, D),
                softmax_max=zeros(T, N, dtype=torch.float32), softmax_sum=zeros(T, N, dtype=torch.float32))


@pytest.mark.parametrize("name,wrong", refusals(
    ["q", "k_pages", "v_pages", "block_table", "kv_lens", "out", "softmax_max", "softmax_sum"],
    ["q", "out", "softmax_max", "softmax_sum"]))
def test_paged_forward(name, wrong):
    args = forward_args()
    swa.paged_forward(geometry(), **args)
    refused(lambda **kw: swa.paged_forward(geometry(), **kw), args, name, wrong)


@pytest.mark.parametrize("layout", ["BNSD", "TND"])
def test_pages_of_the_other_layout(layout):
    args = forward_args(layout)
    swa.paged_forward(geometry(layout), **args)
    other = {"BNSD": "TND", "TND": "BNSD"}[layout]
    with pytest.raises(ValueError, match="k_pages"):
        swa.paged_forward(geometry(other), **args)


def append_args():
    pages = zeros(*geometry().page_shape())
    return dict(k=zeros(T, N_KV, D), v=zeros(T, N_KV, D), k_pages=pages, v_pages=pages.clone(),
                block_table=torch.arange(B * MAX, dtype=torch.int32, device=DEV).view(B, MAX) % PAGES,
                kv_lens=torch.tensor([1, 0, 8], dtype=torch.int32, device=DEV), q=zeros(T, N, D), q_out=zeros(T, N, D),
                positions=zeros(2, T, dtype=torch.int32))


APPEND_ROPE = RopeGeometry("TND", 1, T, N, D, N_kv=N_KV, sections=[16, 16])


@pytest.mark.parametrize("name,wrong", refusals(
    ["k", "v", "k_pages", "v_pages", "block_table", "kv_lens", "q", "q_out", "positions"], ["k", "v", "q", "q_out"]))
def test_paged_append(name, wrong):
    args = append_args()
    swa.paged_append(geometry(), rope=APPEND_ROPE, **args)
    refused(lambda **kw: swa.paged_append(geometry(), rope=APPEND_ROPE, **kw), args, name, wrong)


def test_positions_of_another_number_of_axes():
    args = append_args()
    for bad in (zeros(1, 2, T, dtype=torch.int32), zeros(1, T, dtype=torch.int32), zeros(T, 2, dtype=torch.int32)):
        with pytest.raises(ValueError, match="positions"):
            swa.paged_append(geometry(), rope=APPEND_ROPE, **{**args, "positions": bad})
    with pytest.raises(ValueError, match="positions"):
        swa.paged_append(geometry(), **{**args, "q": None, "q_out": None})
    with pytest.raises(swa.SwaError):
        swa.paged_append(geometry(), **{**args, "positions": None})


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("layout", ["BNSD", "TND"])
@pytest.mark.parametrize("name,wrong", refusals(["q", "k", "q_out", "k_out", "positions"], ["q", "k", "q_out", "k_out"]))
def test_rope(layout, back, name, wrong):
    geom = RopeGeometry(layout, 2, 7, N, D, N_kv=N_KV, sections=[20, 12])
    shape = lambda n: (2, n, 7, D) if layout == "BNSD" else (14, n, D)
    args = dict(q=zeros(*shape(N)), k=zeros(*shape(N_KV)), q_out=zeros(*shape(N)), k_out=zeros(*shape(N_KV)),
                positions=zeros(2, 14, dtype=torch.int32))

    def call(q, k, q_out, k_out, positions):
        fn = swa.rope_backward if back else swa.rope
        return fn(geom, q, k, positions, q_out, k_out)

    call(**args)
    call(**{**args, "positions": args["positions"].view(2, 2, 7)})
    refused(call, args, name, wrong)


def test_table_rows_that_overlap():
    args = forward_args()
    for bad in (args["block_table"][:1].expand(B, MAX), zeros(B * MAX, dtype=torch.int32).as_strided((B, MAX), (2, 1)),
                zeros(B, 2 * MAX, dtype=torch.int32)[:, ::2]):
        with pytest.raises(ValueError, match="block_table"):
            swa.paged_forward(geometry(), **{**args, "block_table": bad})


def test_pointers_off_their_alignment():
    """A slice that starts inside 16 bytes is refused by the library, by name."""
    args = forward_args()
    off = lambda t: torch.cat((t.flatten(), t.flatten()[:8]))[1:t.numel() + 1].view(t.shape)
    for name in ("q", "k_pages", "v_pages", "out"):
        with pytest.raises(swa.SwaError, match=name) as e:
            swa.paged_forward(geometry(), **{**args, name: off(args[name])})
        assert e.value.status == swa.SWA_ERR_PARAM_INVALID
    ws = swa.paged_forward_workspace(geometry(), DEV)
    with pytest.raises(swa.SwaError) as e:
        swa.paged_forward(geometry(), **args, workspace=ws[:-1])
    assert e.value.status == swa.SWA_ERR_WORKSPACE
    # queries that repeat rows are not taken
    with pytest.raises(swa.SwaError) as e:
        swa.paged_forward(geometry(), **{**args, "q": args["q"][:1].expand(T, N, D)})
    assert e.value.status == swa.SWA_ERR_PARAM_INVALID
