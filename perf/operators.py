"""Cases of the serving and position operators: rotary positions with several
axes (forward and backward), appending a chunk of new tokens to a paged cache
(with the rotation of q and k on the way), and attention of a chunk of new
tokens over the paged cache (chunked prefill, and its single-token form).

``run`` computes them in elementary torch operations, or through
attention_swa_forward_gb300.swa when ``own`` is set."""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NO_LIMIT = 2147483647


# ------------------------------------------------------------------ cases --
def attention(name, lens, chunk, N, N_kv, D, page, dtype="bf16", pre=NO_LIMIT, mode=4, cache="BNSD", seed=1):
    """`lens`, `chunk`: "lo-hi" ranges of the lengths of `count` sequences
    ("count*lo-hi", joined by "+"), drawn from the case's own seed."""
    return dict(name=name, op="attention", lens=lens, chunk=chunk, N=N, N_kv=N_kv, D=D, page=page, dtype=dtype,
                pre=pre, mode=mode, cache=cache, lens_seed=seed)


def rotary(name, direction, layout, B, S, N, N_kv, D, sections, rotary_dim=0, interleaved=False, dtype="bf16",
           start=0):
    return dict(name=name, op="rotary", direction=direction, layout=layout, B=B, S=S, N=N, N_kv=N_kv, D=D,
                sections=sections, rotary_dim=rotary_dim or D, interleaved=interleaved, dtype=dtype, start=start)


def append(name, lens, chunk, N, N_kv, D, page, sections, dtype="bf16", cache="BNSD", seed=1):
    return dict(name=name, op="append", lens=lens, chunk=chunk, N=N, N_kv=N_kv, D=D, page=page, sections=sections,
                rotary_dim=D, interleaved=False, dtype=dtype, cache=cache, lens_seed=seed)


def listed():
    return [
        # one conversation, one token at a time: latency
        attention("attention_token_x1", "1*1003-1003", "1*1-1", 32, 8, 128, 16, pre=4096),
        # a serving batch past its window: the bytes of 64 windows
        attention("attention_token_x64_window", "64*200-32768", "64*1-1", 32, 8, 128, 64, pre=4096, seed=2),
        # heads without sharing, half the head dim, fp16, pages of 48 slots
        attention("attention_token_x24_mha_fp16", "24*1-8192", "24*1-1", 16, 16, 64, 48, dtype="fp16", mode=0,
                  cache="TND", seed=3),
        # one very long context, four tokens checked at once: split over the keys
        attention("attention_4_tokens_of_131072", "1*131072-131072", "1*4-4", 32, 8, 128, 64, cache="TND"),
        # one chunk of a long prompt under the headline workload's window
        attention("attention_chunk_2048_window", "1*32768-32768", "1*2048-2048", 32, 8, 128, 64, pre=4096),
        # a mixed batch: chunks of prompts beside single tokens, an odd head dim
        attention("attention_mixed_fp16", "3*700-2500+13*1-4000", "3*150-700+13*1-1", 16, 4, 96, 32, dtype="fp16",
                  cache="TND", seed=4),
        # a whole prompt in one chunk
        attention("attention_prompt_8192", "1*8192-8192", "1*8192-8192", 32, 8, 128, 128),
        # training on images and video: the headline workload's q with shared key heads, three axes
        rotary("rotary_video_32768", "forward", "BNSD", 1, 32768, 32, 8, 128, "16,24,24"),
        # its gradient in fp32, pairs of neighbours, a part of the head, a ragged row count
        rotary("rotary_gradient_fp32", "backward", "TND", 1, 12345, 16, 16, 96, "10,14", rotary_dim=48,
               interleaved=True, dtype="fp32", start=100000),
        # a small batch of token rows: latency
        rotary("rotary_rows_64", "forward", "TND", 1, 64, 32, 8, 128, "64", dtype="fp16", start=30000),
        # the tokens of one decoding step: latency
        append("append_token_x64", "64*1-4096", "64*1-1", 32, 8, 128, 64, "64", seed=5),
        # prompts of images and text written to the cache
        append("append_prompts_fp16", "7*600-2100", "7*500-2000", 32, 8, 96, 48, "12,18,18", dtype="fp16",
               cache="TND", seed=6),
    ]


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "rotary", "append"])
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    dtype = rng.choice(["bf16", "fp16"])
    D = rng.choice([32, 40, 64, 72, 80, 96, 112, 120, 128])
    N_kv = rng.choice([1, 2, 4, 8])
    N = N_kv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    cache = rng.choice(["BNSD", "TND"])
    page = 16 * rng.choice([1, 2, 3, 4, 8, 16])
    half = D // 2
    cut = sorted(rng.sample(range(1, half), 2))
    sections = rng.choice([str(half), "%d,%d" % (cut[0], half - cut[0]),
                           "%d,%d,%d" % (cut[0], cut[1] - cut[0], half - cut[1])])
    if op == "rotary":
        B, S = rng.choice([1, 1, 2, 3]), log(1, 6000)
        c = rotary("", rng.choice(["forward", "backward"]), rng.choice(["BNSD", "TND"]), B, S, N, N_kv, D, sections,
                   interleaved=rng.random() < 0.4, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                   start=rng.choice([0, 0, 5000, 1000000]))
    elif op == "append":
        count, top = log(1, 40), log(2, 1500)
        c = append("", "%d*%d-%d" % (count, top, 2 * top), "%d*1-%d" % (count, top), N, N_kv, D, page, sections,
                   dtype=dtype, cache=cache, seed=rng.randrange(1 << 20))
    else:
        kind = rng.choice(["tokens", "tokens", "chunk", "mixed"])
        if kind == "tokens":
            count, top, few = log(1, 64), log(10, 12000), rng.choice([1, 1, 1, 2, 5])
            lens, chunk = "%d*%d-%d" % (count, few, top + few), "%d*%d-%d" % (count, few, few)
        elif kind == "chunk":
            top = log(20, 2500)
            lens, chunk = "1*%d-%d" % (top, 2 * top), "1*%d-%d" % (max(1, top // 2), top)
        else:
            a, b, top = rng.randint(1, 3), rng.randint(1, 12), log(20, 500)
            lens = "%d*%d-%d+%d*1-%d" % (a, top, 4 * top, b, 4 * top)
            chunk = "%d*1-%d+%d*1-1" % (a, top, b)
        c = attention("", lens, chunk, N, N_kv, D, page, dtype=dtype, cache=cache, seed=rng.randrange(1 << 20),
                      pre=rng.choice([NO_LIMIT, log(30, 4096)]), mode=rng.choice([4, 4, 4, 0]))
    del c["name"]
    return c


def lengths(case):
    """(cache length after the chunk, chunk length) of every sequence."""
    r = random.Random(case["lens_seed"])
    spans = lambda s: [tuple(int(x) for x in t) for p in s.split("+")
                       for t in [p.split("*")[1].split("-")] * int(p.split("*")[0])]
    q = [r.randint(*s) for s in spans(case["chunk"])]
    return [max(n, r.randint(*s)) for n, s in zip(q, spans(case["lens"]))], q


# ----------------------------------------------------------------- inputs --
def inverse_frequencies(case):
    R = case["rotary_dim"]
    return [10000.0 ** (-2.0 * i / R) for i in range(R // 2)]


def pair_axes(case):
    return [a for a, n in enumerate(case["sections"].split(",")) for _ in range(int(n))]


def positions_of(case, rows, start):
    """Integer positions [axes, rows]: time, height and width of patches."""
    t = torch.arange(rows, device="cuda", dtype=torch.int64)
    every = [start + t, start + t // 7 % 301, start + t % 53, start + t % 11]
    return torch.stack(every[: len(case["sections"].split(","))]).to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    dt = TYPES[case["dtype"]]
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)
    N, N_kv, D = case["N"], case["N_kv"], case["D"]
    s = {"case": case}
    if case["op"] == "rotary":
        B, S = case["B"], case["S"]
        bnsd = case["layout"] == "BNSD"
        s["x"] = randn(B, N, S, D) if bnsd else randn(B * S, N, D)
        s["y"] = randn(B, N_kv, S, D) if bnsd else randn(B * S, N_kv, D)
        s["positions"] = positions_of(case, B * S, case["start"])
        if bnsd:
            s["positions"] = s["positions"].view(-1, B, S)
    else:
        kv, q = lengths(case)
        page, B, T = case["page"], len(kv), sum(q)
        most = max(-(-n // page) for n in kv)
        used = sum(-(-n // page) for n in kv)
        order = torch.randperm(used, generator=g, device="cuda").to(torch.int32).cpu()
        table, at = torch.full((B, most), -1, dtype=torch.int32), 0
        for b, n in enumerate(kv):
            n = -(-n // page)
            table[b, :n] = order[at : at + n]
            at += n
        shape = (used, page, N_kv, D) if case["cache"] == "TND" else (used, N_kv, page, D)
        s.update(kv=kv, q=q, table=table.cuda(), kv_lens=torch.tensor(kv, dtype=torch.int32, device="cuda"),
                 k_pages=randn(*shape), v_pages=randn(*shape), x=randn(T, N, D))
        rows = torch.tensor([[b, n - m + i, b * max(q) + i] for b, (n, m) in enumerate(zip(kv, q)) for i in range(m)],
                            device="cuda")
        s["row_seq"], s["row_pos"], s["row_pad"] = rows[:, 0], rows[:, 1], rows[:, 2]
        if case["op"] == "append":
            s["y"], s["v"] = randn(T, N_kv, D), randn(T, N_kv, D)
            s["positions"] = positions_of(case, T, 0)
    if own:
        prepare_own(s)
    return s


def prepare_own(s):
    """The plan, workspace and output buffers that a serving loop keeps."""
    from attention_swa_forward_gb300 import swa
    from attention_swa_forward_gb300.workloads import PagedGeometry, RopeGeometry

    case = s["case"]
    if case["op"] != "attention":
        s["rope"] = swa.RopeParams(RopeGeometry(
            layout=case.get("layout", "TND"), B=case.get("B", 1), S=case.get("S", sum(s.get("q", []))), N=case["N"],
            N_kv=case["N_kv"], D=case["D"], rotary_dim=case["rotary_dim"], interleaved=case["interleaved"],
            sections=[int(x) for x in case["sections"].split(",")], dtype=case["dtype"]))
    s["x_out"] = torch.empty_like(s["x"])
    if case["op"] == "rotary":
        s["y_out"] = torch.empty_like(s["y"])
        return
    s["plan"] = swa.PagedParams(PagedGeometry(
        B=len(s["q"]), N=case["N"], N_kv=case["N_kv"], D=case["D"], cu_seqlens_q=np.cumsum(s["q"]).tolist(),
        cache_layout=case["cache"], num_pages=s["k_pages"].shape[0], page_size=case["page"],
        max_pages=s["table"].shape[1], max_kv_len=max(s["kv"]), scale=case["D"] ** -0.5,
        sparse_mode=case.get("mode", 4), pre_tokens=case.get("pre", NO_LIMIT), next_tokens=0, dtype=case["dtype"]))
    if case["op"] == "attention":
        s["workspace"] = swa.paged_forward_workspace(s["plan"], "cuda")
        s["smax"], s["ssum"] = (torch.empty(s["x"].shape[:2], device="cuda") for _ in range(2))
    else:
        s["workspace"] = swa.paged_append_workspace(s["plan"], "cuda")


# -------------------------------------------------------------------- run --
def run(s):
    op = s["case"]["op"]
    if own:
        return run_own(s)
    if op == "rotary":
        sign = 1.0 if s["case"]["direction"] == "forward" else -1.0
        cos, sin = angles(s["case"], s["positions"])
        cos, sin = cos[:, None], sin[:, None]  # [T, 1, pairs] or [B, 1, S, pairs]
        return rotate(s["case"], s["x"], cos, sin * sign), rotate(s["case"], s["y"], cos, sin * sign)
    return plain_append(s) if op == "append" else plain_attention(s)


def run_own(s):
    from attention_swa_forward_gb300 import swa

    case = s["case"]
    if case["op"] == "rotary":
        call = swa.rope if case["direction"] == "forward" else swa.rope_backward
        return call(s["rope"], s["x"], s["y"], s["positions"], s["x_out"], s["y_out"])
    if case["op"] == "append":
        swa.paged_append(s["plan"], s["y"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"],
                         rope=s["rope"], positions=s["positions"], q=s["x"], q_out=s["x_out"],
                         workspace=s["workspace"])
        return s["x_out"], s["k_pages"], s["v_pages"]
    return swa.paged_forward(s["plan"], s["x"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"],
                             out=s["x_out"], softmax_max=s["smax"], softmax_sum=s["ssum"],
                             workspace=s["workspace"])


def angles(case, positions):
    """cos and sin [..., pairs] in 32 bits of angles formed in 64."""
    freq = torch.tensor(inverse_frequencies(case), dtype=torch.float64, device="cuda")
    axis = torch.tensor(pair_axes(case), device="cuda")
    a = positions.movedim(0, -1).double()[..., axis] * freq
    return a.cos().float(), a.sin().float()


def rotate(case, x, cos, sin):
    R = case["rotary_dim"]
    f = x.float()
    if case["interleaved"]:
        a, b = f[..., 0:R:2], f[..., 1:R:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = f[..., : R // 2], f[..., R // 2 : R]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((y, f[..., R:]), dim=-1).to(x.dtype)


def plain_append(s):
    case = s["case"]
    cos, sin = angles(case, s["positions"])
    cos, sin = cos[:, None], sin[:, None]
    page = s["table"][s["row_seq"], s["row_pos"] // case["page"]].long()
    slot = s["row_pos"] % case["page"]
    at = (page, slot) if case["cache"] == "TND" else (page, slice(None), slot)
    s["k_pages"][at] = rotate(case, s["y"], cos, sin)
    s["v_pages"][at] = s["v"]
    return rotate(case, s["x"], cos, sin), s["k_pages"], s["v_pages"]


def plain_attention(s):
    """Padded to the longest chunk and window of the batch."""
    case, kv, q = s["case"], s["kv"], s["q"]
    N, N_kv, D, page, B, Lq = case["N"], case["N_kv"], case["D"], case["page"], len(kv), max(q)
    pre = case["pre"] if case["mode"] == 4 else NO_LIMIT
    first = [max(0, n - m - pre) for n, m in zip(kv, q)]
    span = max(n - f for n, f in zip(kv, first))
    j = torch.tensor(first, device="cuda")[:, None] + torch.arange(span, device="cuda")
    inside = j < s["kv_lens"][:, None]
    jc = torch.where(inside, j, s["kv_lens"][:, None] - 1)
    at = torch.gather(s["table"].long(), 1, jc // page)
    if case["cache"] == "TND":
        k, v = (t[at, jc % page].float() for t in (s["k_pages"], s["v_pages"]))
    else:
        k, v = (t[at, :, jc % page].float() for t in (s["k_pages"], s["v_pages"]))
    x = torch.zeros(B * Lq, N, D, device="cuda")
    x[s["row_pad"]] = s["x"].float()
    x = x.view(B, Lq, N_kv, N // N_kv, D)
    scores = torch.einsum("bihgd,bjhd->bhgij", x, k) * D ** -0.5
    i = (s["kv_lens"] - torch.tensor(q, device="cuda"))[:, None] + torch.arange(Lq, device="cuda")
    seen = inside[:, None, :]
    if case["mode"] == 4:
        seen = seen & (j[:, None, :] <= i[..., None]) & (j[:, None, :] >= i[..., None] - pre)
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(torch.isinf(m), 0.0, m)).exp_()
    l = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgij,bjhd->bihgd", p, v) / torch.where(l > 0, l, 1.0).permute(0, 3, 1, 2, 4)
    rows = lambda t: t[..., 0].permute(0, 3, 1, 2).reshape(B * Lq, N)[s["row_pad"]]
    return out.reshape(B * Lq, N, D)[s["row_pad"]].to(s["x"].dtype), rows(m), rows(l)


# ------------------------------------------------------------ work, exact --
def pairs_of(case):
    """Visible (query, key) pairs per head, and keys seen by some query."""
    pairs = keys = 0
    for n, m in zip(*lengths(case)):
        p = np.arange(n - m, n, dtype=np.int64)
        if case["mode"] == 4:
            lo = np.maximum(0, p - min(case["pre"], NO_LIMIT))
            pairs += int((p - lo + 1).sum())
            keys += n - int(lo.min())
        else:
            pairs += n * m
            keys += n
    return pairs, keys


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    N, N_kv, D = case["N"], case["N_kv"], case["D"]
    if case["op"] == "rotary":
        rows, axes = case["B"] * case["S"], len(case["sections"].split(","))
        return {"bytes": rows * (2 * (N + N_kv) * D * size + 4 * axes), "flops": 3 * rows * (N + N_kv) * D}
    T = sum(lengths(case)[1])
    if case["op"] == "append":
        axes = len(case["sections"].split(","))
        return {"bytes": T * (2 * (N + 2 * N_kv) * D * size + 4 * axes), "flops": 3 * T * (N + N_kv) * D}
    pairs, keys = pairs_of(case)
    return {"bytes": 2 * keys * N_kv * D * size + T * N * (2 * D * size + 8), "flops": 4 * D * N * pairs}


def exact(case, seed):
    """In 64 bits, sequence by sequence: the rotation as a product with
    e^(i angle), attention as a weighted mean over the visible keys."""
    s = prepare(case, seed)
    if case["op"] == "rotary":
        pos = s["positions"].reshape(s["positions"].shape[0], -1)
        back = case["direction"] == "backward"
        return tuple(turned(case, t, pos, back) for t in (s["x"], s["y"]))
    seqs = list(zip(s["kv"], s["q"], np.cumsum([0] + s["q"]).tolist()))
    page = case["page"]

    def places(b, n):  # the pages of sequence b, token by token
        t = torch.arange(n, device="cuda")
        return s["table"][b].long()[t // page], t % page

    if case["op"] == "append":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        new = turned(case, s["y"], s["positions"], False)
        for b, (n, m, at) in enumerate(seqs):
            p, o = places(b, n)
            p, o = p[n - m :], o[n - m :]
            for h in range(case["N_kv"]):
                where = (p, o, torch.full_like(p, h)) if case["cache"] == "TND" else (p, torch.full_like(p, h), o)
                k.index_put_(where, new[at : at + m, h])
                v.index_put_(where, s["v"][at : at + m, h].double())
        return turned(case, s["x"], s["positions"], False), k, v
    N, N_kv, D = case["N"], case["N_kv"], case["D"]
    T = s["x"].shape[0]
    out = torch.zeros(T, N, D, dtype=torch.float64, device="cuda")
    top, total = (torch.zeros(T, N, dtype=torch.float64, device="cuda") for _ in range(2))
    for b, (n, m, at) in enumerate(seqs):
        p, o = places(b, n)
        for h in range(N_kv):
            k, v = (t[p, o, h].double() if case["cache"] == "TND" else t[p, h, o].double()
                    for t in (s["k_pages"], s["v_pages"]))
            for c in range(0, m, 1024):  # so many rows at a time
                e = min(m, c + 1024)
                here = n - m + torch.arange(c, e, device="cuda")
                lo = max(0, n - m + c - case["pre"]) if case["mode"] == 4 else 0
                hi = n - m + e if case["mode"] == 4 else n
                t = torch.arange(lo, hi, device="cuda")
                hide = torch.zeros(e - c, hi - lo, dtype=torch.bool, device="cuda")
                if case["mode"] == 4:
                    hide = (t > here[:, None]) | (here[:, None] - t > case["pre"])
                for n_q in range(h * (N // N_kv), (h + 1) * (N // N_kv)):
                    z = (s["x"][at + c : at + e, n_q].double() @ k[lo:hi].T) / math.sqrt(D)
                    z[hide] = -math.inf
                    big = z.max(dim=1).values
                    w = torch.exp(z - big[:, None])
                    sums = w.sum(dim=1)
                    out[at + c : at + e, n_q] = (w @ v[lo:hi]) / sums[:, None]
                    top[at + c : at + e, n_q], total[at + c : at + e, n_q] = big, sums
    return out, top, total


def turned(case, x, pos, back):
    """x [..., D] in 64 bits with its pairs turned by their angles; pos [axes, rows]."""
    R, half = case["rotary_dim"], case["rotary_dim"] // 2
    y = x.double().clone()
    rows = y if x.dim() == 3 else y.permute(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])
    first = [2 * i if case["interleaved"] else i for i in range(half)]
    second = [2 * i + 1 if case["interleaved"] else half + i for i in range(half)]
    axes, freq = pair_axes(case), inverse_frequencies(case)
    theta = torch.stack([pos[axes[i]].double() * freq[i] for i in range(half)], dim=1)
    z = torch.complex(rows[..., first], rows[..., second])
    z = z * torch.polar(torch.ones_like(theta), -theta if back else theta)[:, None, :]
    rows[..., first], rows[..., second] = z.real, z.imag
    if x.dim() == 4:
        rows = rows.view(x.shape[0], x.shape[2], x.shape[1], x.shape[3]).permute(0, 2, 1, 3)
    return rows
