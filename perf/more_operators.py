"""Cases of the operators that a windowed model needs for long and for drafted
contexts: attention under a sliding window whose first tokens stay visible
(sinks), trained (forward and backward) and served from a paged cache;
attention of a tree of drafted tokens over that cache; and a cache of 8-bit
floats with an exponent per token and key/value head, quantised as it is
written, read back, and attended over.

``run`` computes them in elementary torch operations, or through
attention_swa_forward_gb300.swa when ``own`` is set."""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
NO_LIMIT = 2147483647
INF = math.inf
# exponents that a row of an 8-bit cache may have, per element type of the values it stands for
LEAST = {"bf16": -100, "fp16": -15}
MOST = 7


# ------------------------------------------------------------------ cases --
def training(name, layout, lens, N, N_kv, D, pre, sinks, dtype="bf16", seed=1):
    """Forward and backward.  lens: "count*length" (BNSD) or "count*lo-hi" joined by "+" (TND)."""
    return dict(name=name, op="training", layout=layout, lens=lens, N=N, N_kv=N_kv, D=D, pre=pre, sinks=sinks,
                dtype=dtype, lens_seed=seed)


def attention(name, lens, chunk, N, N_kv, D, page, dtype="bf16", pre=NO_LIMIT, sinks=0, tree=False, bits=16,
              cache="BNSD", seed=1):
    """Over a paged cache.  `lens`, `chunk`: "count*lo-hi" (joined by "+") lengths with the chunk, and of the chunk,
    drawn from the case's own seed.  tree: the chunk is a tree of drafted tokens."""
    return dict(name=name, op="attention", lens=lens, chunk=chunk, N=N, N_kv=N_kv, D=D, page=page, dtype=dtype,
                pre=pre, sinks=sinks, tree=tree, bits=bits, cache=cache, lens_seed=seed)


def write(name, lens, chunk, N_kv, D, page, dtype="bf16", cache="BNSD", seed=1):
    """A chunk quantised into the cache, and read back from it."""
    return dict(name=name, op="write", lens=lens, chunk=chunk, N=N_kv, N_kv=N_kv, D=D, page=page, dtype=dtype,
                bits=8, cache=cache, lens_seed=seed)


def read(name, lens, N_kv, D, page, dtype="bf16", cache="BNSD", seed=1):
    """Whole sequences read back from the cache."""
    return dict(name=name, op="read", lens=lens, chunk=lens, N=N_kv, N_kv=N_kv, D=D, page=page, dtype=dtype, bits=8,
                cache=cache, lens_seed=seed)


def listed():
    return [
        # the length and window of the long training workload, with shared key heads and the usual four sinks
        training("sinks_training_32768", "BNSD", "1*32768", 16, 4, 128, 4096, 4),
        # packed documents of unequal length, sinks past one tile, an odd head dim
        training("sinks_training_ragged_fp16", "TND", "7*1-5000", 12, 4, 96, 300, 150, dtype="fp16", seed=2),
        # a serving batch past its window: single tokens, whose window left the sinks' pages behind
        attention("sinks_token_x64", "64*200-32768", "64*1-1", 32, 8, 128, 64, pre=4096, sinks=4, seed=3),
        # a chunk of a long prompt beside single tokens
        attention("sinks_chunk_mixed_fp16", "1*9000-20000+11*30-9000", "1*1500-1500+11*1-1", 16, 4, 80, 48,
                  dtype="fp16", pre=1024, sinks=64, cache="TND", seed=4),
        # one conversation with a wide tree of drafts over a long context
        attention("tree_61_of_32768", "1*32768-32768", "1*61-61", 32, 8, 128, 64, tree=True, seed=5),
        # small trees of a batch under a window
        attention("tree_x24_window_fp16", "24*40-6000", "24*2-8", 16, 8, 64, 32, dtype="fp16", pre=2048, sinks=4,
                  tree=True, cache="TND", seed=6),
        # a serving batch from the 8-bit cache
        attention("e4m3_token_x64", "64*100-16384", "64*1-1", 32, 8, 128, 64, bits=8, seed=7),
        # a chunk of a prompt behind a long context in the 8-bit cache
        attention("e4m3_chunk_1024_of_16384", "1*16384-16384", "1*1024-1024", 32, 8, 128, 64, bits=8, seed=8),
        # the tokens of one decoding step: latency
        write("e4m3_write_token_x64", "64*1-4096", "64*1-1", 8, 128, 64, seed=9),
        # prompts written to the cache
        write("e4m3_write_prompts_fp16", "9*600-4100", "9*500-4000", 8, 96, 48, dtype="fp16", cache="TND", seed=10),
        # a few short sequences fetched for reuse: latency
        read("e4m3_read_x3_fp16", "3*1-200", 8, 64, 16, dtype="fp16", seed=11),
        # long sequences fetched for another engine
        read("e4m3_read_131072", "1*131072-131072", 8, 128, 64, cache="TND", seed=12),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    op = rng.choice(["training", "sinks", "tree", "e4m3", "e4m3", "write", "read"])
    dtype = rng.choice(["bf16", "fp16"])
    D = rng.choice([16, 40, 64, 72, 80, 96, 104, 128])
    N_kv = rng.choice([1, 2, 4, 8])
    N = N_kv * rng.choice([1, 2, 3, 4, 5, 8])
    cache, page = rng.choice(["BNSD", "TND"]), 16 * rng.choice([1, 2, 3, 4, 8])
    seed = rng.randrange(1 << 20)
    if op == "training":
        pre, sinks = log(1, 4096), log(1, 300)
        if rng.random() < 0.5:
            c = training("", "BNSD", "%d*%d" % (rng.choice([1, 1, 2]), log(48, 6000)), N, N_kv, D, pre, sinks, dtype)
        else:
            c = training("", "TND", "%d*20-%d" % (rng.randint(1, 9), log(200, 3000)), N, N_kv, D, pre, sinks, dtype,
                         seed)
    elif op == "write":
        count, top = log(1, 40), log(2, 1500)
        c = write("", "%d*%d-%d" % (count, top, 2 * top), "%d*1-%d" % (count, top), N_kv, D, page, dtype, cache, seed)
    elif op == "read":
        c = read("", "%d*1-%d" % (log(1, 40), log(2, 3000)), N_kv, D, page, dtype, cache, seed)
    else:
        tree, bits = op == "tree", 8 if op == "e4m3" else rng.choice([16, 16, 8])
        pre = rng.choice([NO_LIMIT, log(30, 4096)]) if op != "sinks" else log(30, 4096)
        sinks = 0 if pre == NO_LIMIT else rng.choice([0, log(1, 300)]) if op != "sinks" else log(1, 300)
        kind = "tokens" if tree else rng.choice(["tokens", "tokens", "chunk", "mixed"])
        if kind == "tokens":
            count, top = log(1, 48), log(10, 10000)
            few = log(2, 70) if tree else rng.choice([1, 1, 1, 2, 5])
            lens, chunk = "%d*%d-%d" % (count, few, top + few), "%d*%d-%d" % (count, max(1, few // 2), few)
        elif kind == "chunk":
            top = log(20, 2500)
            lens, chunk = "1*%d-%d" % (top, 3 * top), "1*%d-%d" % (max(1, top // 2), top)
        else:
            a, b, top = rng.randint(1, 3), rng.randint(1, 12), log(20, 500)
            lens = "%d*%d-%d+%d*1-%d" % (a, top, 4 * top, b, 4 * top)
            chunk = "%d*1-%d+%d*1-1" % (a, top, b)
        c = attention("", lens, chunk, N, N_kv, D, page, dtype, pre, sinks, tree, bits, cache, seed)
    del c["name"]
    return c


def spans(text):
    out = []
    for part in text.split("+"):
        count, span = part.split("*")
        lo, hi = (span.split("-") * 2)[:2]
        out += [(int(lo), int(hi))] * int(count)
    return out


def lengths(case):
    """(cache length after the chunk, chunk length) of every sequence; of a training case, its length twice."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "training":
        n = [r.randint(*s) for s in spans(case["lens"])]
        return n, n
    q = [r.randint(*s) for s in spans(case["chunk"])]
    if case["op"] == "read":
        return q, q
    return [max(n, r.randint(*s)) for n, s in zip(q, spans(case["lens"]))], q


# ----------------------------------------------------------------- inputs --
def draw_trees(case, seed):
    """The parent of every drafted token (an earlier token of its chunk, or -1: the last token of the context)."""
    r = random.Random("%s %s" % (case["lens_seed"], seed))
    out = []
    for m in lengths(case)[1]:
        out.append([-1 if i == 0 else max(-1, i - 1 - int(r.expovariate(0.4))) for i in range(m)])
    return out


def tree_inputs(case, seed):
    """Per token: the tokens of its chunk it sees (itself and its ancestors) as bits, and its depth."""
    trees = draw_trees(case, seed)
    words = -(-max(len(t) for t in trees) // 32)
    bits, depth = [], []
    for parents in trees:
        seen = []
        for i, p in enumerate(parents):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
            depth.append(depth[len(depth) - i + p] + 1 if p >= 0 else 0)
        bits += seen
    rows = [[(b >> 32 * w) & 0xFFFFFFFF for w in range(words)] for b in bits]
    mask = torch.from_numpy(np.array(rows, dtype=np.uint32).view(np.int32)).cuda()
    return mask, torch.tensor(depth, dtype=torch.int32, device="cuda")


def power(e):
    """2^e in 32 bits, from its bits (a power function may be off in the last place)."""
    return (e.int() + 127 << 23).view(torch.float32)


def encode(case, x):
    """Rows of x as 8-bit floats and the exponents that scale them: 2^e is the
    least power of two (in the type's limits) that brings the row within 448."""
    f = x.float()
    m, e = torch.frexp(f.abs().amax(-1))
    e = (e - 9 + (m > 0.875)).clamp(LEAST[case["dtype"]], MOST)
    e = torch.where(m == 0, LEAST[case["dtype"]], e).to(torch.int8)
    f = (f * power(-e)[..., None]).clamp(-448.0, 448.0)
    return f.to(torch.float8_e4m3fn), e


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    dt = TYPES[case["dtype"]]
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)
    N, N_kv, D = case["N"], case["N_kv"], case["D"]
    kv, q = lengths(case)
    s = {"case": case, "kv": kv, "q": q, "at": np.cumsum([0] + q).tolist()}
    if case["op"] == "training":
        shape = (lambda n: (len(q), n, q[0], D)) if case["layout"] == "BNSD" else (lambda n: (sum(q), n, D))
        s.update(x=randn(*shape(N)), k=randn(*shape(N_kv)), v=randn(*shape(N_kv)), dy=randn(*shape(N)))
    else:
        page, B, T = case["page"], len(kv), sum(q)
        most, used = max(-(-n // page) for n in kv), sum(-(-n // page) for n in kv)
        order = torch.randperm(used, generator=g, device="cuda").to(torch.int32).cpu()
        table, at = torch.full((B, most), -1, dtype=torch.int32), 0
        for b, n in enumerate(kv):
            n = -(-n // page)
            table[b, :n] = order[at : at + n]
            at += n
        shape = (used, page, N_kv, D) if case["cache"] == "TND" else (used, N_kv, page, D)
        # keys have a few channels far above the others, as models have them
        loud = torch.where(torch.rand(D, generator=g, device="cuda") < 0.05, 6.0, 1.0) if case["bits"] == 8 else None
        s.update(table=table.cuda(), kv_lens=torch.tensor(kv, dtype=torch.int32, device="cuda"))
        for name in ("k", "v"):
            pages = randn(*shape)
            if case["bits"] == 8:
                if name == "k":
                    pages = (pages.float() * loud).to(dt)
                pages, e = encode(case, pages)
                # exponents lie [pages, heads, slots] in either layout
                s[name + "_exp"] = (e.transpose(1, 2) if case["cache"] == "TND" else e).contiguous()
            s[name + "_pages"] = pages
        rows = torch.tensor([[b, n - m + i, b * max(q) + i] for b, (n, m) in enumerate(zip(kv, q)) for i in range(m)],
                            device="cuda")
        s["row_seq"], s["row_pos"], s["row_pad"] = rows[:, 0], rows[:, 1], rows[:, 2]
        if case["op"] == "attention":
            s["x"] = randn(T, N, D)
            if case["tree"]:
                s["tree"], s["depth"] = tree_inputs(case, seed)
        elif case["op"] == "write":
            s["y"], s["v"] = (randn(T, N_kv, D).float() * loud).to(dt), randn(T, N_kv, D)
    if own:
        prepare_own(s)
    return s


def prepare_own(s):
    """The plan, workspace and output buffers that a program keeps."""
    from attention_swa_forward_gb300 import swa
    from attention_swa_forward_gb300.workloads import Geometry, PagedGeometry

    case = s["case"]
    if case["op"] == "training":
        cu = np.cumsum(s["q"]).tolist()
        where = dict(S_q=s["q"][0], S_kv=s["q"][0]) if case["layout"] == "BNSD" else dict(
            cu_seqlens_q=cu, cu_seqlens_kv=cu)
        s["geom"] = Geometry(case["layout"], len(s["q"]), case["N"], case["D"], N_kv=case["N_kv"],
                             scale=case["D"] ** -0.5, sparse_mode=4, pre_tokens=case["pre"], next_tokens=0,
                             sink_tokens=case["sinks"], dtype=case["dtype"], **where)
        params = swa.Params(s["geom"])
        for name, size in (("fwd_ws", swa.swa_forward_workspace_size), ("bwd_ws", swa.swa_backward_workspace_size)):
            s[name] = torch.empty(size(params), dtype=torch.uint8, device="cuda")
        s["out"], s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[n]) for n in ("x", "x", "k", "v"))
        s["smax"], s["ssum"] = (torch.empty(s["x"].shape[:-1], device="cuda") for _ in range(2))
        return
    s["plan"] = swa.PagedParams(PagedGeometry(
        B=len(s["q"]), N=case["N"], N_kv=case["N_kv"], D=case["D"], cu_seqlens_q=np.cumsum(s["q"]).tolist(),
        cache_layout=case["cache"], num_pages=s["k_pages"].shape[0], page_size=case["page"],
        max_pages=s["table"].shape[1], max_kv_len=max(s["kv"]), scale=case["D"] ** -0.5, sparse_mode=4,
        pre_tokens=case.get("pre", NO_LIMIT), next_tokens=0, sink_tokens=case.get("sinks", 0), dtype=case["dtype"],
        cache_dtype="e4m3" if case["bits"] == 8 else ""))
    if case["op"] == "attention":
        s["workspace"] = swa.paged_forward_workspace(s["plan"], "cuda")
        s["x_out"] = torch.empty_like(s["x"])
        s["smax"], s["ssum"] = (torch.empty(s["x"].shape[:2], device="cuda") for _ in range(2))
        return
    s["k_out"], s["v_out"] = (torch.empty(sum(s["q"]), case["N_kv"], case["D"], dtype=TYPES[case["dtype"]],
                                          device="cuda") for _ in range(2))
    s["workspace"] = swa.paged_append_workspace(s["plan"], "cuda")


# -------------------------------------------------------------------- run --
def run(s):
    if own:
        return run_own(s)
    op = s["case"]["op"]
    if op == "training":
        return plain_training(s)
    if op == "attention":
        return plain_attention(s)
    if op == "write":
        plain_write(s)
    return plain_read(s)


def run_own(s):
    from attention_swa_forward_gb300 import swa

    op = s["case"]["op"]
    if op == "training":
        swa.forward(s["geom"], s["x"], s["k"], s["v"], out=s["out"], softmax_max=s["smax"], softmax_sum=s["ssum"],
                    workspace=s["fwd_ws"])
        swa.backward(s["geom"], s["x"], s["k"], s["v"], s["dy"], s["out"], s["smax"], s["ssum"], dq=s["dq"],
                     dk=s["dk"], dv=s["dv"], workspace=s["bwd_ws"])
        return tuple(s[n] for n in ("out", "smax", "ssum", "dq", "dk", "dv"))
    exponents = dict(k_exponents=s.get("k_exp"), v_exponents=s.get("v_exp"))
    cache = (s["k_pages"], s["v_pages"], s["table"], s["kv_lens"])
    if op == "attention":
        return swa.paged_forward(s["plan"], s["x"], *cache, out=s["x_out"], softmax_max=s["smax"],
                                 softmax_sum=s["ssum"], workspace=s["workspace"], tree=s.get("tree"),
                                 depth=s.get("depth"), **exponents)
    if op == "write":
        swa.paged_append(s["plan"], s["y"], s["v"], *cache, workspace=s["workspace"], **exponents)
    return swa.paged_gather(s["plan"], *cache, k=s["k_out"], v=s["v_out"], workspace=s["workspace"], **exponents)


def sequences(s):
    """Query head groups and key/value heads of every sequence of a training case, [G, n, D] and [n, D]."""
    case = s["case"]
    G = case["N"] // case["N_kv"]
    for b in range(len(s["q"])):
        for h in range(case["N_kv"]):
            if case["layout"] == "BNSD":
                heads, one = (b, slice(h * G, h * G + G)), (b, h)
                yield heads, one, lambda t: t, s["q"][b]
            else:
                rows = slice(s["at"][b], s["at"][b + 1])
                heads, one = (rows, slice(h * G, h * G + G)), (rows, h)
                yield heads, one, lambda t: t.transpose(0, 1), s["q"][b]


def plain_training(s):
    """Blocks of queries over the window's keys and, apart from them, the sinks before it."""
    case, scale = s["case"], s["case"]["D"] ** -0.5
    x = s["x"]
    out, dq = torch.empty_like(x), torch.empty_like(x)
    dk, dv = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    smax, ssum = (torch.empty(x.shape[:-1], device="cuda") for _ in range(2))
    for heads, one, flip, n in sequences(s):
        q, dy = flip(x[heads]).float(), flip(s["dy"][heads]).float()
        k, v = s["k"][one].float(), s["v"][one].float()
        gk, gv = torch.zeros_like(k), torch.zeros_like(v)
        o, gq = torch.empty_like(q), torch.empty_like(q)
        mx, sm = (torch.empty(q.shape[:2], device="cuda") for _ in range(2))
        for c in range(0, n, 2048):
            e = min(n, c + 2048)
            lo = max(0, c - case["pre"])
            keys = torch.cat((torch.arange(min(case["sinks"], lo), device="cuda"), torch.arange(lo, e, device="cuda")))
            i = torch.arange(c, e, device="cuda")[:, None]
            seen = (keys <= i) & ((keys >= i - case["pre"]) | (keys < case["sinks"]))
            kb, vb = k[keys], v[keys]
            p = (q[:, c:e] @ kb.T).mul_(scale).masked_fill_(~seen, -INF)
            m = p.amax(-1, keepdim=True)
            p = p.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            p = p.div_(l)
            o[:, c:e] = ob = p @ vb
            d = dy[:, c:e]
            ds = (d @ vb.T).sub_((d * ob).sum(-1, keepdim=True)).mul_(p)
            gq[:, c:e] = (ds @ kb).mul_(scale)
            gv.index_add_(0, keys, (p.transpose(1, 2) @ d).sum(0))
            gk.index_add_(0, keys, (ds.transpose(1, 2) @ q[:, c:e]).sum(0).mul_(scale))
            mx[:, c:e], sm[:, c:e] = m[..., 0], l[..., 0]
        out[heads], dq[heads] = flip(o).to(x.dtype), flip(gq).to(x.dtype)
        dk[one], dv[one] = gk.to(x.dtype), gv.to(x.dtype)
        smax[heads], ssum[heads] = flip(mx), flip(sm)
    return out, smax, ssum, dq, dk, dv


def fetch(s, name, seq, pos):
    """Values of the cache at places (seq, pos) of any shape, [..., N_kv, D] in 32 bits."""
    case = s["case"]
    page, slot = s["table"].long()[seq, pos // case["page"]], pos % case["page"]
    t = s[name + "_pages"]
    t = t.view(torch.uint8) if case["bits"] == 8 else t
    x = t[page, slot] if case["cache"] == "TND" else t[page, :, slot]
    if case["bits"] == 8:
        e = s[name + "_exp"][page, :, slot]
        return x.view(torch.float8_e4m3fn).float() * power(e)[..., None]
    return x.float()


def plain_attention(s):
    """Padded to the longest chunk, and to the sinks and the longest window of the batch."""
    case, kv, q = s["case"], s["kv"], s["q"]
    N, N_kv, D, B, Lq, pre = case["N"], case["N_kv"], case["D"], len(kv), max(q), case["pre"]
    first = torch.tensor([max(0, n - m - pre) for n, m in zip(kv, q)], device="cuda")
    span = max(n - max(0, n - m - pre) for n, m in zip(kv, q))
    j = first[:, None] + torch.arange(span, device="cuda")
    n_sinks = min(case["sinks"], int(max(max(0, n - m - pre) for n, m in zip(kv, q))))
    sink = torch.arange(n_sinks, device="cuda").expand(B, -1)
    inside = torch.cat((sink < first[:, None], j < s["kv_lens"][:, None]), dim=1)
    j = torch.cat((sink, j), dim=1)
    jc = torch.minimum(j, s["kv_lens"][:, None].long() - 1)
    seq = torch.arange(B, device="cuda")[:, None]
    k, v = fetch(s, "k", seq, jc), fetch(s, "v", seq, jc)
    x = torch.zeros(B * Lq, N, D, device="cuda")
    x[s["row_pad"]] = s["x"].float()
    x = x.view(B, Lq, N_kv, N // N_kv, D)
    scores = torch.einsum("bihgd,bjhd->bhgij", x, k) * D ** -0.5
    prefix = (s["kv_lens"] - torch.tensor(q, device="cuda", dtype=torch.int32)).long()
    if case["tree"]:
        depth = torch.zeros(B * Lq, dtype=torch.long, device="cuda")
        depth[s["row_pad"]] = s["depth"].long()
        i = prefix[:, None] + depth.view(B, Lq)
        words = torch.zeros(B * Lq, s["tree"].shape[1], dtype=torch.long, device="cuda")
        words[s["row_pad"]] = s["tree"].long() & 0xFFFFFFFF
        own_j = j - prefix[:, None]  # >= 0: a token of the chunk
        at = own_j.clamp(0, 32 * words.shape[1] - 1)
        word = torch.gather(words.view(B, Lq, -1), 2, (at // 32)[:, None].expand(-1, Lq, -1))
        drafted = (word >> (at % 32)[:, None]) & 1 > 0
        window = (j[:, None] >= i[..., None] - pre) | (j < case["sinks"])[:, None]
        seen = inside[:, None] & torch.where((own_j >= 0)[:, None], drafted, window)
    else:
        i = prefix[:, None] + torch.arange(Lq, device="cuda")
        window = (j[:, None] >= i[..., None] - pre) | (j < case["sinks"])[:, None]
        seen = inside[:, None] & (j[:, None] <= i[..., None]) & window
    scores = scores.masked_fill(~seen[:, None, None], -INF)
    m = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(torch.isinf(m), 0.0, m)).exp_()
    l = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgij,bjhd->bihgd", p, v) / torch.where(l > 0, l, 1.0).permute(0, 3, 1, 2, 4)
    rows = lambda t: t[..., 0].permute(0, 3, 1, 2).reshape(B * Lq, N)[s["row_pad"]]
    return out.reshape(B * Lq, N, D)[s["row_pad"]].to(s["x"].dtype), rows(m), rows(l)


def plain_write(s):
    case = s["case"]
    page = s["table"][s["row_seq"], s["row_pos"] // case["page"]].long()
    slot = s["row_pos"] % case["page"]
    at = (page, slot) if case["cache"] == "TND" else (page, slice(None), slot)
    for name, x in (("k", s["y"]), ("v", s["v"])):
        codes, e = encode(case, x)
        s[name + "_pages"].view(torch.uint8)[at] = codes.view(torch.uint8)
        s[name + "_exp"][page, :, slot] = e


def plain_read(s):
    dt = TYPES[s["case"]["dtype"]]
    return tuple(fetch(s, name, s["row_seq"], s["row_pos"]).to(dt) for name in ("k", "v"))


# ------------------------------------------------------------ work, exact --
def visible(case, n, m):
    """Pairs of a query and a key it sees, and the keys that some query sees, of a causal chunk of m of n tokens."""
    i = np.arange(n - m, n, dtype=np.int64)
    lo = np.maximum(0, i - case["pre"])
    pairs = int((i - lo + 1).sum() + np.minimum(case["sinks"], lo).sum())
    first = int(lo.min()) if m else 0
    return pairs, n - first + min(case["sinks"], first)


def work(case):
    N, N_kv, D = case["N"], case["N_kv"], case["D"]
    kv, q = lengths(case)
    T = sum(q)
    row = N_kv * (D + 1 if case.get("bits") == 8 else 2 * D)  # bytes of a token's keys (or values) in the cache
    if case["op"] == "training":
        pairs = sum(visible(case, n, n)[0] for n in q)
        # forward: q, k, v read, out and statistics written; backward: q, k, v, dy, out, statistics read, three written
        return {"bytes": T * (2 * D * (6 * N + 6 * N_kv) + 16 * N), "flops": 14 * D * N * pairs}
    if case["op"] == "write":
        return {"bytes": T * (2 * N_kv * 2 * D * 2 + 2 * row), "flops": 4 * T * N_kv * D}
    if case["op"] == "read":
        return {"bytes": T * (2 * N_kv * D * 2 + 2 * row), "flops": 2 * T * N_kv * D}
    counts = [visible(case, n, m) for n, m in zip(kv, q)]
    keys = sum(c[1] for c in counts)
    pairs = sum(c[0] for c in counts)
    extra = 0
    if case["tree"]:
        # about half of a causal chunk's own pairs at most: count the context, and the bits
        pairs = sum(m * (min(n - m, case["pre"]) + 1) for n, m in zip(kv, q))
        extra = T * (4 * -(-max(q) // 32) + 4)
    return {"bytes": 2 * keys * row + T * N * (4 * D + 8) + extra, "flops": 4 * D * N * pairs}


def exact(case, seed):
    """In 64 bits, head by head and a few rows at a time, from a matrix that says who sees whom."""
    s = prepare(case, seed)
    kv, q, at = s["kv"], s["q"], s["at"]
    N, N_kv, D = case["N"], case["N_kv"], case["D"]
    G = N // N_kv
    dev = dict(dtype=torch.float64, device="cuda")
    if case["op"] in ("write", "read"):
        if case["op"] == "write":
            return tuple(nearest(case, t) for t in (s["y"], s["v"]))
        return tuple(torch.cat([cached(s, name, b, n) for b, n in enumerate(q)]) for name in ("k", "v"))
    if case["op"] == "training":
        bnsd = case["layout"] == "BNSD"
        res = {n: torch.zeros(s[t].shape, **dev) for n, t in (("o", "x"), ("dq", "x"), ("dk", "k"), ("dv", "v"))}
        top, total = (torch.zeros(s["x"].shape[:-1], **dev) for _ in range(2))
        for b in range(len(q)):
            pick = lambda t, h: t[b, h] if bnsd else t[at[b] : at[b + 1], h]
            for h in range(N):
                x, dy = pick(s["x"], h).double(), pick(s["dy"], h).double()
                k, v = pick(s["k"], h // G).double(), pick(s["v"], h // G).double()
                gk, gv = pick(res["dk"], h // G), pick(res["dv"], h // G)
                for c in range(0, q[b], 1024):
                    e = min(q[b], c + 1024)
                    hide = hidden(case, torch.arange(c, e, device="cuda"), torch.arange(e, device="cuda"))
                    live = (~hide).any(0).nonzero()[:, 0]
                    big, sums, w, o = weighted(x[c:e], k[live], v[live], hide[:, live])
                    grad = w * (dy[c:e] @ v[live].T - (dy[c:e] * o).sum(1, keepdim=True)) / math.sqrt(D)
                    pick(res["o"], h)[c:e], pick(res["dq"], h)[c:e] = o, grad @ k[live]
                    gv[live] += w.T @ dy[c:e]
                    gk[live] += grad.T @ x[c:e]
                    pick(top, h)[c:e], pick(total, h)[c:e] = big, sums
        return res["o"], top, total, res["dq"], res["dk"], res["dv"]
    out, top, total = torch.zeros(sum(q), N, D, **dev), torch.zeros(sum(q), N, **dev), torch.zeros(sum(q), N, **dev)
    trees = draw_trees(case, seed) if case["tree"] else None
    for b, (n, m) in enumerate(zip(kv, q)):
        k, v = cached(s, "k", b, n), cached(s, "v", b, n)
        for c in range(0, m, 1024):
            e = min(m, c + 1024)
            j = torch.arange(n, device="cuda")
            if trees:
                line, hide = [], torch.ones(m, n, dtype=torch.bool)
                for i, parent in enumerate(trees[b]):
                    line.append((line[parent] if parent >= 0 else []) + [i])
                    here = n - m + len(line[i]) - 1
                    hide[i, max(0, here - case["pre"]) : n - m] = False
                    hide[i, : min(case["sinks"], n - m)] = False
                    hide[i, [n - m + a for a in line[i]]] = False
                hide = hide[c:e].cuda()
            else:
                hide = hidden(case, n - m + torch.arange(c, e, device="cuda"), j)
            live = (~hide).any(0).nonzero()[:, 0]
            for h in range(N):
                big, sums, _, o = weighted(s["x"][at[b] + c : at[b] + e, h].double(), k[live, h // G], v[live, h // G],
                                           hide[:, live])
                rows = slice(at[b] + c, at[b] + e)
                out[rows, h], top[rows, h], total[rows, h] = o, big, sums
    return out, top, total


def hidden(case, i, j):
    """Keys j that queries at positions i do not see."""
    late = j[None] > i[:, None]
    old = (i[:, None] - j[None] > case["pre"]) & (j[None] >= case["sinks"])
    return late | old


def weighted(x, k, v, hide):
    z = (x @ k.T) / math.sqrt(x.shape[1])
    z[hide] = -INF
    big = z.max(dim=1).values
    w = torch.exp(z - big[:, None])
    sums = w.sum(dim=1)
    w = w / sums[:, None]
    return big, sums, w, w @ v


def cached(s, name, b, n):
    """Sequence b's n keys or values, [n, N_kv, D], page by page."""
    case, parts = s["case"], []
    pages = s[name + "_pages"]
    for e in range(-(-n // case["page"])):
        p = int(s["table"][b, e])
        t = pages[p].double() if case["cache"] == "TND" else pages[p].double().transpose(0, 1)
        if case["bits"] == 8:
            t = t * doubled(s[name + "_exp"][p]).T[..., None]
        parts.append(t)
    return torch.cat(parts)[:n] if parts else torch.zeros(0, case["N_kv"], case["D"], dtype=torch.float64,
                                                          device="cuda")


def nearest(case, x):
    """x [T, N_kv, D] on the grid of its rows' 8-bit floats, by arithmetic: 3
    bits behind the leading one, steps of 2^-9 at least, half to even."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    e = torch.full_like(top, LEAST[case["dtype"]])
    for n in range(LEAST[case["dtype"]], MOST):  # one more for as long as the row does not fit
        e += top > 448.0 * 2.0 ** n
    y = x * doubled(-e)
    n = torch.full_like(y, -9.0)  # the exponent of y's step
    for k in range(-5, 9):
        n += y.abs() >= 2.0 ** k
    return torch.round(y * doubled(-n)).mul(doubled(n)).clamp(-448.0, 448.0) * doubled(e)


def doubled(e):
    """2^e in 64 bits."""
    return (e.long() + 1023 << 52).view(torch.float64)
