"""64-bit reference of paged attention with sinks, trees of drafted tokens and an
8-bit cache, and the problems their tests draw.

Tolerances are those of tests/paged_ref.py.  Over an 8-bit cache a row of q may lose
2^-39 of its largest, and weights are rounded to fp16 as p 2^(e - E + 7) (E the
largest exponent so far, p at most 1 here), to 2^-25 absolutely where they are
small: 2^-32 2^E in the weight of a code up to 448, and 2^E is at most 2^-7 of the
largest value with the codes from 224 on that an exponent above the least has, so
2^-31 of the largest value in the result for each key (the least exponent: codes of
less, and weights of p 2^7)."""
import torch

from tests.paged_ref import DT, U

LEAST = {"bf16": -100, "fp16": -15}
MOST = 7


def encode(x, dtype):
    """Codes and exponents of rows of x (the last dimension), by the documented rule."""
    f = x.double()
    top = f.abs().amax(-1)
    e = torch.full(top.shape, LEAST[dtype], dtype=torch.int32)
    for n in range(LEAST[dtype], MOST):
        e += (top > 448.0 * 2.0 ** n).int()
    scaled = (f * torch.pow(torch.tensor(2.0, dtype=torch.float64), -e[..., None])).clamp(-448, 448)
    return scaled.float().to(torch.float8_e4m3fn), e.to(torch.int8)


def decode(codes, e):
    return codes.double() * torch.pow(torch.tensor(2.0, dtype=torch.float64), e[..., None].double())


def draw_tree(m, seed, span=4):
    """Parents of m tokens: each an earlier one (mostly a near one) or -1."""
    g = torch.Generator().manual_seed(seed)
    return [-1 if i == 0 else max(-1, i - 1 - int(torch.randint(0, span, (1,), generator=g))) for i in range(m)]


def tree_of(parents):
    """Who sees whom [m, m], and the depths."""
    m = len(parents)
    see, depth = torch.zeros(m, m, dtype=torch.bool), []
    for i, p in enumerate(parents):
        if p >= 0:
            see[i] = see[p]
        see[i, i] = True
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return see, depth


def pack(rows, words):
    """Bool rows as int32 words, bit c mod 32 of word c / 32."""
    out = torch.zeros(len(rows), words, dtype=torch.int64)
    for t, r in enumerate(rows):
        for c in r.nonzero()[:, 0].tolist():
            out[t, c // 32] |= 1 << (c % 32)
    return torch.where(out >= 2 ** 31, out - 2 ** 32, out).to(torch.int32)


def seen_of(geom, n, m, see=None, depth=None):
    """[m, n]: which keys of an n-token sequence its m chunk tokens see."""
    j = torch.arange(n)[None, :]
    p = torch.arange(m)[:, None] + (n - m)
    if see is not None:
        p = torch.tensor(depth).clamp(0, max(m - 1, 0))[:, None] + (n - m)
    seen = torch.ones(m, n, dtype=torch.bool)
    if geom.sparse_mode == 4:
        seen = (j <= p + geom.next_tokens) & ((j >= p - geom.pre_tokens) | (j < geom.sink_tokens))
    if see is not None:
        c = j - (n - m)
        bits = see[:, c[0].clamp(min=0)] if n else see[:, :0]
        seen = torch.where(c >= 0, bits, seen)
    return seen


def draw_cache(geom, kv_lens, seed, trees=None, spread=0):
    """Random sequences in shuffled pages.  Slots that a call may not need hold
    NaN (and a NaN's exponent), and their table entries are -1.  Rows differ by up
    to 2^spread in size, with rows of zeros among them."""
    g = torch.Generator().manual_seed(seed)
    P, q8 = geom.page_size, geom.cache_dtype == "e4m3"
    dt = torch.float8_e4m3fn if q8 else DT[geom.dtype]
    pages = [torch.full(geom.page_shape(), float("nan")).to(dt) for _ in range(2)]
    exps = [torch.full(geom.exponent_shape(), 127, dtype=torch.int8) for _ in range(2)] if q8 else [None, None]
    order = torch.randperm(geom.num_pages, generator=g).tolist()
    table = torch.full((geom.B, geom.max_pages), -1, dtype=torch.int32)
    dense = ([], [])
    for b, (n, m) in enumerate(zip(kv_lens, geom.q_lens())):
        need = torch.zeros(n, dtype=torch.bool)
        if m and n:
            need |= seen_of(geom, n, m).any(0)
            if trees is not None:
                need |= seen_of(geom, n, m, *trees[b]).any(0)
                need[max(0, n - m):] = True
        loud = 1.0 + 15.0 * (torch.rand(geom.D, generator=g) < 0.1)
        values = []
        for x in range(2):
            v = torch.randn(n, geom.n_kv, geom.D, generator=g) * (loud if x == 0 else 1.0)
            if spread:
                v *= torch.pow(2.0, -torch.randint(0, spread + 1, (n, geom.n_kv, 1), generator=g).float())
                v *= (torch.rand(n, geom.n_kv, 1, generator=g) > 0.1)
            if q8:
                codes, e = encode(v.to(DT[geom.dtype]) / (4.0 if x == 0 else 1.0), geom.dtype)
                values.append((codes, e))
                dense[x].append(decode(codes, e))
            else:
                v = (v / (4.0 if x == 0 else 1.0)).to(DT[geom.dtype])
                values.append((v, None))
                dense[x].append(v.double())
        for j in need.nonzero()[:, 0].tolist():
            if table[b, j // P] < 0:
                table[b, j // P] = order.pop()
            page, slot = int(table[b, j // P]), j % P
            at = (page, slice(None), slot) if geom.cache_layout == "BNSD" else (page, slot)
            for x in range(2):
                if q8:
                    pages[x].view(torch.uint8)[at] = values[x][0][j].view(torch.uint8)
                    exps[x][page, :, slot] = values[x][1][j]
                else:
                    pages[x][at] = values[x][0][j]
    return dense[0], dense[1], pages, exps, table, torch.tensor(kv_lens, dtype=torch.int32)


def attention_ref(geom, q, ks, vs, kv_lens, trees=None):
    """out, smax, ssum and their error bounds, in 64 bits (bounds as in tests/paged_ref.py)."""
    T, N, D = q.shape
    G, u = N // geom.n_kv, U[geom.dtype]
    out, eo = (torch.zeros(T, N, D, dtype=torch.float64) for _ in range(2))
    smax, ssum, em, es = (torch.zeros(T, N, dtype=torch.float64) for _ in range(4))
    smax -= float("inf")
    row = 0
    for b, (n, m) in enumerate(zip(kv_lens, geom.q_lens())):
        r = slice(row, row + m)
        row += m
        if n == 0 or m == 0:
            continue
        seen = seen_of(geom, n, m, *(trees[b] if trees is not None else ()))
        for h in range(N):
            x, k, v = q[r, h].double(), ks[b][:, h // G], vs[b][:, h // G]
            s = (x @ k.T) * geom.scale
            size = (x.abs() @ k.abs().T) * abs(geom.scale)
            size = torch.where(seen, size, torch.zeros((), dtype=torch.float64)).amax(1)
            s = torch.where(seen, s, torch.full((), -float("inf"), dtype=torch.float64))
            mx = s.amax(1)
            live = torch.isfinite(mx)
            w = torch.where(live[:, None], torch.exp(s - torch.where(live, mx, 0.0)[:, None]), 0.0)
            l = w.sum(1)
            P = w / torch.where(l > 0, l, 1.0)[:, None]
            out[r, h], smax[r, h], ssum[r, h] = P @ v, torch.where(live, mx, -float("inf")), l
            e = D * 2.0 ** -23 * size + 2.0 ** -22 * (size + 1)
            if geom.cache_dtype:
                e = e + abs(geom.scale) * x.abs().amax(1) * 2.0 ** -39 * k.abs().sum(1).amax()
            eo[r, h] = (P @ v.abs()) * (u + 2 * e + n * 2.0 ** -24)[:, None]
            if geom.dtype == "fp16":
                eo[r, h] += n * 2.0 ** -25 * v.abs().amax()
            if geom.cache_dtype:
                eo[r, h] += n * 2.0 ** -31 * v.abs().amax()
            eo[r, h] += u * (out[r, h].abs() + eo[r, h]) + (2.0 ** -25 if geom.dtype == "fp16" else 0.0)
            em[r, h] = e
            es[r, h] = l * (2 * e + n * 2.0 ** -24)
    return (out, smax, ssum), (eo, em, es)
