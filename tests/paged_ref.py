"""64-bit reference of the rotary and paged-cache operators, and the problems
their tests draw.  Plain loops over sequences and heads on the CPU; shares
nothing with the library but the geometry classes.

Tolerances (u = half a step of the element type, 2^-8 bf16, 2^-11 fp16):
- rotation: y = a cos t - b sin t.  The angle in half turns is rounded to fp32
  (error <= 2^-25, so pi 2^-25 radians), sine and cosine are within 2 ulp
  (2^-23), two products and a sum round by 2^-24 each: together below
  2^-21 (|a| + |b|); storing y adds u |y|.
- attention, one row with weights P_j (sum 1): scores are sums of D fp32
  products, off by at most e = D 2^-23 scale max_j sum_d |q_d k_jd| (+ 2^-22 of
  the largest score for the scale, exponent argument and exp2), which moves a
  weight by 2 e relative; each P is rounded to the element type (u); fp32
  sums over n keys add n 2^-24; storing the output adds u |out|.  In fp16 a
  weight below 2^-14 loses up to 2^-25 absolutely, n of them at most.
"""
import torch

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- rotation --
def rope_angles(geom, positions):
    """[rows, pairs] in 64 bits; positions int [axes, rows]."""
    R = geom.rotary_dim or geom.D
    freq = geom.inv_freq if geom.inv_freq is not None else [geom.base ** (-2.0 * i / R) for i in range(R // 2)]
    pos = positions.reshape(positions.shape[0], -1).double().cpu()
    return torch.stack([pos[a] * f for a, f in zip(geom.axes(), freq)], dim=1)


def rope_ref(geom, x, positions, inverse=False):
    """(y, bound) in 64 bits for x [B,n,S,D] or [T,n,D]."""
    R, half = geom.rotary_dim or geom.D, (geom.rotary_dim or geom.D) // 2
    t = rope_angles(geom, positions)
    if inverse:
        t = -t
    c, s = torch.cos(t), torch.sin(t)
    x = x.detach().cpu()
    if x.dim() == 4:
        c, s = (z.view(x.shape[0], 1, x.shape[2], half) for z in (c, s))
    else:
        c, s = c[:, None], s[:, None]
    f = x.double()
    if geom.interleaved:
        ia, ib = torch.arange(0, R, 2), torch.arange(1, R, 2)
    else:
        ia, ib = torch.arange(half), torch.arange(half, R)
    a, b = f[..., ia], f[..., ib]
    y, err = f.clone(), torch.zeros_like(f)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    err[..., ia] = err[..., ib] = (a.abs() + b.abs()) * 2.0 ** -21
    err[..., :R] += U[geom.dtype] * (y[..., :R].abs() + err[..., :R])
    if geom.dtype == "fp16":
        err[..., :R] += 2.0 ** -25  # subnormal results
    return y, err


# ------------------------------------------------------------------- cache --
def draw_cache(geom, kv_lens, seed, keys="all", poison=float("nan")):
    """Random sequences in shuffled pages.  Returns k, v (dense, per sequence,
    [kv_len, N_kv, D]), k_pages, v_pages, block_table, kv_lens (CPU).  Slots
    and pages without a token hold `poison`; so do tokens that no query of the
    chunk sees, and their table entries are -1, with keys="seen"."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[geom.dtype]
    P = geom.page_size
    k_pages = torch.full(geom.page_shape(), poison, dtype=dt)
    v_pages = torch.full(geom.page_shape(), poison, dtype=dt)
    order = torch.randperm(geom.num_pages, generator=g).tolist()
    table = torch.full((geom.B, geom.max_pages), -1, dtype=torch.int32)
    ks, vs = [], []
    for b, (n, m) in enumerate(zip(kv_lens, geom.q_lens())):
        k = torch.randn(n, geom.n_kv, geom.D, generator=g).to(dt)
        v = torch.randn(n, geom.n_kv, geom.D, generator=g).to(dt)
        ks.append(k)
        vs.append(v)
        lo, hi = seen_range(geom, n, m) if keys == "seen" else (0, n - 1)
        for j in range(max(lo, 0), hi + 1):
            if table[b, j // P] < 0:
                table[b, j // P] = order.pop()
            at = (int(table[b, j // P]), slice(None), j % P) if geom.cache_layout == "BNSD" else \
                (int(table[b, j // P]), j % P)
            k_pages[at], v_pages[at] = k[j], v[j]
    return ks, vs, k_pages, v_pages, table, torch.tensor(kv_lens, dtype=torch.int32)


def seen_range(geom, n, m):
    """First and last key that some of the m chunk tokens of an n-token sequence sees."""
    if n == 0 or m == 0:
        return 0, -1
    if geom.sparse_mode == 0:
        return 0, n - 1
    return max(0, n - m - geom.pre_tokens), min(n - 1, n - 1 + geom.next_tokens)


def attention_ref(geom, q, ks, vs, kv_lens):
    """out, smax, ssum and their error bounds, in 64 bits."""
    T, N, D = q.shape
    G, u = N // geom.n_kv, U[geom.dtype]
    out, eo = (torch.zeros(T, N, D, dtype=torch.float64) for _ in range(2))
    smax, ssum, em, es = (torch.zeros(T, N, dtype=torch.float64) for _ in range(4))
    smax -= float("inf")
    row = 0
    for b, (n, m) in enumerate(zip(kv_lens, geom.q_lens())):
        p = torch.arange(m)[:, None] + (n - m)
        j = torch.arange(n)[None, :]
        seen = torch.ones(m, n, dtype=torch.bool)
        if geom.sparse_mode == 4:
            seen = (j >= p - geom.pre_tokens) & (j <= p + geom.next_tokens)
        for h in range(N):
            x = q[row:row + m, h].double()
            if n == 0 or m == 0:
                continue
            k, v = ks[b][:, h // G].double(), vs[b][:, h // G].double()
            s = (x @ k.T) * geom.scale
            size = (x.abs() @ k.abs().T) * abs(geom.scale)
            size = torch.where(seen, size, torch.zeros(())).amax(1)
            s = torch.where(seen, s, torch.full((), -float("inf"), dtype=torch.float64))
            mx = s.amax(1)
            live = torch.isfinite(mx)
            w = torch.where(live[:, None], torch.exp(s - torch.where(live, mx, 0.0)[:, None]), 0.0)
            l = w.sum(1)
            P = w / torch.where(l > 0, l, 1.0)[:, None]
            r = slice(row, row + m)
            out[r, h], smax[r, h], ssum[r, h] = P @ v, torch.where(live, mx, -float("inf")), l
            e = D * 2.0 ** -23 * size + 2.0 ** -22 * (size + 1)
            mean = P @ v.abs()
            eo[r, h] = mean * (u + 2 * e + n * 2.0 ** -24)[:, None]
            if geom.dtype == "fp16":
                eo[r, h] += n * 2.0 ** -25 * v.abs().amax()
            eo[r, h] += u * (out[r, h].abs() + eo[r, h]) + (2.0 ** -25 if geom.dtype == "fp16" else 0.0)
            em[r, h] = e
            es[r, h] = l * (2 * e + n * 2.0 ** -24)
        row += m
    return (out, smax, ssum), (eo, em, es)


def assert_within(got, ref, bound, what):
    got, ref = got.detach().cpu().double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))  # infinities and NaN by place
    off = torch.where(same, torch.zeros((), dtype=torch.float64), (got - ref).abs() - bound)
    off = torch.where(torch.isnan(off), torch.full((), float("inf"), dtype=torch.float64), off)
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0.0, (what, "beyond its bound by", worst, "at", tuple(int(i) for i in (off == worst).nonzero()[0]))
