"""64-bit reference of dense attention under a window with sinks, forward and
backward, with the error that the library's roundings may leave in each result.

First order, per head, u = half a step of the products' 16-bit operands (2^-8
bf16 and fp32, 2^-11 fp16), w = half a step of the results' type:
- scores: a sum of D fp32 products, off by e = D 2^-23 scale max_j sum_d |q_d k_jd|
  + 2^-22 (largest score + 1) for the scale, the exponent's argument and exp2;
- a weight P is off by 2 e of itself, and by u once rounded for a product;
- fp32 sums of n terms add n 2^-24 of the sum of magnitudes;
- D_i = dy_i . out_i takes the stored out: its error, and D 2^-23 of the sum of magnitudes;
- dS = P (z dP - D) is off by P (error of dP and D) + 2 e |dS|, and by u once rounded;
- storing adds w of the value.
In fp16 a rounded P or dS below 2^-14 may lose up to 2^-25 absolutely, a stored
result as much."""
import torch

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -8}
W = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def visible(geom, n_q, n_kv):
    i, j = torch.arange(n_q)[:, None], torch.arange(n_kv)[None, :]
    if geom.sparse_mode != 4:
        return torch.ones(n_q, n_kv, dtype=torch.bool)
    return (j <= i + geom.next_tokens) & ((j >= i - geom.pre_tokens) | (j < geom.sink_tokens))


def head(geom, x, k, v, dy, seen, keep):
    """(results, bounds) of one head: out, smax, ssum, dq, dk, dv; keep: the dropout mask (0 / 1)."""
    u, w, D, scale = U[geom.dtype], W[geom.dtype], x.shape[1], geom.scale
    tiny = 2.0 ** -25 if geom.dtype == "fp16" else 0.0
    n, rows = seen.shape[1], seen.shape[0]
    z = keep / geom.keep_prob
    none = torch.zeros((), dtype=torch.float64)
    s = torch.where(seen, (x @ k.T) * scale, torch.full((), -float("inf"), dtype=torch.float64))
    size = torch.where(seen, (x.abs() @ k.abs().T) * abs(scale), none)
    size = size.amax(1) if n else torch.zeros(rows, dtype=torch.float64)
    mx = s.amax(1) if n else torch.full((rows,), -float("inf"), dtype=torch.float64)
    live = torch.isfinite(mx)
    p = torch.where(seen & live[:, None], torch.exp(s - torch.where(live, mx, none)[:, None]), none)
    l = p.sum(1)
    p = p / torch.where(l > 0, l, 1.0)[:, None]
    e = (D * 2.0 ** -23 * size + 2.0 ** -22 * (size + 1))[:, None]
    pz = p * z
    out = pz @ v
    eo = (pz @ v.abs()) * (u + 2 * e + n * 2.0 ** -24) + tiny * (z @ v.abs())
    eo = eo + w * (out.abs() + eo) + tiny
    dp = dy @ v.T
    d = (dy * out).sum(1, keepdim=True)
    ed = (dy.abs() * eo).sum(1, keepdim=True) + D * 2.0 ** -23 * (dy.abs() * out.abs()).sum(1, keepdim=True)
    edp = D * 2.0 ** -23 * (dy.abs() @ v.abs().T)
    ds = p * (z * dp - d)
    eds = p * (z * edp + ed) + (2 * e + 2.0 ** -22) * p * ((z * dp).abs() + d.abs())
    eds = torch.where(seen, eds + u * ds.abs() + tiny, none)
    epz = torch.where(seen, pz * (u + 2 * e + 2.0 ** -22) + tiny * z, none)
    ads = ds.abs()

    def stored(value, err):
        return err + w * (value.abs() + err) + tiny

    dq = (ds @ k) * scale
    dk = (ds.T @ x) * scale
    dv = pz.T @ dy
    edq = abs(scale) * ((eds + n * 2.0 ** -24 * ads) @ k.abs())
    edk = abs(scale) * ((eds + rows * 2.0 ** -24 * ads).T @ x.abs())
    edv = (epz + rows * 2.0 ** -24 * pz).T @ dy.abs()
    smax = torch.where(live, mx, torch.full((), -float("inf"), dtype=torch.float64))
    return (out, smax, l, dq, dk, dv), (eo, e[:, 0], l * (2 * e[:, 0] + n * 2.0 ** -24), stored(dq, edq), edk, edv)


def reference(geom, q, k, v, dy, keep_bits=None):
    """out, smax, ssum, dq, dk, dv and their bounds, in the geometry's layout.  keep_bits: the packed dropout mask."""
    bnsd = geom.layout == "BNSD"
    w = W[geom.dtype]
    tiny = 2.0 ** -25 if geom.dtype == "fp16" else 0.0
    f64 = lambda shape: torch.zeros(shape, dtype=torch.float64)
    res = [f64(geom.q_shape()), f64(geom.stat_shape()) - float("inf"), f64(geom.stat_shape()), f64(geom.q_shape()),
           f64(geom.kv_shape()), f64(geom.kv_shape())]
    err = [torch.zeros_like(t) for t in res]
    err[1].zero_()
    bits = None
    if keep_bits is not None:
        by = keep_bits.cpu()
        bits = ((by[:, None] >> torch.arange(8, dtype=torch.uint8)) & 1).reshape(-1).double()
    G = geom.N // geom.n_kv
    at_q = at_k = base = 0
    for b, (n_q, n_kv) in enumerate(geom.seq_lens()):
        seen = visible(geom, n_q, n_kv)
        for h in range(geom.N):
            qs = (b, h) if bnsd else (slice(at_q, at_q + n_q), h)
            ks = (b, h // G) if bnsd else (slice(at_k, at_k + n_kv), h // G)
            keep = torch.ones(n_q, n_kv, dtype=torch.float64)
            if bits is not None:
                keep = bits[base:base + n_q * n_kv].view(n_q, n_kv)
            base += n_q * n_kv
            r, e = head(geom, q[qs].double(), k[ks].double(), v[ks].double(), dy[qs].double(), seen, keep)
            for x in range(4):
                res[x][qs], err[x][qs] = r[x], e[x]
            for x in (4, 5):
                res[x][ks] += r[x]
                err[x][ks] += e[x]
        at_q += n_q
        at_k += n_kv
    for x in (4, 5):
        err[x] += w * (res[x].abs() + err[x]) + tiny
    return res, err
