"""The few-token layer and the 4-bit weight format in 64 bits, from their
definitions, with error bounds for the kernels' arithmetic.

Bounds.  u = 2^-24 is half a step of fp32, 2^-8 half a step of bf16 (relative).
  * logits: accumulated in fp64, rounded once: u |l| (+ 2^-50 of the sum of
    magnitudes for the fp64 sums of both sides, d <= 2^13 terms).
  * gate weights, from the returned fp32 logits: the difference l_j - l_0 is
    rounded (u D as an absolute error of the exponent, D the largest
    difference), expf is within 2 steps (4 u), twice (numerator and sum), the
    sum of k <= 8 terms adds 7 u, the quotient u: relative (2 D + 20) u.
  * a product of n terms accumulated in fp32: n u sum |a b|.
  * h = silu(g) u: |silu'| <= 1.1, silu within 8 steps (exp, add, divide,
    product: 16 u), the product u; errors of g and u carried through.  On bf16
    weights h enters the next product as two bf16 terms, which leaves 2^-16 |h|.
  * On 4-bit codes x and h enter their products as fixed-point digits, in units of
    at most 2^-21 of the largest of each 128 values: half a unit is 2^-22 of it.
  * y: the errors above carried through the down projection and the weighted
    sum of k terms (8 more roundings), then one rounding to bf16 (2^-8).
"""
import numpy as np
import torch

U32 = 2.0 ** -24
U16 = 2.0 ** -8


def capacity(T, E, k, cf):
    return T if cf == 0 else int(np.ceil(((cf * k) * T) / E))


def order_key(v):
    """Selection order of fp32 values: descending, NaN last."""
    return (1, 0.0) if np.isnan(v) else (0, -float(v))


def route(logits32, k):
    """Top-k rows of fp32 logits (numpy), ties to the lower index."""
    T, E = logits32.shape
    idx = np.zeros((T, k), np.int32)
    for t in range(T):
        idx[t] = sorted(range(E), key=lambda e: (*order_key(logits32[t, e]), e))[:k]
    return idx


def slots(idx, E, C):
    T, k = idx.shape
    slot = np.full((T, k), -1, np.int32)
    n = np.zeros(E, np.int64)
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if n[e] < C:
                slot[t, j] = n[e]
            n[e] += 1
    return slot, np.minimum(n, C).astype(np.int32)


def logits64(x, w_router, bias):
    out = x.double().cpu() @ w_router.double().cpu()
    return out if bias is None else out + bias.double().cpu()


def weights64(l32, idx):
    """Softmax over the selected fp32 logits, and its error bound."""
    sel = np.take_along_axis(l32.astype(np.float64), idx.astype(np.int64), 1)
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.exp(sel - sel[:, :1])
        w = p / p.sum(1, keepdims=True)
        D = np.where(np.isfinite(sel), np.abs(sel - sel[:, :1]), 0).max(1, keepdims=True)
    return w, (2 * D + 20) * U32 * w


def largest_of_128(v):
    """Each value's largest magnitude among its 128 (the last ones fewer)."""
    out = torch.empty_like(v)
    for i in range(0, v.shape[1], 128):
        out[:, i:i + 128] = v[:, i:i + 128].abs().amax(1, keepdim=True)
    return out


def layer64(x, experts, idx, slot, w, digits=False):
    """(y, bound) in fp64.  experts: function e -> (Wg, Wu, Wd) fp64 on some
    device; idx, slot, w numpy; rows whose pairs are all dropped return x
    itself with bound 0.  digits: on 4-bit codes."""
    T, d = x.shape
    k = idx.shape[1]
    X = x.double()
    y = torch.zeros(T, d, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)          # sum of |terms| for the weighted sum's roundings
    err = torch.zeros_like(y)
    served = torch.zeros(T, dtype=torch.bool, device=x.device)
    for e in sorted(set(idx[slot >= 0].tolist())):
        pairs = [(t, j) for t in range(T) for j in range(k) if idx[t, j] == e and slot[t, j] >= 0]
        Wg, Wu, Wd = experts(e)
        r = X[[t for t, _ in pairs]]
        g, u = r @ Wg, r @ Wu
        dx = 2.0 ** -22 * largest_of_128(r) if digits else torch.zeros_like(r)
        dg, du = (d * U32 * ((r.abs() + dx) @ W.abs()) + dx @ W.abs() for W in (Wg, Wu))
        f = g.shape[1]
        s = g * torch.sigmoid(g)
        h = s * u
        dh = 1.1 * dg * (u.abs() + du) + s.abs() * du + 17 * U32 * h.abs()
        dh = dh + (2.0 ** -22 * largest_of_128(h.abs() + dh) if digits else 2.0 ** -16 * h.abs())
        o = h @ Wd
        do = dh @ Wd.abs() + f * U32 * ((h.abs() + dh) @ Wd.abs())
        for i, (t, j) in enumerate(pairs):
            wt = float(w[t, j])
            y[t] += wt * o[i]
            mag[t] += abs(wt) * (o[i].abs() + do[i])
            err[t] += abs(wt) * do[i]
            served[t] = True
    err = err + 60 * U32 * mag         # gate weights ((2 D + 20) u, D <= 16) and 8 roundings
    bound = err + U16 * (y.abs() + err)
    y = torch.where(served[:, None], y, X)
    return y, torch.where(served[:, None], bound, torch.zeros_like(bound))


# ------------------------------------------------------------- 4-bit format
def quantize64(w, group):
    """bf16 [E,K,N] (CPU) -> (values u - 8 as int [E,K,N], scales float64
    [E,groups,N], exact bf16 values)."""
    E, K, N = w.shape
    codes = torch.zeros(E, K, N, dtype=torch.int64)
    scales = []
    for k0 in range(0, K, group):
        v = w[:, k0:k0 + group].double()
        mx = v.abs().amax(1, keepdim=True)              # NaN propagates
        s = (mx / 7).to(torch.bfloat16).double()
        s = torch.where(s == 0, torch.ones_like(s), s)
        c = torch.round(v / s)                          # half to even
        c = torch.where(torch.isfinite(s).expand_as(c), c, torch.zeros_like(c))
        codes[:, k0:k0 + group] = c.clamp(-7, 7).to(torch.int64)
        scales.append(s)
    return codes, torch.cat(scales, 1)


def place(k, n, K):
    """(byte, shift) of the code of row k, column n in one packed matrix."""
    tile = (n // 64) * (K // 64) + k // 64
    block, lane = (n % 64) // 16, 4 * (n % 8) + (k % 8) // 2
    word = (k % 64) // 16
    nibble = (n % 16) // 8 + 2 * ((k % 16) // 8) + 4 * (k % 2)
    return tile * 2048 + block * 512 + lane * 16 + word * 4 + nibble // 2, 4 * (nibble % 2)


def pack(codes):
    """int values u - 8 [E,K,N] -> uint8 [E, N/64, K/64, 2048], by place()."""
    E, K, N = codes.shape
    kk, nn = np.meshgrid(np.arange(K), np.arange(N), indexing="ij")
    byte, shift = place(kk, nn, K)
    out = np.zeros((E, K * N // 2), np.uint8)
    u = (codes.numpy() + 8).astype(np.uint8)
    for half in (0, 4):
        m = shift == half
        out[:, byte[m]] |= (u[:, m] << half).astype(np.uint8)
    return torch.from_numpy(out).view(E, N // 64, K // 64, 2048)


def unpack(q):
    """uint8 [E, N/64, K/64, 2048] -> int values u - 8 [E,K,N], by place()."""
    E, N, K = q.shape[0], q.shape[1] * 64, q.shape[2] * 64
    kk, nn = np.meshgrid(np.arange(K), np.arange(N), indexing="ij")
    byte, shift = place(kk, nn, K)
    flat = q.cpu().numpy().reshape(E, -1)
    return torch.from_numpy(((flat[:, byte] >> shift) & 15).astype(np.int64) - 8)


def values64(codes, scales, group):
    """(u - 8) * s in fp64 [E,K,N]."""
    K = codes.shape[1]
    return codes.double() * scales.double().repeat_interleave(group, 1)[:, :K]
