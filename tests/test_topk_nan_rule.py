"""Router logits that are NaN: every selection ranks them below all numbers,
-inf included, lower expert index first among them.  The oracle and host models
of the router's two rules on the CPU; the kernels, and the few-token layer
beside the layer call, on the GPU."""
import math

import numpy as np
import pytest
import torch

import oracle

NAN, INF = math.nan, math.inf
ROWS = [
    # row, the four experts chosen
    ([NAN, 1, 2, 3, 4, 5, 6, 7], [7, 6, 5, 4]),
    ([0, 1, 2, 3, 4, 5, 6, NAN], [6, 5, 4, 3]),
    ([0, NAN, 2, NAN, 4, 5, 6, 7], [7, 6, 5, 4]),
    ([NAN] * 8, [0, 1, 2, 3]),
    ([NAN, -INF, NAN, -INF, NAN, 3, NAN, NAN], [5, 1, 3, 0]),
    ([-INF, NAN, -INF, NAN, NAN, NAN, NAN, NAN], [0, 2, 1, 3]),
    ([NAN, INF, NAN, -INF, INF, NAN, NAN, 0], [1, 4, 7, 3]),
    ([-INF] * 8, [0, 1, 2, 3]),
    ([-0.0, 0.0, NAN, 0.0, -0.0, -1, NAN, -2], [0, 1, 3, 4]),
]


def special_rows(T, E, seed):
    """Rows of coarse values with NaN and infinities strewn in, some all NaN."""
    rng = np.random.default_rng(seed)
    rows = (np.round(rng.normal(size=(T, E)) * 2) / 2).astype(np.float32)
    kind = rng.random((T, E))
    share = rng.choice([0.05, 0.5, 0.98], size=(T, 1))
    rows[kind < share * 0.6] = np.nan
    rows[(kind >= share * 0.6) & (kind < share * 0.9)] = -np.inf
    rows[(kind >= share * 0.9) & (kind < share)] = np.inf
    rows[0] = np.nan
    return rows


def test_oracle_ranks_nan_last():
    for row, want in ROWS:
        idx, _ = oracle.topk(np.array([row], np.float32), 4)
        assert idx[0].tolist() == want, row
    for E in (8, 33, 130):
        rows = special_rows(200, E, E)
        idx, _ = oracle.topk(rows, 8)
        for r, i in zip(rows, idx):
            order = sorted(range(E), key=lambda e: (np.isnan(r[e]), 0 if np.isnan(r[e]) else -r[e],
                                                    e))
            assert i.tolist() == order[:8]


def insertion_rule(row, k):
    """topk_insert, then topk_fill (router.cu)."""
    sv, se = [-INF] * 8, [-1] * 8
    for e, v in enumerate(row):
        if not v > sv[7]:
            continue
        shifting = False
        for i in range(8):
            if shifting or v > sv[i]:
                sv[i], v = v, sv[i]
                se[i], e = e, se[i]
                shifting = True
    kept = [e for e in se if e >= 0][:k]
    for nan in (False, True):
        for e, v in enumerate(row):
            if len(kept) < k and (np.isnan(v) if nan else v == -INF):
                kept.append(e)
    return kept


def logit_key(v):
    if np.isnan(v):
        return 1
    b = int(np.float32(0 if v == 0 else v).view(np.uint32))
    return (~b & 0xFFFFFFFF) if b >> 31 else b | 0x80000000


def key_rule(row, k):
    """k rounds of the largest key, lowest index first (router_topk_kernel and
    the few-token layer)."""
    key, out = [logit_key(v) for v in row], []
    for _ in range(k):
        out.append(key.index(max(key)))
        key[out[-1]] = 0
    return out


@pytest.mark.parametrize("E", [8, 9, 33, 64, 256])
def test_kernel_rules_match_the_oracle(E):
    rows = special_rows(150, E, E + 1)
    for k in (1, 3, 8):
        idx, _ = oracle.topk(rows, k)
        for r, i in zip(rows, idx):
            assert insertion_rule(r, k) == i.tolist()
            assert key_rule(r, k) == i.tolist()


# ------------------------------------------------------------------ kernels
def _bias(E, where, low=None):
    b = torch.linspace(-0.5, 0.5, E)
    if low is not None:
        b[low] = -INF
    b[where] = NAN
    return b.cuda()


# d = 64: K is not split and the GEMM's epilogue selects; 128 and 1024: the top-k
# kernel, one warp and one CTA a token
@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 1024])
@pytest.mark.parametrize("E", [4, 12, 64, 100, 256])
def test_route_with_nan_logits(d, E, cuda_ok):
    import mixture_experts_layer_36_b200 as moe
    T, k = 37, min(E, 4)
    g = torch.Generator().manual_seed(d + E)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16)
    x[5, 3] = NAN                                   # all logits of a token NaN
    x, wr = x.cuda(), (torch.randn(d, E, generator=g) * d ** -0.5).cuda()
    some = sorted({1, E // 2, E - 1})
    for where, low in (([0], None), ([E - 1], None), (some, None), (list(range(E)), None),
                       (list(range(1, E)), None), (list(range(2, E, 2)), list(range(1, E, 2))),
                       ([], list(range(E)))):
        logits, idx, w = moe.moe_route(x, wr, _bias(E, where, low), k)
        torch.cuda.synchronize()
        l32 = logits.cpu().numpy()
        assert np.isnan(l32[:, where]).all() and np.isnan(l32[5]).all()
        want, ww = oracle.topk(l32, k)
        assert np.array_equal(idx.cpu().numpy(), want)
        got = w.cpu().double().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(ww))
        assert np.abs(got - ww)[~np.isnan(ww)].max(initial=0) <= 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 64], ids=["bf16", "w4"])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("E", [5, 40, 200])
def test_both_layers_choose_alike(d, E, group, cuda_ok):
    """NaN logits of the first, the last and several experts: the few-token layer
    and moe_layer_forward_ex choose the same experts and places, and a token
    whose choice has no NaN agrees in y."""
    import mixture_experts_layer_36_b200 as moe
    T, k, f, cf = 7, 3, 64, 1.0
    g = torch.Generator().manual_seed(d * E)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = n(T, d).to(torch.bfloat16)
    x[2, 1] = NAN
    x, wr = x.cuda(), (n(d, E) * d ** -0.5).cuda()
    ws = [(n(E, a, b) * a ** -0.5).to(torch.bfloat16).cuda() for a, b in ((d, f), (d, f), (f, d))]
    if group:
        q = [moe.moe_quantize_weights_w4(w, group) for w in ws]
        ws = [moe.moe_dequantize_weights_w4(*t, group) for t in q]
    for where, low in (([0], None), ([E - 1], None), ([0, 1, E - 1], None),
                       (list(range(2, E)), None), (list(range(0, E, 2)), list(range(1, E, 2)))):
        bias = _bias(E, where, low)
        o, o2 = ({"topk_idx": torch.full((T, k), -7, dtype=torch.int32, device="cuda"),
                  "slot": torch.full((T, k), -7, dtype=torch.int32, device="cuda"),
                  "counts": torch.full((E,), -7, dtype=torch.int32, device="cuda")}
                 for _ in range(2))
        if group:
            y, _ = moe.moe_layer_forward_few_w4(x, wr, bias, *[t for p in q for t in p], k, cf,
                                                group, **o)
        else:
            y, _ = moe.moe_layer_forward_few(x, wr, bias, *ws, k, cf, **o)
        y2, _ = moe.moe_layer_forward_ex(x, wr, bias, *ws, k, cf, **o2)
        torch.cuda.synchronize()
        for name in o:
            assert torch.equal(o[name], o2[name]), (name, where)
        assert torch.equal(torch.isnan(y), torch.isnan(y2)), where
        ok = ~torch.isnan(y)
        if bool(ok.any()):
            # h and y rounded to bf16 (and the weights, on codes): 3 half steps of
            # values of the outputs' rms, 4 times over
            rms = float(y2[ok].double().square().mean().sqrt())
            assert float((y - y2)[ok].double().abs().max()) <= 4 * 4 * 2.0 ** -8 * rms
