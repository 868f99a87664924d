"""The few-token layer (bf16 and 4-bit experts) and the 4-bit conversions on a
GPU, against 64-bit definitions with derived bounds (few_reference.py)."""
import math

import numpy as np
import pytest
import torch

import few_reference as ref
import mixture_experts_layer_36_b200 as moe

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(autouse=True)
def _cuda(cuda_ok):
    torch.cuda.set_device(0)


def make(T, d, E, k, f, seed, group=0, bias=False):
    """Inputs on the GPU; group > 0: 4-bit experts quantized from the bf16 ones."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = {"x": n(T, d).to(BF).cuda(), "w_router": (n(d, E) * d ** -0.5).cuda(),
         "bias": (n(E) * 0.5).cuda() if bias else None}
    p["w"] = [(n(E, K, N) * K ** -0.5).to(BF).cuda() for K, N in ((d, f), (d, f), (f, d))]
    p["group"] = group
    if group:
        p["q"] = [moe.moe_quantize_weights_w4(w, group) for w in p["w"]]
    return p


def call(p, k, cf, **kw):
    if p["group"]:
        flat = [t for qs in p["q"] for t in qs]
        return moe.moe_layer_forward_few_w4(p["x"], p["w_router"], p["bias"], *flat, k, cf,
                                            p["group"], **kw)
    return moe.moe_layer_forward_few(p["x"], p["w_router"], p["bias"], *p["w"], k, cf, **kw)


def outputs(T, E, k):
    z = lambda *s, dt: torch.full(s, -7, dtype=dt, device="cuda")  # noqa: E731
    return {"logits": z(T, E, dt=F32), "topk_idx": z(T, k, dt=I32), "topk_w": z(T, k, dt=F32),
            "slot": z(T, k, dt=I32), "counts": z(E, dt=I32)}


def experts64(p):
    def get(e):
        if not p["group"]:
            return [w[e].double() for w in p["w"]]
        return [ref.values64(ref.unpack(q[e:e + 1]), s[e:e + 1].cpu(), p["group"])[0].cuda()
                for q, s in p["q"]]
    return get


def check(p, k, cf, y, o, status):
    """Everything the call returned against the definitions."""
    x = p["x"]
    T, E = x.shape[0], p["w_router"].shape[1]
    assert status == 0
    l64 = ref.logits64(x, p["w_router"], p["bias"])
    mag = ref.logits64(x.abs(), p["w_router"].abs(), None if p["bias"] is None else
                       p["bias"].abs())
    got = o["logits"].cpu().double()
    fin = torch.isfinite(l64)
    assert torch.equal(torch.isnan(l64), torch.isnan(got))
    assert bool(((got - l64).abs() <= ref.U32 * l64.abs() + 2.0 ** -40 * mag)[fin].all())
    l32 = o["logits"].cpu().numpy()
    idx = o["topk_idx"].cpu().numpy()
    assert np.array_equal(idx, ref.route(l32, k))
    w, dw = ref.weights64(l32, idx)
    gw = o["topk_w"].cpu().double().numpy()
    ok = np.isfinite(w)
    assert np.array_equal(np.isnan(w), np.isnan(gw))
    assert (np.abs(gw - w) <= dw + 2.0 ** -126)[ok].all()
    slot, counts = ref.slots(idx, E, ref.capacity(T, E, k, cf))
    assert np.array_equal(o["slot"].cpu().numpy(), slot)
    assert np.array_equal(o["counts"].cpu().numpy(), counts)
    y64, bound = ref.layer64(x, experts64(p), idx, slot, w, digits=bool(p["group"]))
    err = (y.double() - y64).abs()
    fine = torch.isfinite(y64)
    assert torch.equal(fine, torch.isfinite(y))
    worst = (err / bound.clamp_min(1e-300))[fine & (bound > 0)]
    assert bool((err <= bound)[fine].all()), f"worst {float(worst.max()):.2f} of the bound"


CASES = [
    # T, d, E, k, f, cf, bias
    (1, 64, 1, 1, 64, 0.0, False),
    (1, 128, 8, 2, 256, 0.0, False),
    (1, 1024, 256, 8, 192, 0.0, True),
    (2, 320, 5, 5, 64, 0.0, False),
    (3, 192, 61, 5, 704, 1.0, True),
    (4, 448, 64, 6, 320, 1.0, False),
    (5, 64, 3, 2, 1408, 0.0, False),
    (7, 256, 2, 1, 128, 0.5, False),
    (8, 512, 8, 2, 448, 0.0, False),
    (9, 192, 8, 2, 192, 1.25, True),
    (16, 128, 130, 8, 128, 0.0, False),
    (17, 320, 4, 3, 320, 1.0, False),
    (31, 64, 33, 7, 192, 1.0, True),
    (32, 256, 256, 8, 64, 0.0, False),
    (32, 192, 1, 1, 320, 0.0, False),
    (32, 128, 2, 2, 128, 0.0, False),
]


@pytest.mark.parametrize("group", [0, 32, 64, 128], ids=["bf16", "g32", "g64", "g128"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d-d%d-E%d-k%d-f%d-cf%g" % c[:6])
def test_layer_against_definition(case, group):
    T, d, E, k, f, cf, bias = case
    p = make(T, d, E, k, f, seed=T * 1000 + d + E, group=group, bias=bias)
    o = outputs(T, E, k)
    y, ws = call(p, k, cf, **o)
    torch.cuda.synchronize()
    check(p, k, cf, y, o, int(ws[:4].view(I32).item()))


@pytest.mark.parametrize("group", [0, 64], ids=["bf16", "w4"])
def test_skewed_routing_fills_one_expert(group):
    """Every token on the same experts: 32 rows of one expert, others empty."""
    T, d, E, k, f = 32, 128, 16, 2, 192
    p = make(T, d, E, k, f, seed=5, group=group)
    p["bias"] = torch.zeros(E, device="cuda")
    p["bias"][3], p["bias"][11] = 100.0, 90.0
    for cf in (0.0, 1.0):
        o = outputs(T, E, k)
        y, ws = call(p, k, cf, **o)
        torch.cuda.synchronize()
        check(p, k, cf, y, o, int(ws[:4].view(I32).item()))
        assert o["counts"][3].item() == (T if cf == 0 else 4)
        if cf:
            assert torch.equal(y[4:], p["x"][4:])      # all pairs dropped: the token itself


@pytest.mark.parametrize("group", [0, 128], ids=["bf16", "w4"])
def test_ties_and_masked_experts(group):
    """Equal router columns rank by index; experts masked by a bias of -inf or
    of the lowest finite value are chosen last, with weight 0."""
    T, d, E, k, f = 6, 64, 12, 4, 64
    p = make(T, d, E, k, f, seed=6, group=group)
    p["w_router"][:, 7] = p["w_router"][:, 2]
    p["w_router"][:, 9] = p["w_router"][:, 2]
    p["x"][1] = 0                                       # all logits equal: 0, 1, 2, 3
    for low in (-math.inf, torch.finfo(F32).min):
        p["bias"] = torch.zeros(E, device="cuda")
        p["bias"][[0, 1, 3, 4, 5, 6, 8, 10, 11]] = low
        o = outputs(T, E, k)
        y, ws = call(p, k, 0.0, **o)
        torch.cuda.synchronize()
        assert o["topk_idx"][:, :3].tolist() == [[2, 7, 9]] * T
        assert o["topk_w"][:, 3].tolist() == [0.0] * T
        check(p, k, 0.0, y, o, int(ws[:4].view(I32).item()))
    p["bias"] = None
    o = outputs(T, E, k)
    y, ws = call(p, k, 0.0, **o)
    torch.cuda.synchronize()
    assert o["topk_idx"][1].tolist() == [0, 1, 2, 3]
    check(p, k, 0.0, y, o, int(ws[:4].view(I32).item()))


@pytest.mark.parametrize("group", [0, 32], ids=["bf16", "w4"])
def test_logits_that_are_no_numbers(group):
    """An expert whose logit is NaN is not chosen while k others are numbers (as
    in moe_layer_forward); all experts masked: the first k, with NaN weights."""
    T, d, E, k, f = 5, 128, 12, 3, 64
    p = make(T, d, E, k, f, seed=12, group=group)
    p["bias"] = torch.zeros(E, device="cuda")
    p["bias"][7] = math.nan
    o, o2 = outputs(T, E, k), outputs(T, E, k)
    y, ws = call(p, k, 0.0, **o)
    moe.moe_layer_forward_ex(p["x"], p["w_router"], p["bias"], *p["w"], k, 0.0, **o2)
    torch.cuda.synchronize()
    assert torch.equal(o["topk_idx"], o2["topk_idx"]) and bool((o["topk_idx"] != 7).all())
    check(p, k, 0.0, y, o, int(ws[:4].view(I32).item()))
    p["bias"] = torch.full((E,), -math.inf, device="cuda")
    o = outputs(T, E, k)
    y, ws = call(p, k, 0.0, **o)
    torch.cuda.synchronize()
    assert o["topk_idx"].tolist() == [[0, 1, 2]] * T
    assert bool(torch.isnan(o["topk_w"]).all()) and bool(torch.isnan(y).all())
    assert int(ws[:4].view(I32).item()) == 0


@pytest.mark.parametrize("group", [0, 32], ids=["bf16", "w4"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_bad_token_stays_alone(group, bad):
    """A NaN or an infinity in one token leaves every other token's bits."""
    T, d, E, k, f = 11, 128, 8, 2, 128
    p = make(T, d, E, k, f, seed=7, group=group)
    y0, _ = call(p, k, 0.0)
    p["x"][4, 37] = bad
    o = outputs(T, E, k)
    y1, ws = call(p, k, 0.0, **o)
    torch.cuda.synchronize()
    keep = [t for t in range(T) if t != 4]
    assert torch.equal(y0[keep], y1[keep])
    assert not torch.isfinite(y1[4]).any()
    idx = o["topk_idx"][4].tolist()
    assert len(set(idx)) == k and all(0 <= e < E for e in idx)
    assert int(ws[:4].view(I32).item()) == 0


@pytest.mark.parametrize("group", [0, 64], ids=["bf16", "w4"])
def test_bad_weights_of_an_unused_expert_are_not_read(group):
    """Poisoned weights of experts that no token chose change nothing, and a
    poisoned column of a used one stays in its column."""
    T, d, E, k, f = 3, 64, 8, 1, 128
    p = make(T, d, E, k, f, seed=8, group=group)
    p["bias"] = torch.zeros(E, device="cuda")
    p["bias"][5] = 50.0
    y0, _ = call(p, k, 0.0)
    for i in range(3):
        for e in range(E):
            if e != 5:
                (p["q"][i][1] if group else p["w"][i])[e] = math.nan
    (p["q"][2][1] if group else p["w"][2])[5, 0, 17] = math.nan
    y1, _ = call(p, k, 0.0)
    torch.cuda.synchronize()
    cols = [c for c in range(d) if c != 17]
    assert torch.equal(y0[:, cols], y1[:, cols])
    assert torch.isnan(y1[:, 17]).all()


@pytest.mark.parametrize("group", [0, 128], ids=["bf16", "w4"])
def test_buffers_of_the_caller(group):
    """A workspace full of garbage, of exactly the size asked for; what lies
    behind it and behind y stays; results are the same bits call after call."""
    T, d, E, k, f = 5, 192, 9, 3, 320
    p = make(T, d, E, k, f, seed=9, group=group)
    need = moe.moe_workspace_size_few(T, d, E, k, f)
    buf = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    ybuf = torch.full((T + 3, d), 3.0, dtype=BF, device="cuda")
    ref_y, _ = call(p, k, 0.0)
    for fill in (0xA5, 0xFF, 0x00, None):
        if fill is not None:
            buf[:need] = fill
        y, ws = call(p, k, 0.0, y=ybuf[:T], ws=buf[:need])
        torch.cuda.synchronize()
        assert y.data_ptr() == ybuf.data_ptr() and ws.data_ptr() == buf.data_ptr()
        assert torch.equal(y, ref_y)
        assert bool((buf[need:] == 0xA5).all()) and bool((ybuf[T:] == 3.0).all())


@pytest.mark.parametrize("group", [0, 64], ids=["bf16", "w4"])
def test_streams_and_graphs(group):
    """On a side stream; captured and replayed on new tokens; two graphs on one
    workspace replayed in turn; two streams at once on two workspaces."""
    T, d, E, k, f = 4, 256, 32, 4, 192
    p = make(T, d, E, k, f, seed=10, group=group)
    xs = [torch.randn(T, d, device="cuda").to(BF) for _ in range(4)]
    want = []
    for x in xs:
        p["x"].copy_(x)
        want.append(call(p, k, 0.0)[0].clone())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    p["x"].copy_(xs[0])
    side.wait_stream(torch.cuda.current_stream())
    y, ws = call(p, k, 0.0, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0])

    graphs, ys = [], []
    for _ in range(2):                                   # two graphs, one workspace
        g = torch.cuda.CUDAGraph()
        yb = torch.empty_like(p["x"])
        with torch.cuda.graph(g):
            call(p, k, 0.0, y=yb, ws=ws)
        graphs.append(g)
        ys.append(yb)
    for i, x in enumerate(xs):
        p["x"].copy_(x)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[i % 2], want[i])

    q = [dict(p, x=x.clone()) for x in xs[:2]]
    streams = [torch.cuda.Stream() for _ in q]
    wss = [torch.empty_like(ws) for _ in q]
    outs = [torch.empty_like(p["x"]) for _ in q]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, s, b, o in zip(q, streams, wss, outs):
            call(a, k, 0.0, y=o, ws=b, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@pytest.mark.parametrize("group", [0, 64], ids=["bf16", "w4"])
@pytest.mark.parametrize("T, cf", [(1, 0.0), (7, 0.5), (32, 0.5)])
def test_in_place(T, cf, group):
    """y = x, with dropped tokens that pass through: the bits of a call out of place."""
    p = make(T, 320, 4, 2, 192, seed=T, group=group)
    want = call(p, 2, cf)[0].clone()
    y, _ = call(p, 2, cf, y=p["x"])
    assert y.data_ptr() == p["x"].data_ptr() and torch.equal(y, want)


def test_agrees_with_the_layer_call():
    """The few-token layer and moe_layer_forward on the same inputs: same
    routing results, outputs within both calls' roundings of h and y to bf16."""
    T, d, E, k, f = 24, 512, 16, 4, 256
    for cf in (0.0, 1.0):
        p = make(T, d, E, k, f, seed=11)
        o = outputs(T, E, k)
        y, _ = call(p, k, cf, **o)
        o2 = outputs(T, E, k)
        y2, _ = moe.moe_layer_forward_ex(p["x"], p["w_router"], None, *p["w"], k, cf, **o2)
        torch.cuda.synchronize()
        for n in ("topk_idx", "slot", "counts"):
            assert torch.equal(o[n], o2[n]), n
        # y: half a step each; h: half a step of bf16 on each of f terms
        _, bound = ref.layer64(p["x"], experts64(p), o["topk_idx"].cpu().numpy(),
                               o["slot"].cpu().numpy(), o["topk_w"].cpu().double().numpy())
        terms = torch.zeros(T, d, dtype=torch.float64, device="cuda")
        for t in range(T):
            for j in range(k):
                if o["slot"][t, j] >= 0:
                    e = int(o["topk_idx"][t, j])
                    Wg, Wu, Wd = experts64(p)(e)
                    r = p["x"][t].double()
                    g = r @ Wg
                    terms[t] += float(o["topk_w"][t, j]) * (
                        (g * torch.sigmoid(g) * (r @ Wu)).abs() @ Wd.abs())
        assert bool(((y.double() - y2.double()).abs() <=
                     2 * bound + 1.01 * ref.U16 * terms).all())


# ------------------------------------------------------------------ conversions
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 64, 64), (3, 320, 192), (2, 192, 1408), (5, 704, 64)])
def test_quantize_and_back(shape, group):
    E, K, N = shape
    g = torch.Generator().manual_seed(K + N)
    w = (torch.randn(E, K, N, generator=g) * torch.rand(E, 1, N, generator=g) * 3).to(BF)
    w[0, :, 1] = 0                                       # zero groups
    w[0, 0, 2], w[0, K - 1, 3], w[0, 5, 4] = math.nan, math.inf, -math.inf
    w[-1, :, 5] = torch.arange(K).remainder(29).sub(14).div(2).to(BF)      # ties
    w[-1, :, 6] = 2.0 ** -133                            # smallest bf16: the scale rounds to 0
    q, s = moe.moe_quantize_weights_w4(w.cuda(), group)
    codes, scales = ref.quantize64(w, group)
    torch.cuda.synchronize()
    got = s.cpu().double()
    fin = torch.isfinite(scales)
    assert torch.equal(fin, torch.isfinite(got)) and torch.equal(got[fin], scales[fin])
    assert torch.equal(q.cpu(), ref.pack(codes))
    back = moe.moe_dequantize_weights_w4(q, s, group).cpu()
    want = ref.values64(codes, scales, group).to(BF)
    nan = torch.isnan(want)
    assert torch.equal(nan, torch.isnan(back)) and torch.equal(back[~nan], want[~nan])
    # half a step of the code on every finite group
    step = scales.repeat_interleave(group, 1)[:, :K]
    ok = torch.isfinite(step) & (step < 1e30)
    off = (back.double() - w.double()).abs()
    assert bool((off <= 0.52 * step + ref.U16 * w.double().abs())[ok].all())


def test_dequantize_takes_any_code():
    q = torch.randint(0, 256, (2, 3, 5, 2048), dtype=torch.uint8, device="cuda")
    s = torch.randn(2, 5, 192, device="cuda").to(BF)     # K = 320, group 64
    back = moe.moe_dequantize_weights_w4(q, s, 64)
    want = ref.values64(ref.unpack(q), s.cpu(), 64).to(BF)
    assert torch.equal(back.cpu(), want)


def test_conversions_leave_their_surroundings_and_run_in_graphs():
    E, K, N, group = 2, 192, 128, 128
    w = torch.randn(E, K, N, device="cuda").to(BF)
    q0, s0 = moe.moe_quantize_weights_w4(w, group)
    b0 = moe.moe_dequantize_weights_w4(q0, s0, group)
    qb = torch.full((E + 1, 2, 3, 2048), 0x5A, dtype=torch.uint8, device="cuda")
    sb = torch.full((E + 1, 2, N), 2.5, dtype=BF, device="cuda")
    bb = torch.full((E + 1, K, N), 2.5, dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        moe.moe_quantize_weights_w4(w, group, q=qb[:E], scale=sb[:E])
        moe.moe_dequantize_weights_w4(qb[:E], sb[:E], group, w=bb[:E])
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qb[:E], q0) and torch.equal(sb[:E], s0) and torch.equal(bb[:E], b0)
    assert bool((qb[E] == 0x5A).all()) and bool((sb[E] == 2.5).all()) and bool((bb[E] == 2.5).all())


def test_quantize_decode_prefill_together():
    """As a server uses them: the experts of a bf16 layer are quantized once,
    decode steps run on the codes (one graph, one workspace), a long prompt on
    the dequantized weights; token by token both agree."""
    T, d, E, k, f, group = 8, 256, 16, 2, 192, 64
    p = make(T, d, E, k, f, seed=12, group=group)
    back = [moe.moe_dequantize_weights_w4(q, s, group) for q, s in p["q"]]
    prompt = torch.randn(200, d, device="cuda").to(BF)
    y_long, _ = moe.moe_layer_forward(prompt, p["w_router"], None, *back, k, 0.0)
    ws = torch.empty(moe.moe_workspace_size_few(T, d, E, k, f), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(p["x"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(p, k, 0.0, y=y, ws=ws)
    for i in range(0, 200, T):
        p["x"].copy_(prompt[i:i + T])
        graph.replay()
        ref_rows = y_long[i:i + T].double()
        # the bf16 weights differ from code * scale by half a step (2^-8), in
        # three products; h and y are rounded to bf16: about 5 half steps of
        # values of the size of the row's rms, taken 4 times over
        rms = ref_rows.square().mean().sqrt()
        assert float((y.double() - ref_rows).abs().max()) <= 4 * 5 * ref.U16 * float(rms)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_over_the_whole_range(group):
    """Codes and scales equal the 64-bit rule for magnitudes from the smallest
    bf16 to the largest: the path without divisions, and the one with."""
    E, K, N = 2, 448, 128
    g = torch.Generator().manual_seed(group)
    base = torch.randint(-133, 128, (E, -(-K // group), N), generator=g)
    fall = torch.randint(0, 5, (E, K, N), generator=g)
    mant = 1 + torch.randint(0, 128, (E, K, N), generator=g).double() / 128
    sign = torch.randint(0, 2, (E, K, N), generator=g).double() * 2 - 1
    exp = base.repeat_interleave(group, 1)[:, :K].double() - fall.double()
    w = (sign * mant * torch.exp2(exp)).clamp(-3.38e38, 3.38e38).to(BF)
    w[0] = torch.randn(K, N, generator=g).to(BF)          # plain tiles as well
    q, s = moe.moe_quantize_weights_w4(w.cuda(), group)
    codes, scales = ref.quantize64(w, group)
    torch.cuda.synchronize()
    assert torch.equal(s.cpu().double(), scales)
    assert torch.equal(q.cpu(), ref.pack(codes))
    back = moe.moe_dequantize_weights_w4(q, s, group).cpu()
    assert torch.equal(back, ref.values64(codes, scales, group).to(BF))


# ------------------------------------------------------------------ larger, and refusals
@pytest.mark.parametrize("group", [0, 32, 128], ids=["bf16", "g32", "g128"])
@pytest.mark.parametrize("case", [(2, 7168, 4, 2, 2048, 0.0, False),
                                  (9, 1024, 40, 8, 1408, 1.25, True),
                                  (32, 2048, 6, 2, 1408, 0.0, False)],
                         ids=lambda c: "T%d-d%d-E%d-k%d-f%d" % c[:5])
def test_layer_at_full_widths(case, group):
    """Units cut in several chunks, many column tiles, experts of several units."""
    T, d, E, k, f, cf, bias = case
    p = make(T, d, E, k, f, seed=T + d, group=group, bias=bias)
    o = outputs(T, E, k)
    y, ws = call(p, k, cf, **o)
    torch.cuda.synchronize()
    check(p, k, cf, y, o, int(ws[:4].view(I32).item()))


@pytest.mark.parametrize("group", [0, 64], ids=["bf16", "w4"])
@pytest.mark.parametrize("T, d, E", [(1, 12352, 8), (3, 15040, 7), (12, 12352, 6), (32, 15040, 8),
                                     (2, 7168, 250), (9, 7168, 256), (32, 7168, 254)])
def test_router_rows_of_two_passes(T, d, E, group):
    """Wide layers, whose router rows a CTA stages in two passes of 384 and the rest
    (d / 32 rows of 8 experts; of 225 experts and more d / 18 on 148 SMs)."""
    k, f = 2, 64
    p = make(T, d, E, k, f, seed=T + E, group=group, bias=E % 4 == 0)
    o = outputs(T, E, k)
    y, ws = call(p, k, 0.0, **o)
    torch.cuda.synchronize()
    check(p, k, 0.0, y, o, int(ws[:4].view(I32).item()))


@pytest.mark.parametrize("group", [0, 32, 128], ids=["bf16", "g32", "g128"])
@pytest.mark.parametrize("zeroed", [False, True], ids=["weighed", "unweighed"])
def test_tokens_with_one_very_large_value(group, zeroed):
    """One feature 2^14 times the others, as some models have; also where its
    weights are zero, so that only the others make the result."""
    T, d, E, k, f = 5, 320, 3, 2, 256
    p = make(T, d, E, k, f, seed=14, group=0)
    p["x"][:, 133] = 2.0 ** 14
    p["w_router"][133] = 0
    if zeroed:
        for w in p["w"][:2]:
            w[:, 133] = 0
    if group:
        p["group"], p["q"] = group, [moe.moe_quantize_weights_w4(w, group) for w in p["w"]]
    o = outputs(T, E, k)
    y, ws = call(p, k, 0.0, **o)
    torch.cuda.synchronize()
    check(p, k, 0.0, y, o, int(ws[:4].view(I32).item()))


@pytest.mark.parametrize("group", [0, 32, 64, 128], ids=["bf16", "g32", "g64", "g128"])
@pytest.mark.parametrize("large", ["x", "h"])
def test_activations_near_the_largest(large, group):
    """x, or h, up to fp32's largest exponent against small weights: finite."""
    T, d, E, k, f = 3, 128, 4, 2, 256
    p = make(T, d, E, k, f, seed=15, group=0)
    if large == "x":
        p["x"] *= 2.0 ** 120
        p["x"][:, 77] = torch.finfo(BF).max
        p["w_router"] *= 2.0 ** -120
        for w in p["w"][:2]:
            w *= 2.0 ** -110
    else:
        p["w"][1] *= 2.0 ** 122
        p["w"][2] *= 2.0 ** -110
    if group:
        p["group"], p["q"] = group, [moe.moe_quantize_weights_w4(w, group) for w in p["w"]]
    o = outputs(T, E, k)
    y, ws = call(p, k, 0.0, **o)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y).all())
    check(p, k, 0.0, y, o, int(ws[:4].view(I32).item()))


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_h_between_the_largest_bf16_and_the_largest_float(sign):
    """h = (1 - 2^-10) 2^128 is finite in fp32 and would round to infinity in bf16."""
    T, d, E, k, f = 1, 64, 1, 1, 64
    p = make(T, d, E, k, f, seed=16, group=0)
    p["x"].zero_()
    p["x"][0, :2] = 1.0
    for w in p["w"][:2]:
        w.zero_()
    p["w"][0][0, 0] = 2.0 ** 64                          # g = 2^64
    p["w"][1][0, 0] = sign * 2.0 ** 64 * 1020 / 1024     # u = 2^64 1023 / 1024
    p["w"][1][0, 1] = sign * 2.0 ** 64 * 3 / 1024
    p["w"][2] *= 2.0 ** -100
    o = outputs(T, E, k)
    y, ws = call(p, k, 0.0, **o)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y).all())
    check(p, k, 0.0, y, o, int(ws[:4].view(I32).item()))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("low", [-14, -15])
def test_digits_of_small_values(low, group):
    """On codes x is exact down to 2^-14 of the largest of its 128 values, and
    within 2^-22 of that value below: a small x beside a 1 that has no weight."""
    T, d, E, k, f = 32, 128, 1, 1, 128
    p = make(T, d, E, k, f, seed=17, group=0)
    p["x"].zero_()
    p["x"][:, 0] = 1.0
    odd = 2 * torch.arange(T, dtype=torch.float64, device="cuda") + 1
    p["x"][:, 1] = (2.0 ** low * (1 + odd / 128)).to(BF)
    for w, v in zip(p["w"], (7 * 2.0 ** 12, 7 * 2.0 ** 12, 7 * 2.0 ** -10)):
        w.zero_()
        w[0, 1] = v
    p["w"][2][:] = 7 * 2.0 ** -10
    p["group"], p["q"] = group, [moe.moe_quantize_weights_w4(w, group) for w in p["w"]]
    o = outputs(T, E, k)
    y, ws = call(p, k, 0.0, **o)
    torch.cuda.synchronize()
    check(p, k, 0.0, y, o, int(ws[:4].view(I32).item()))
    if low == -14:                                       # the bounds of an exact x
        slot = o["slot"].cpu().numpy()
        w = o["topk_w"].cpu().double().numpy()
        y64, bound = ref.layer64(p["x"], experts64(p), o["topk_idx"].cpu().numpy(), slot, w)
        assert bool(((y.double() - y64).abs() <= bound).all())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T, cf", [(1, 0.0), (9, 1.25), (32, 0.0)])
def test_layer_takes_any_code_and_scale(T, cf, group):
    """Codes 0..15, which the quantizer does not all make, and scales of both signs
    and zero."""
    d, E, k, f = 320, 5, 2, 192
    p = make(T, d, E, k, f, seed=18, group=0)
    g = torch.Generator().manual_seed(19)
    p["group"], p["q"] = group, []
    for K, N in ((d, f), (d, f), (f, d)):
        q = torch.randint(0, 256, (E, N // 64, K // 64, 2048), generator=g, dtype=torch.uint8)
        s = torch.randn(E, -(-K // group), N, generator=g) * K ** -0.5 / 4
        s[:, 0, 3::7] = 0
        p["q"].append((q.cuda(), s.to(BF).cuda()))
    o = outputs(T, E, k)
    y, ws = call(p, k, cf, **o)
    torch.cuda.synchronize()
    check(p, k, cf, y, o, int(ws[:4].view(I32).item()))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_largest_sums_of_digits(sign, group):
    """Code 0 against digits of -128 in all rows: x = 1 + 2^-6 is 2^21 + 2^15 units,
    whose middle digit is -128."""
    T, d, E, k, f = 3, 256, 1, 1, 128
    p = make(T, d, E, k, f, seed=20, group=0)
    p["x"][:] = sign * (1 + 2.0 ** -6)
    p["group"] = group
    p["q"] = [(torch.zeros(E, N // 64, K // 64, 2048, dtype=torch.uint8, device="cuda"),
               torch.full((E, -(-K // group), N), 2.0 ** -9, dtype=BF, device="cuda"))
              for K, N in ((d, f), (d, f), (f, d))]
    o = outputs(T, E, k)
    y, ws = call(p, k, 0.0, **o)
    torch.cuda.synchronize()
    check(p, k, 0.0, y, o, int(ws[:4].view(I32).item()))


@pytest.mark.parametrize("group", [0, 64], ids=["bf16", "w4"])
def test_weights_past_32_bit_offsets(group):
    """Experts that begin beyond 2^31 elements (and 2^32 bytes) of their tensor:
    the same result as with those experts alone."""
    d = f = 4096
    E, k, T = 140, 2, 3                                   # 2.3 G weights a matrix
    g = torch.Generator().manual_seed(13)
    x = torch.randn(T, d, generator=g).to(BF).cuda()
    last = [(torch.randn(k, d, f, generator=g) * d ** -0.5).to(BF).cuda() for _ in range(3)]
    wr = torch.zeros(d, E, device="cuda")
    wr[:, E - k:] = (torch.randn(d, k, generator=g) * d ** -0.5).cuda()
    bias = torch.full((E,), -1000.0, device="cuda")
    bias[E - k:] = 0
    small = {"x": x, "w_router": wr[:, E - k:].contiguous(), "bias": None, "group": group,
             "w": last}
    big = dict(small, w_router=wr, bias=bias)
    if group:
        small["q"] = [moe.moe_quantize_weights_w4(w, group) for w in last]
        big["q"] = []
        for q, s in small["q"]:
            Q = torch.zeros(E, *q.shape[1:], dtype=torch.uint8, device="cuda")
            S = torch.zeros(E, *s.shape[1:], dtype=BF, device="cuda")
            Q[E - k:], S[E - k:] = q, s
            big["q"].append((Q, S))
    else:
        big["w"] = []
        for w in last:
            W = torch.zeros(E, d, f, dtype=BF, device="cuda")
            W[E - k:] = w
            big["w"].append(W)
    o, ob = outputs(T, k, k), outputs(T, E, k)
    y, _ = call(small, k, 0.0, **o)
    yb, ws = call(big, k, 0.0, **ob)
    torch.cuda.synchronize()
    assert int(ws[:4].view(I32).item()) == 0
    assert torch.equal(ob["topk_idx"] - (E - k), o["topk_idx"])
    # the gate weights may differ in the last bit (another split of the router)
    assert bool(((y.double() - yb.double()).abs() <= 2.02 * ref.U16 * y.double().abs() + 1e-30).all())
    if not group:
        q, s = moe.moe_quantize_weights_w4(big["w"][0], 128)
        back = moe.moe_dequantize_weights_w4(q, s, 128)
        q1, s1 = moe.moe_quantize_weights_w4(last[0], 128)
        assert torch.equal(q[E - k:], q1) and torch.equal(s[E - k:], s1)
        assert torch.equal(back[E - k:], moe.moe_dequantize_weights_w4(q1, s1, 128))


@pytest.mark.parametrize("T, d, f, group", [(2, 1 << 20, 64, 0), (3, 64, 1 << 20, 0),
                                            (2, 1 << 17, 64, 64), (9, 64, 1 << 17, 32)])
def test_widest_layers(T, d, f, group):
    """Widths up to the largest allowed."""
    E, k = 2, 1
    p = make(T, d, E, k, f, seed=21, group=group)
    o = outputs(T, E, k)
    y, ws = call(p, k, 0.0, **o)
    torch.cuda.synchronize()
    check(p, k, 0.0, y, o, int(ws[:4].view(I32).item()))


def test_layers_one_after_another():
    """Four layers of a model on one workspace, bf16 and codes in turn, each call's
    tokens written by the kernel before it: the bits of the same calls with a
    synchronization between, called and as a graph."""
    T, d, E, k, f, group = 6, 256, 12, 3, 192, 64
    layers = [make(T, d, E, k, f, seed=30 + i, group=group if i % 2 else 0, bias=True)
              for i in range(4)]
    ws = torch.empty(moe.moe_workspace_size_few(T, d, E, k, f), dtype=torch.uint8, device="cuda")
    x0 = layers[0]["x"].clone()
    bufs = [torch.empty_like(x0) for _ in range(5)]

    def model(sync):
        torch.mul(x0, 1.5, out=bufs[0])
        for i, p in enumerate(layers):
            call(dict(p, x=bufs[i]), k, 1.0, y=bufs[i + 1], ws=ws)
            if sync:
                torch.cuda.synchronize()
            bufs[i + 1].add_(bufs[i])
            if sync:
                torch.cuda.synchronize()
    model(True)
    want = bufs[4].clone()
    assert bool(torch.isfinite(want).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        model(False)
    for run in (lambda: model(False), graph.replay) * 10:
        for b in bufs:
            b.fill_(math.nan)
        run()
        torch.cuda.synchronize()
        assert torch.equal(bufs[4], want)


@pytest.mark.parametrize("E, K, N, group", [(65535, 64, 64, 128), (1, 1 << 20, 64, 32),
                                            (1, 64, 1 << 20, 64)])
def test_largest_conversions(E, K, N, group):
    """The most experts, the longest and the widest matrix: corners against the same
    corners alone."""
    g = torch.Generator(device="cuda").manual_seed(22)
    w = torch.randn(E, K, N, generator=g, device="cuda", dtype=BF)
    q, s = moe.moe_quantize_weights_w4(w, group)
    back = moe.moe_dequantize_weights_w4(q, s, group)
    for e in {0, E // 2, E - 1}:
        for k0 in {0, (K - 64) // 128 * 128}:
            for n0 in {0, N - 64}:
                part = w[e:e + 1, k0:k0 + 64, n0:n0 + 64].contiguous()
                codes, scales = ref.quantize64(part.cpu(), group)
                assert torch.equal(back[e:e + 1, k0:k0 + 64, n0:n0 + 64].cpu(),
                                   ref.values64(codes, scales, group).to(BF))
    half = ref.U16 * w.abs().max().double()
    step = s.abs().max().double()
    assert float((back.double() - w.double()).abs().max()) <= float(0.52 * step + half)


def test_no_tokens():
    p = make(1, 64, 4, 2, 64, seed=1, group=32)
    p["x"] = torch.empty(0, 64, dtype=BF, device="cuda")
    assert call(p, 2, 0.0)[0].shape == (0, 64)
    assert call(dict(p, group=0), 2, 1.0)[0].shape == (0, 64)


def test_binding_refusals():
    T, d, E, k, f = 4, 128, 8, 2, 64
    p = make(T, d, E, k, f, seed=1, group=64)
    b = dict(p, group=0)
    flat = [t for qs in p["q"] for t in qs]

    def few(**kw):
        a = {**b, **kw}
        return moe.moe_layer_forward_few(a["x"], a["w_router"], a["bias"], *a["w"], a.get("k", k),
                                         a.get("cf", 0.0), **a.get("out", {}))

    def w4(i=None, t=None, **kw):
        fl = list(flat)
        if i is not None:
            fl[i] = t
        return moe.moe_layer_forward_few_w4(p["x"], p["w_router"], None, *fl, k, 0.0,
                                            kw.get("group", 64))
    few()
    w4()
    x = p["x"]
    with pytest.raises(ValueError, match="at most 32"):
        few(x=torch.zeros(33, d, dtype=BF, device="cuda"))
    with pytest.raises(TypeError):
        few(x=x.float())
    with pytest.raises(ValueError):
        few(x=torch.zeros(d, T, dtype=BF, device="cuda").t())         # not contiguous
    with pytest.raises(ValueError):
        few(x=x[:, :64].contiguous())                                 # another width
    with pytest.raises(ValueError):
        few(x=x[0])
    with pytest.raises(TypeError):
        few(w_router=p["w_router"].double())
    with pytest.raises(ValueError):
        few(w_router=p["w_router"].cpu())
    with pytest.raises(ValueError):
        few(bias=torch.zeros(E + 1, device="cuda"))
    for i in range(3):
        ws = list(p["w"])
        ws[i] = ws[i][:-1].contiguous()
        with pytest.raises(ValueError):
            few(w=ws)
        ws[i] = p["w"][i].cpu()
        with pytest.raises(ValueError):
            few(w=ws)
    for name, t in outputs(T, E, k).items():
        with pytest.raises(ValueError):
            few(out={name: t[:-1].contiguous()})
        with pytest.raises(TypeError):
            few(out={name: t.double()})
    with pytest.raises(ValueError):
        few(out={"y": torch.empty(T + 1, d, dtype=BF, device="cuda")})
    need = moe.moe_workspace_size_few(T, d, E, k, f)
    with pytest.raises(moe.MoEError, match="WORKSPACE"):
        few(out={"ws": torch.empty(need - 1, dtype=torch.uint8, device="cuda")})
    with pytest.raises(moe.MoEError, match="INVALID"):
        few(out={"ws": torch.empty(need + 16, dtype=torch.uint8, device="cuda")[1:]})
    for kw in ({"k": 0}, {"k": 9}, {"cf": -1.0}, {"cf": math.nan}):
        with pytest.raises((moe.MoEError, ValueError)):
            few(**kw)
    for i, t in enumerate(flat):
        with pytest.raises(ValueError):
            w4(i, t[:-1].contiguous())
        with pytest.raises(TypeError):
            w4(i, t.float())
    for group in (0, 16, 32, 128, 256):                               # not the scales' one
        with pytest.raises(ValueError):
            w4(group=group)
    with pytest.raises(TypeError):
        moe.moe_quantize_weights_w4(p["w"][0].float())
    with pytest.raises(ValueError):
        moe.moe_quantize_weights_w4(p["w"][0], 48)
    with pytest.raises(ValueError):
        moe.moe_quantize_weights_w4(torch.zeros(2, 96, 64, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_quantize_weights_w4(p["w"][0].transpose(1, 2))
    with pytest.raises(ValueError):
        moe.moe_dequantize_weights_w4(flat[0], flat[1], 32)
    with pytest.raises(ValueError):
        moe.moe_dequantize_weights_w4(flat[0][..., :1024], flat[1], 64)
