"""Cases that measure the few-token operators of the MoE layer: the whole layer
for the tokens of a decode step, on bf16 experts and on experts held as 4-bit
codes with group scales, and the two conversions between those forms.

`run` computes each in plain torch operations, or, where `own` is set, calls
the library.  The 4-bit form is the library's: codes u in 0..15 stand for
(u - 8) * scale; uint8 [E, N/64, K/64, 2048], a 64-column by 64-row tile of the
weight being 4 blocks of 16 columns, each 32 lanes (8 column residues g by 4
row pairs c) of four 32-bit words (16 rows each), whose nibble i + 4 h holds
column g + 8 (i % 2) and row 2 c + h + 8 (i / 2); scales bf16
[E, ceil(K / group), N].
"""
import math

import torch

own = False


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one token through a toy layer: what a call costs when nothing else does
        dict(name="few.bf16.tiny.t1", op="few", T=1, d=128, E=8, k=2, f=256, cf=0.0, bias=False),
        # a single chat's decode step through the fine-grained layer
        dict(name="few.bf16.fine.t1", op="few", T=1, d=7168, E=256, k=8, f=2048, cf=0.0,
             bias=False),
        # two chats, few large experts
        dict(name="few.bf16.mixtral.t2", op="few", T=2, d=4096, E=8, k=2, f=14336, cf=0.0,
             bias=False),
        # the largest batch of the call: a small server's decode step
        dict(name="few.bf16.fine.t32", op="few", T=32, d=7168, E=256, k=8, f=2048, cf=0.0,
             bias=False),
        # the same single chat with the experts in 4 bits
        dict(name="few.w4.fine.t1", op="few_w4", T=1, d=7168, E=256, k=8, f=2048, cf=0.0,
             bias=False, group=128),
        # a draft of three tokens, odd expert count, narrow groups, router bias, capacity limit
        dict(name="few.w4.odd.t3", op="few_w4", T=3, d=2048, E=61, k=5, f=1408, cf=1.0, bias=True,
             group=32),
        # eight chats, few large experts
        dict(name="few.w4.mixtral.t8", op="few_w4", T=8, d=4096, E=8, k=2, f=14336, cf=0.0,
             bias=False, group=64),
        dict(name="few.w4.fine.t32", op="few_w4", T=32, d=7168, E=256, k=8, f=2048, cf=0.0,
             bias=False, group=128),
        # converting one layer's matrices: a small odd one, and a large one
        dict(name="quantize.odd", op="quantize", E=3, K=320, N=1408, group=32),
        dict(name="quantize.mixtral", op="quantize", E=8, K=4096, N=14336, group=128),
        # the experts of one layer back in bf16, before a long prompt goes through it
        dict(name="dequantize.odd", op="dequantize", E=5, K=448, N=704, group=128),
        dict(name="dequantize.skewed", op="dequantize", E=64, K=2048, N=1408, group=64),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["few", "few", "few_w4", "few_w4", "quantize", "dequantize"])
    group = rng.choice([32, 64, 128])
    if op in ("quantize", "dequantize"):
        E, K, N = _spread(rng, 1, 64), 64 * _spread(rng, 1, 112), 64 * _spread(rng, 1, 224)
        return dict(op=op, E=max(1, min(E, (1 << 31) // (K * N))), K=K, N=N, group=group)
    d, f = 64 * _spread(rng, 1, 112), 64 * _spread(rng, 1, 224)
    E = _spread(rng, 1, 256)
    E = max(1, min(E, 256 * 7168 * 2048 // (d * f)))
    case = dict(op=op, T=_spread(rng, 1, 32), d=d, E=E, k=min(E, rng.randint(1, 8)), f=f,
                cf=rng.choice([0.0, 0.0, 1.0, 1.25]), bias=rng.random() < 0.5)
    if op == "few_w4":
        case["group"] = group
    while work(case)["bytes"] > work(listed()[3])["bytes"] and case["T"] > 1:
        case["T"] -= 1
    return case


def work(case):
    c = case
    if c["op"] in ("quantize", "dequantize"):
        n, groups = c["E"] * c["K"] * c["N"], c["E"] * -(-c["K"] // c["group"]) * c["N"]
        codes, values = n / 2 + 2 * groups, 2 * n
        # quantize: the weights in, the codes out; then the codes in, their values out
        return {"bytes": codes + values + (codes + values if c["op"] == "quantize" else 0),
                "flops": n}
    T, d, E, k, f = (c[n] for n in ("T", "d", "E", "k", "f"))
    p = k / E                                   # a token's chance to choose a given expert
    cap = T if c["cf"] == 0 else math.ceil(c["cf"] * k * T / E)
    active = E * (1 - (1 - p) ** T)             # experts that any token chose
    pairs = E * sum(min(n, cap) * math.comb(T, n) * p ** n * (1 - p) ** (T - n)
                    for n in range(T + 1))
    weight = 0.5 + 2 / c["group"] if c["op"] == "few_w4" else 2
    return {"bytes": 3 * active * d * f * weight + 4 * d * E + 4 * T * d + 4 * T * E + 8 * T * k,
            "flops": 6 * pairs * d * f + 2 * T * d * E}


# -------------------------------------------------------------------- inputs
def _codes(gen, E, K, N, group, std):
    """Codes and scales as quantizing N(0, std^2) weights leaves them: the
    largest of a group at 7, the others spread normally below it."""
    top = math.sqrt(2 * math.log(2 * group))    # about the largest of `group` normal values
    v = torch.randn(E, N // 64, K // 64, 4096, generator=gen, device="cuda", dtype=torch.float16)
    v = v.mul_(7 / top).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
    q = v[..., 0::2] | (v[..., 1::2] << 4)
    spread = torch.rand(E, -(-K // group), N, generator=gen, device="cuda")
    return q, (spread.mul_(0.3).add_(0.85) * (std * top / 7)).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(shape, std, dtype):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(std)

    if c["op"] == "quantize":
        return dict(case=c, w=normal((c["E"], c["K"], c["N"]), c["K"] ** -0.5, torch.bfloat16))
    if c["op"] == "dequantize":
        q, s = _codes(gen, c["E"], c["K"], c["N"], c["group"], c["K"] ** -0.5)
        return dict(case=c, q=q, s=s)
    T, d, E, k, f = (c[n] for n in ("T", "d", "E", "k", "f"))
    st = dict(case=c, x=normal((T, d), 1.0, torch.float32).to(torch.bfloat16),
              w_router=normal((d, E), d ** -0.5, torch.float32),
              bias=normal((E,), 0.5, torch.float32) if c["bias"] else None)
    for name, K, N in (("gate", d, f), ("up", d, f), ("down", f, d)):
        if c["op"] == "few":
            st["w_" + name] = normal((E, K, N), K ** -0.5, torch.bfloat16)
        else:
            st["q_" + name], st["s_" + name] = _codes(gen, E, K, N, c["group"], K ** -0.5)
    # the caller's buffers for the routing results
    st["logits"] = torch.empty(T, E, dtype=torch.float32, device="cuda")
    st["topk_idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
    st["topk_w"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
    return st


# --------------------------------------------------------------------- passes
def run(state):
    op = state["case"]["op"]
    if own:
        return {"few": _own_few, "few_w4": _own_few_w4, "quantize": _own_quantize,
                "dequantize": _own_dequantize}[op](state)
    if op == "quantize":
        return _plain_quantize(state)
    if op == "dequantize":
        return _plain_values(state["q"], state["s"], state["case"]["group"]).to(torch.bfloat16)
    return _plain_layer(state)


def _own_few(st):
    import mixture_experts_layer_36_b200 as moe
    c = st["case"]
    # the workspace of the first call is kept, as a decode loop keeps it
    y, st["ws"] = moe.moe_layer_forward_few(
        st["x"], st["w_router"], st["bias"], st["w_gate"], st["w_up"], st["w_down"], c["k"],
        c["cf"], logits=st["logits"], topk_idx=st["topk_idx"], topk_w=st["topk_w"],
        ws=st.get("ws"))
    return y, st["logits"], st["topk_idx"], st["topk_w"]


def _own_few_w4(st):
    import mixture_experts_layer_36_b200 as moe
    c = st["case"]
    y, st["ws"] = moe.moe_layer_forward_few_w4(
        st["x"], st["w_router"], st["bias"], st["q_gate"], st["s_gate"], st["q_up"], st["s_up"],
        st["q_down"], st["s_down"], c["k"], c["cf"], c["group"], logits=st["logits"],
        topk_idx=st["topk_idx"], topk_w=st["topk_w"], ws=st.get("ws"))
    return y, st["logits"], st["topk_idx"], st["topk_w"]


def _own_quantize(st):
    import mixture_experts_layer_36_b200 as moe
    q, s = moe.moe_quantize_weights_w4(st["w"], st["case"]["group"])
    return s, moe.moe_dequantize_weights_w4(q, s, st["case"]["group"])


def _own_dequantize(st):
    import mixture_experts_layer_36_b200 as moe
    return moe.moe_dequantize_weights_w4(st["q"], st["s"], st["case"]["group"])


def _plain_unpack(q):
    """The codes of packed [P, N/64, K/64, 2048] matrices as integers [P, K, N]."""
    P, nt, kt = q.shape[:3]
    # tile bytes: block b of 16 columns, column residue g, row pair c, word s,
    # and within a word byte -> nibble = 4 h + 2 ih + il
    v = torch.stack((q & 15, q >> 4), -1).view(P, nt, kt, 4, 8, 4, 4, 2, 2, 2)
    # dims: 0 P, 1 nt, 2 kt, 3 b, 4 g, 5 c, 6 s, 7 h, 8 ih, 9 il
    return v.permute(0, 2, 6, 8, 5, 7, 1, 3, 9, 4).reshape(P, kt * 64, nt * 64)


def _plain_values(q, s, group):
    v = _plain_unpack(q)
    v = v.float().sub_(8)
    return v.mul_(s.float().repeat_interleave(group, 1)[:, :v.shape[1]])


def _plain_quantize(st):
    w, group = st["w"], st["case"]["group"]
    E, K, N = w.shape
    groups = -(-K // group)
    v = torch.zeros(E, groups * group, N, device=w.device)
    v[:, :K] = w
    v = v.view(E, groups, group, N)
    s = (v.abs().amax(2) / 7).to(torch.bfloat16)
    s = torch.where(s == 0, torch.ones_like(s), s)
    code = (v / s.float()[:, :, None]).round_().clamp_(-7, 7)
    return s, code.mul_(s.float()[:, :, None]).view(E, -1, N)[:, :K].to(torch.bfloat16)


def _kept(idx, E, cf):
    """Whether each (token, choice) has a place among its expert's, places
    being taken in token order up to the capacity."""
    T, k = idx.shape
    chosen = torch.zeros(T, E, dtype=torch.int64, device=idx.device).scatter_(1, idx, 1)
    slot = (chosen.cumsum(0) - chosen).gather(1, idx)
    return slot < (T if cf == 0 else math.ceil(cf * k * T / E))


def _plain_layer(st):
    c, x = st["case"], st["x"]
    T, d, E, k, f = (c[n] for n in ("T", "d", "E", "k", "f"))
    # values next to a border decide which experts run: the scores in 64 bits
    logits = x.double() @ st["w_router"].double()
    if st["bias"] is not None:
        logits = logits + st["bias"].double()
    logits = logits.float()
    best, idx = logits.sort(dim=1, descending=True, stable=True)
    best, idx = best[:, :k], idx[:, :k]
    p = (best - best[:, :1]).exp()
    topk_w = p / p.sum(1, keepdim=True)
    kept = _kept(idx, E, c["cf"])
    pair = idx.reshape(-1)

    def product(rows, name):
        w = (st["w_" + name][pair].float() if c["op"] == "few" else
             _plain_values(st["q_" + name][pair], st["s_" + name][pair], c["group"]))
        return (rows[:, None, :] @ w)[:, 0]

    rows = x.float().repeat_interleave(k, 0)
    g = product(rows, "gate")
    h = g / (1 + (-g).exp()) * product(rows, "up")
    o = product(h, "down").view(T, k, d)
    y = torch.where(kept[:, :, None], o * topk_w[:, :, None], torch.zeros_like(o)).sum(1)
    y = torch.where(kept.any(1, keepdim=True), y, x.float())
    return y.to(torch.bfloat16), logits, idx.to(torch.int32), topk_w


# ---------------------------------------------------------------- definitions
def exact(case, seed):
    """The definitions in 64 bits, element by element of the routing table."""
    c, st = case, prepare(case, seed)
    f64 = torch.float64

    def matrix(q, s):
        # nibble j of word s of lane (g, c): its row and column, written out
        K, N = q.shape[1] * 64, q.shape[0] * 64
        nib = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], q.shape[1], 4, 32, 4, 8)
        at = [torch.arange(n, device=q.device).view([-1 if a == b else 1 for b in range(6)])
              for a, n in enumerate(nib.shape)]
        nt, kt, b, lane, word, j = at
        col = nt * 64 + b * 16 + torch.div(lane, 4, rounding_mode="floor") + 8 * (j % 2)
        row = (kt * 64 + word * 16 + 2 * (lane % 4) + torch.div(j, 4, rounding_mode="floor")
               + 8 * (torch.div(j, 2, rounding_mode="floor") % 2))
        out = torch.empty(K * N, dtype=f64, device=q.device)
        out[(row * N + col).expand(nib.shape).reshape(-1)] = nib.reshape(-1).to(f64) - 8
        group = torch.arange(K, device=q.device) // c["group"]
        return out.view(K, N) * s.to(f64)[group]

    if c["op"] == "quantize":
        w, group = st["w"], c["group"]
        scales, values = [], []
        for k0 in range(0, c["K"], group):
            v = w[:, k0:k0 + group].to(f64)
            s = (v.abs().amax(1, keepdim=True) / 7).to(torch.bfloat16).to(f64)
            s = s + (s == 0)
            scales.append(s)
            values.append(torch.clamp(torch.round(v / s), -7, 7) * s)
        return torch.cat(scales, 1), torch.cat(values, 1)
    if c["op"] == "dequantize":
        return torch.stack([matrix(st["q"][e], st["s"][e]) for e in range(c["E"])])

    x = st["x"].to(f64)
    logits = torch.einsum("td,de->te", x, st["w_router"].to(f64))
    if st["bias"] is not None:
        logits = logits + st["bias"].to(f64)
    seen = logits.float().cpu().tolist()        # the choice is made on the values as returned
    cap = c["T"] if c["cf"] == 0 else math.ceil(c["cf"] * c["k"] * c["T"] / c["E"])
    taken, by_expert, gates = [0] * c["E"], {}, torch.zeros(c["T"], c["k"], dtype=f64)
    served = [False] * c["T"]
    for t in range(c["T"]):
        order = sorted(range(c["E"]), key=lambda e: (-seen[t][e], e))[:c["k"]]
        p = torch.exp(torch.tensor([seen[t][e] for e in order], dtype=f64) - seen[t][order[0]])
        gates[t] = p / p.sum()
        for j, e in enumerate(order):
            taken[e] += 1
            if taken[e] <= cap:
                by_expert.setdefault(e, []).append((t, j))
                served[t] = True
    y = torch.zeros_like(x)
    for e, pairs in by_expert.items():
        w = [st["w_" + n][e].to(f64) if c["op"] == "few" else matrix(st["q_" + n][e], st["s_" + n][e])
             for n in ("gate", "up", "down")]
        rows = x[[t for t, _ in pairs]]
        g = rows @ w[0]
        o = (g * torch.sigmoid(g) * (rows @ w[1])) @ w[2]
        for i, (t, j) in enumerate(pairs):
            y[t] += gates[t, j].item() * o[i]
    for t in range(c["T"]):
        if not served[t]:
            y[t] = x[t]
    return y, logits, None, gates
