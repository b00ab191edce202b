"""The expert products of a mixture-of-experts layer, as cases to be timed and compared.

Three operators, each in its plain form (elementary torch operations) and, where `own` is true, as a user calls
them in this package:

  int8     w8a8_grouped_linear / w8a8_grouped_gemm: rows sorted by expert (offsets[e] .. offsets[e + 1] belong to
           expert e) times that expert's INT8 weight, one scale for each token and output channel;
  moe8     w8a8_moe_grouped_gemm: routing, INT8 gate_up with silu(gate) * up, INT8 down, weighted combine;
  weight4  w4a16_grouped_gemm: bf16 rows sorted by expert times that expert's packed 4-bit weight.

A case holds sizes only.  The rows of each expert follow from the case, so every seed has the same raggedness and
other values.
"""
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one token of a 64-expert top-6 layer: its six rows through gate_up, bf16 in (latency counts)
        dict(name="int8 one token", op="int8", bf16_in=True, rows=6, pad=0, E=64, K=2048, N=2816, skew=False, empty=0),
        # 64 tokens, top-8 of 32 skewed experts, gate_up of a wide layer: weight streaming
        dict(name="int8 decode batch", op="int8", bf16_in=True, rows=512, pad=0, E=32, K=7168, N=4096, skew=True, empty=0),
        # 4096 prompt tokens, top-6 of 64 experts, the down product on rows quantized before
        dict(name="int8 prompt down", op="int8", bf16_in=False, rows=24576, pad=0, E=64, K=1408, N=2048, skew=False, empty=0),
        # odd sizes: experts without rows, a padded batch whose last rows belong to nobody
        dict(name="int8 ragged odd", op="int8", bf16_in=False, rows=741, pad=27, E=11, K=1152, N=1040, skew=True, empty=3),
        # one token through the whole layer: seven short steps, latency counts
        dict(name="moe8 one token", op="moe8", T=1, E=64, topk=6, H=2048, I=1408, skew=False),
        # a decode batch over skewed wide experts: weight streaming
        dict(name="moe8 decode batch", op="moe8", T=64, E=32, topk=8, H=7168, I=2048, skew=True),
        # a prompt through a 64-expert layer: tensor work
        dict(name="moe8 prompt", op="moe8", T=4096, E=64, topk=6, H=2048, I=1408, skew=False),
        # odd sizes
        dict(name="moe8 odd", op="moe8", T=333, E=13, topk=3, H=1152, I=640, skew=True),
        # weight-only: one token's rows, symmetric groups of 128
        dict(name="weight4 one token", op="weight4", rows=6, pad=0, E=64, K=2048, N=2816, group=128, sym=True, skew=False, empty=0),
        # weight-only decode batch, asymmetric groups of 64
        dict(name="weight4 decode batch", op="weight4", rows=512, pad=0, E=32, K=7168, N=4096, group=64, sym=False, skew=True, empty=0),
        # weight-only prompt
        dict(name="weight4 prompt", op="weight4", rows=24576, pad=0, E=64, K=2048, N=2816, group=128, sym=True, skew=False, empty=0),
        # weight-only, odd sizes, empty experts, rows of nobody
        dict(name="weight4 ragged odd", op="weight4", rows=777, pad=23, E=10, K=1344, N=1088, group=64, sym=False, skew=True, empty=2),
    ]


def draw(rng):
    span = lambda a, b: int(round(a * (b / a) ** rng.random()))  # noqa: E731  spread over the logarithm
    while True:
        op = rng.choice(["int8", "moe8", "weight4"])
        E = span(1, 64)
        skew = rng.random() < 0.5
        if op == "moe8":
            H, I = 128 * span(1, 56), 128 * span(1, 16)
            topk, T = rng.randint(1, min(8, E)), span(1, 4096)
            if T * topk * 3 * H * I <= 24576 * 3 * 2048 * 1408 and E * H * I <= 32 * 7168 * 2048:
                return dict(op=op, T=T, E=E, topk=topk, H=H, I=I, skew=skew)
            continue
        rows = span(1, 24576)
        pad, empty = rng.choice([0, 0, rng.randint(1, 40)]), rng.randint(0, E // 4)
        if op == "int8":
            K, N = 128 * span(1, 56), 16 * span(1, 256)
            more = dict(bf16_in=rng.random() < 0.5)
        else:
            group = rng.choice([64, 128])
            K, N = group * span(1, 7168 // group), 64 * span(1, 64)
            more = dict(group=group, sym=rng.random() < 0.5)
        if rows * K * N <= 24576 * 2048 * 2816 and E * K * N <= 32 * 7168 * 4096:
            return dict(op=op, rows=rows, pad=pad, E=E, K=K, N=N, skew=skew, empty=empty, **more)


def shares(E, skew, empty, g):
    """How the rows spread over the experts: evenly, or by a Zipf law over a random order; `empty` experts get none."""
    order = torch.randperm(E, generator=g)
    p = (order.double() + 1).pow(-1.1) if skew else torch.ones(E, dtype=torch.float64)
    p[torch.randperm(E, generator=g)[:empty]] = 0
    return p / p.sum()


def counts_of(c):
    """Rows of each expert (from the sizes alone)."""
    g = torch.Generator().manual_seed(c["rows"] * 131 + c["E"])
    pick = torch.multinomial(shares(c["E"], c["skew"], c["empty"], g), c["rows"], replacement=True, generator=g)
    return torch.bincount(pick, minlength=c["E"])


# ----------------------------------------------------------------- inputs ---

def generator(seed, device=DEV):
    return torch.Generator(device=device).manual_seed(int(seed))


def activations(g, rows, K):
    """bf16 rows with a few channels 50 times as large, as activations in front of a linear layer have them."""
    x = torch.randn(rows, K, generator=g, device=DEV)
    x[:, torch.randperm(K, generator=g, device=DEV)[:8]] *= 50.0
    return x.to(torch.bfloat16)


def int8_weight(g, E, K, N):
    """Codes [E, N, K] and channel scales [E, N] of normal weights with deviation 0.02."""
    q = torch.empty(E, N, K, dtype=torch.int8, device=DEV)
    for e in range(E):
        q[e] = torch.randn(N, K, generator=g, device=DEV).mul_(30.0).round_().clamp_(-127, 127).to(torch.int8)
    s = (0.02 / 30.0) * (0.5 + torch.rand(E, N, generator=g, device=DEV))
    return q, s


def int4_weight(g, E, K, N, group, sym):
    """Packed codes, group scales [E, K / group, N] and zero-points of normal weights.  The codes are drawn one by
    one from the same law, so the bytes can be drawn in packed order."""
    n = K * N // 2
    packed = torch.empty(E, n, dtype=torch.uint8, device=DEV)
    for e in range(E):
        v = torch.randn(2, n, generator=g, device=DEV)
        v = v.mul_(2.3).round_().clamp_(-7, 7).to(torch.int16) & 15 if sym else \
            v.mul_(3.0).add_(7.5).round_().clamp_(0, 15).to(torch.int16)
        packed[e] = (v[0] | (v[1] << 4)).to(torch.uint8)
    s = (0.02 / (2.3 if sym else 3.0)) * (0.5 + torch.rand(E, K // group, N, generator=g, device=DEV))
    z = None if sym else torch.randint(6, 10, (E, K // group, N), generator=g, device=DEV, dtype=torch.uint8)
    return packed, s, z


def router_logits(g, c):
    logits = torch.randn(c["T"], c["E"], generator=g, device=DEV)
    p = shares(c["E"], c["skew"], 0, torch.Generator().manual_seed(c["E"]))
    return logits + p.log().float().to(DEV)


def plan_table(s, counts):
    """What a batched product over experts with rows is laid out by: which they are, and the most rows of one."""
    s["busy"] = (counts > 0).nonzero().flatten().to(DEV)
    s["cap"] = int(counts.max())


def prepare(case, seed):
    c, g = case, generator(seed)
    s = dict(case=c)
    if c["op"] == "moe8":
        s["x"] = activations(g, c["T"], c["H"])
        s["logits"] = router_logits(g, c)
        s["q1"], s["s1"] = int8_weight(g, c["E"], c["H"], 2 * c["I"])
        s["q2"], s["s2"] = int8_weight(g, c["E"], c["I"], c["H"])
        picked = s["logits"].topk(c["topk"], dim=1).indices.flatten()
        plan_table(s, torch.bincount(picked, minlength=c["E"]))
        return s
    n = counts_of(c)
    plan_table(s, n)
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(torch.int32).to(DEV)
    rows = c["rows"] + c["pad"]
    s["out"] = torch.zeros(rows, c["N"], dtype=torch.bfloat16, device=DEV)
    x = activations(g, rows, c["K"])
    if c["op"] == "int8":
        s["q"], s["s"] = int8_weight(g, c["E"], c["K"], c["N"])
        if c["bf16_in"]:
            s["x"] = x
        else:
            s["qx"], s["sx"] = token_codes(x)
    else:
        s["x"] = x
        s["packed"], s["s"], s["z"] = int4_weight(g, c["E"], c["K"], c["N"], c["group"], c["sym"])
    return s


# ------------------------------------------------------------- plain form ---

def token_codes(x):
    """INT8 codes and the scale of each row: s = max|x| / 127, q = round(x / s), ties to even."""
    x = x.float()
    s = x.abs().amax(1) / 127
    q = (x / torch.where(s > 0, s, torch.ones_like(s))[:, None]).round().clamp(-127, 127)
    return q.to(torch.int8), s


def places(offsets, rows, cap):
    """For rows sorted by expert: each row's place in a table of `cap` rows for each expert that has any."""
    offsets = offsets.long()
    r = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets[1:], r, right=True)
    rank = (offsets[1:] > offsets[:-1]).cumsum(0) - 1
    return rank[e] * cap + r - offsets[e]


def spread(x, place, E, cap):
    table = torch.zeros(E * cap, x.shape[1], dtype=torch.float32, device=x.device)
    table[place] = x.float()
    return table.view(E, cap, -1)


def of_busy(w, busy):
    """The weights (or scales) of the experts that have rows."""
    return w if w is None or busy.numel() == w.shape[0] else w[busy]


def int8_products(qx, place, cap, q):
    """sum_k qx[r, k] q[e(r), n, k], exactly: products of pieces of at most 1024 k stay below 2^24 in fp32, and the
    pieces are added in fp64."""
    E, N, K = q.shape
    piece = max(d for d in range(1, 1025) if K % d == 0)
    a = spread(qx, place, E, cap).view(E, cap, K // piece, piece).transpose(1, 2)
    b = q.view(E, N, K // piece, piece).permute(0, 2, 3, 1).float()
    acc = torch.matmul(a, b).sum(1, dtype=torch.float64)
    return acc.view(E * cap, N)[place].float()


def int8_rows(qx, sx, place, t, q, s):
    """The rows of the grouped INT8 product in fp32: s_x s_w sum_k q_x q_w."""
    cap, q, s = t["cap"], of_busy(q, t["busy"]), of_busy(s, t["busy"])
    acc = int8_products(qx, place, cap, q)
    return sx[:, None] * (s[torch.div(place, cap, rounding_mode="floor")] * acc)


def plain_int8(t):
    c, out = t["case"], t["out"]
    rows = c["rows"]
    qx, sx = token_codes(t["x"][:rows]) if c["bf16_in"] else (t["qx"][:rows], t["sx"][:rows])
    place = places(t["offsets"], rows, t["cap"])
    out[:rows] = int8_rows(qx, sx, place, t, t["q"], t["s"]).to(torch.bfloat16)
    return out


def plain_moe8(t):
    c, logits = t["case"], t["logits"]
    E, k, I = c["E"], c["topk"], c["I"]
    idx = logits.sort(dim=1, descending=True, stable=True).indices[:, :k]
    ex = (logits - logits.amax(1, keepdim=True)).exp()
    weight = (ex / ex.sum(1, keepdim=True)).gather(1, idx)
    flat = idx.flatten()
    order = flat.sort(stable=True).indices  # by expert, then token, then slot
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    qx, sx = token_codes(t["x"])
    src = torch.div(order, k, rounding_mode="floor")
    place = places(offsets, flat.numel(), t["cap"])
    gu = int8_rows(qx[src], sx[src], place, t, t["q1"], t["s1"])
    gate, up = gu[:, :I], gu[:, I:]
    h = (gate / (1 + (-gate).exp()) * up).to(torch.bfloat16)
    qh, sh = token_codes(h)
    y = int8_rows(qh, sh, place, t, t["q2"], t["s2"]).to(torch.bfloat16)
    back = torch.empty_like(y)
    back[order] = y
    out = (weight[:, :, None] * back.float().view(-1, k, c["H"])).sum(1)
    return out.to(torch.bfloat16), idx.to(torch.int32), weight, offsets.to(torch.int32)


def int4_weights(packed, s, z, K, N, group, sym):
    """The bf16 weights [E, K, N] that packed codes stand for: 64 columns by one group of k to a block, chunks of 32 k
    of one column in 16 bytes, byte b holding k = b in its low and k = b + 16 in its high nibble."""
    E, G = packed.shape[0], K // group
    p = packed.view(E, N // 64, G, group // 32, 64, 16)
    q = torch.stack([p & 15, p >> 4], dim=-2)  # [E, column block, group, chunk, column, half, byte]
    q = q.permute(0, 2, 3, 5, 6, 1, 4).reshape(E, G, group, N)
    q = (q ^ 8).float() - 8 if sym else q.float() - z[:, :, None, :].float()
    return (s[:, :, None, :] * q).to(torch.bfloat16).view(E, K, N)


def plain_weight4(t):
    c, out = t["case"], t["out"]
    rows, cap = c["rows"], t["cap"]
    place = places(t["offsets"], rows, cap)
    packed, s, z = (of_busy(v, t["busy"]) for v in (t["packed"], t["s"], t["z"]))
    w = int4_weights(packed, s, z, c["K"], c["N"], c["group"], c["sym"])
    y = torch.matmul(spread(t["x"][:rows], place, w.shape[0], cap), w.float())
    out[:rows] = y.view(-1, c["N"])[place].to(torch.bfloat16)
    return out


# --------------------------------------------------------------- own calls --

def own_run(t):
    import moe_linear_layers_w4a8_b200 as m
    c = t["case"]

    def int8(q, s):
        E, N, K = q.shape
        return m.PackedW8(q_w=q, s_w=s, desc=m.WDesc(8, 1, K, K, N, m.LAYOUT_VERSION), experts=E)

    if c["op"] == "int8":
        if c["bf16_in"]:
            return m.w8a8_grouped_linear(t["x"], t["offsets"], int8(t["q"], t["s"]), out=t["out"])
        return m.w8a8_grouped_gemm(t["qx"], t["sx"], t["offsets"], int8(t["q"], t["s"]), out=t["out"])
    if c["op"] == "moe8":
        r = m.w8a8_moe_grouped_gemm(t["x"], t["logits"], c["topk"], int8(t["q1"], t["s1"]), int8(t["q2"], t["s2"]))
        return r["out"], r["topk_idx"], r["topk_w"], r["expert_offsets"]
    w = m.PackedWeight(packed=t["packed"], s_w=t["s"], z=t["z"],
                       desc=m.WDesc(4, int(c["sym"]), c["group"], c["K"], c["N"], m.LAYOUT_VERSION), experts=c["E"])
    return m.w4a16_grouped_gemm(t["x"], t["offsets"], w, out=t["out"])


def run(state):
    if own:
        return own_run(state)
    return {"int8": plain_int8, "moe8": plain_moe8, "weight4": plain_weight4}[state["case"]["op"]](state)


# ------------------------------------------------------------------- work ---

def work(case):
    """What one pass cannot do without: inputs and the weights of experts that have rows read once, outputs written
    once, two operations for each product."""
    c = case
    E = c["E"]
    if c["op"] == "moe8":
        T, k, H, I = c["T"], c["topk"], c["H"], c["I"]
        g = torch.Generator().manual_seed(1)  # the experts that a batch of such tokens reaches
        logits = torch.randn(T, E, generator=g) + shares(E, c["skew"], 0, torch.Generator().manual_seed(E)).log().float()
        busy = logits.topk(k, dim=1).indices.unique().numel()
        b = T * H * 4 + T * E * 4 + T * k * 8 + 4 * (E + 1) + busy * (3 * H * I + 4 * (2 * I + H))
        return dict(bytes=b, flops=2 * T * k * 3 * H * I)
    R, K, N = c["rows"], c["K"], c["N"]
    busy = int((counts_of(c) > 0).sum())
    b = R * N * 2 + 4 * (E + 1)
    if c["op"] == "int8":
        b += R * (2 * K if c["bf16_in"] else K + 4) + busy * (K * N + 4 * N)
    else:
        b += R * 2 * K + busy * (K * N // 2 + K // c["group"] * N * (4 if c["sym"] else 5))
    return dict(bytes=b, flops=2 * R * K * N)


# ------------------------------------------------------------------ exact ---

def exact_codes(x):
    """Row codes from the definition: scale and quotient are fp32 numbers, each rounded once from its exact value (a
    value half as large as its row's largest has the quotient 63.5 in fp32, and 63.5 is a tie)."""
    x = x.double()
    s = (x.abs().max(dim=1).values / 127.0).float().double()
    d = s.clone()
    d[d == 0] = 1.0
    return torch.clamp(torch.round((x / d.unsqueeze(1)).float().double()), -127, 127), s


def exact_group(a, w_of, counts, N):
    """One fp64 product for each expert that has rows."""
    y = torch.empty(a.shape[0], N, dtype=torch.float64, device=a.device)
    at = 0
    for e, n in enumerate(counts):
        if n:
            y[at:at + n] = a[at:at + n] @ w_of(e)
        at += n
    return y


def exact(case, seed):
    c, t = case, prepare(case, seed)
    if c["op"] == "moe8":
        k, H, I, E = c["topk"], c["H"], c["I"], c["E"]
        logits = t["logits"].double()
        val, idx = torch.topk(logits, k, dim=1)
        weight = torch.exp(val - torch.logsumexp(logits, dim=1, keepdim=True))
        pair_expert = idx.reshape(-1).cpu()
        by_expert = [torch.nonzero(pair_expert == e).reshape(-1) for e in range(E)]
        n = [int(p.numel()) for p in by_expert]
        order = torch.cat(by_expert).to(DEV)
        q, s = exact_codes(t["x"])
        tok = order // k
        gu = exact_group(q[tok], lambda e: (t["q1"][e].double() * t["s1"][e].double().unsqueeze(1)).T, n, 2 * I)
        gu *= s[tok].unsqueeze(1)
        # the layer's own roundings between its two products: h in bf16, then its INT8 codes; expert rows in bf16
        h = (gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]).to(torch.bfloat16)
        q, s = exact_codes(h)
        y = exact_group(q, lambda e: (t["q2"][e].double() * t["s2"][e].double().unsqueeze(1)).T, n, H)
        y = (y * s.unsqueeze(1)).to(torch.bfloat16).double()
        out = torch.zeros(c["T"], H, dtype=torch.float64, device=DEV)
        out.index_add_(0, tok, y * weight.reshape(-1)[order].unsqueeze(1))
        return out, None, weight, None
    n = counts_of(c).tolist()
    R, N, K = c["rows"], c["N"], c["K"]
    out = torch.zeros(R + c["pad"], N, dtype=torch.float64, device=DEV)
    if c["op"] == "int8":
        q, s = exact_codes(t["x"][:R]) if c["bf16_in"] else (t["qx"][:R].double(), t["sx"][:R].double())
        out[:R] = exact_group(q, lambda e: (t["q"][e].double() * t["s"][e].double().unsqueeze(1)).T, n, N) * s.unsqueeze(1)
        return out

    def weight(e):
        # code of (k, n): block (n / 64, k / group), chunk (k % group) / 32, column n % 64, byte k % 16, nibble (k / 16) % 2
        k = torch.arange(K, device=DEV).unsqueeze(1)
        col = torch.arange(N, device=DEV).unsqueeze(0)
        grp, kk = k // c["group"], k % c["group"]
        at = ((col // 64) * (K // c["group"]) + grp) * (32 * c["group"]) + ((kk // 32) * 64 + col % 64) * 16 + kk % 16
        v = (t["packed"][e][at].to(torch.int32) >> (4 * ((kk % 32) // 16))) & 15
        if c["sym"]:
            v = torch.where(v > 7, v - 16, v)
        else:
            v = v - t["z"][e].to(torch.int32)[grp.squeeze(1)]
        # the operator's weights are bf16 numbers, rounded from the fp32 product of scale and code
        return (v.double() * t["s"][e].double()[grp.squeeze(1)]).float().to(torch.bfloat16).double()

    out[:R] = exact_group(t["x"][:R].double(), weight, n, N)
    return out
