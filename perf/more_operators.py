"""Workloads of the scored router and of the products with 4-bit weights: cases, inputs, plain
forms and exact values.

Four operators of the layer and of the dense parts around it:

  route    the router of models that balance their experts by a bias: softmax or sigmoid scores,
           a bias that takes part in the choice and not in the gates, groups of experts of which
           the best are kept, top-k, and the token-by-expert permutation
           (``moe_route_scored``);
  train    the same with its gradient: from the gates' gradients to the logits'
           (``moe_route_scored_backward``);
  linear4  y = x . W^T with W held in 4-bit codes, a scale and a zero point for each group of 32,
           64 or 128 along K, one power of two per output channel (``moe_i4_matmul``; the weights
           are quantised once by ``moe_i4_quantize``);
  experts4 the routed experts and the shared one from 4-bit blobs, gate, up and down products, one
           result for each pair of a token and an expert (``moe_i4_expert_ffn`` on blobs of
           ``moe_i4_pack``).

``own`` chooses between the plain form (elementary torch operations) and the library.

4-bit rows: weight = S * s * (code - z) with codes 0..15, the row's scale S (a power of two), the
group's scale s (an e4m3 number up to 448) and zero point z (0..15; 8 where the rows are held without
zero points).  The product has eight significant bits, so every weight is exact in bf16.
"""
import torch

own = False

F32, BF16 = 0, 1                      # element types of the C interface
TORCH = {F32: torch.float32, BF16: torch.bfloat16}
LARGEST = 2 * 8192 * 4096 * 8192      # operations of the largest product


def listed():
    return [
        # a decode step of 4 sequences: 256 experts in 8 groups, 4 kept, sigmoid scores with a balance bias
        dict(name="route_decode_4", op="route", T=4, E=256, k=8, score="sigmoid", bias=1, groups=8, keep=4, top=2,
             renorm=1, scale=2.5),
        # an 8,192-token prefill chunk through the same router
        dict(name="route_prefill_8k", op="route", T=8192, E=256, k=8, score="sigmoid", bias=1, groups=8, keep=4, top=2,
             renorm=1, scale=2.5),
        # a ragged chunk, softmax scores over an odd number of experts, biased, without groups
        dict(name="route_odd", op="route", T=1021, E=141, k=6, score="softmax", bias=1, groups=1, keep=1, top=1,
             renorm=0, scale=1.0),
        # a training step of a micro-batch: softmax over all experts, gates not renormalised, so every logit has a gradient
        dict(name="route_train_8k", op="train", T=8192, E=128, k=8, score="softmax", bias=0, groups=1, keep=1, top=1,
             renorm=0, scale=1.0),
        # a training step of the grouped sigmoid router on a short ragged batch
        dict(name="route_train_515", op="train", T=515, E=256, k=8, score="sigmoid", bias=1, groups=8, keep=4, top=2,
             renorm=1, scale=2.5),
        # one token through a square projection at hidden width 2048: the latency of a call
        dict(name="linear4_1", op="linear4", T=1, K=2048, N=2048, group=128, zero=0, x=BF16, y=BF16, pad=0),
        # a decode batch of 4 through an output head with an odd number of rows: the stream of codes
        dict(name="linear4_head_4", op="linear4", T=4, K=4096, N=100003, group=64, zero=1, x=BF16, y=F32, pad=0),
        # a short prompt, fp32 activations cut out of wider rows, a last group of 32 where groups have 128
        dict(name="linear4_ragged", op="linear4", T=77, K=1568, N=1037, group=128, zero=1, x=F32, y=F32, pad=8),
        # an 8,192-token prefill chunk through a wide projection: the matrix rate
        dict(name="linear4_prefill_8k", op="linear4", T=8192, K=4096, N=8192, group=128, zero=0, x=BF16, y=BF16, pad=0),
        # one token through 6 of 256 experts and the shared one, 4096 x 1536: the stream of codes
        dict(name="experts4_1", op="experts4", T=1, H=4096, I=1536, E=256, k=6, group=32, zero=0, shared=1),
        # a decode batch of 16 through 8 of 128 experts of 2048 x 768: most experts have a token or two
        dict(name="experts4_16", op="experts4", T=16, H=2048, I=768, E=128, k=8, group=128, zero=1, shared=0),
        # an 8,192-token prefill chunk through every expert of the layer
        dict(name="experts4_prefill_8k", op="experts4", T=8192, H=2048, I=768, E=128, k=8, group=64, zero=0, shared=0),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], uniform over the logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return min(hi // step * step, max(step, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["route", "train", "linear4", "linear4", "linear4", "experts4", "experts4", "experts4"])
    if op in ("route", "train"):
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        size = _log_int(rng, 4, 512 // groups)
        keep = rng.randint((groups + 1) // 2, groups)
        return dict(op=op, T=_log_int(rng, 1, 8192), E=groups * size, k=rng.randint(1, min(16, keep * size)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.choice([0, 1]), groups=groups, keep=keep,
                    top=rng.choice([1, 2]), renorm=rng.choice([0, 1]), scale=rng.choice([1.0, 2.5]))
    group, zero = rng.choice([32, 64, 128]), rng.choice([0, 1])
    if op == "linear4":
        while True:
            T, K, N = _log_int(rng, 1, 8192), _log_int(rng, 256, 12288, 32), _log_int(rng, 128, 100003)
            if 2 * T * K * N <= LARGEST:
                break
        return dict(op=op, T=T, K=K, N=N, group=group, zero=zero, x=rng.choice([BF16, BF16, F32]),
                    y=rng.choice([BF16, F32]), pad=rng.choice([0, 0, 8, 63]))
    while True:
        T, E = _log_int(rng, 1, 8192), _log_int(rng, 8, 256)
        H, I, k = _log_int(rng, 256, 4096, 64), _log_int(rng, 128, 2048, 32), rng.randint(1, 8)
        if 6 * T * k * H * I <= LARGEST and E * H * I <= 128 * 2048 * 2048:
            break
    return dict(op=op, T=T, H=H, I=I, E=E, k=k, group=group, zero=zero, shared=rng.choice([0, 1]))


def work(case):
    T, op = case["T"], case["op"]
    if op in ("route", "train"):
        # logits and bias in; ids, gates, permutation and its inverse, counts and offsets out
        E, k = case["E"], case["k"]
        n = 4 * T * E + 4 * E * case["bias"] + 16 * T * k + 8 * E + 4
        if op == "train":                    # the gates' gradients in, the logits' out
            n += 4 * T * k + 4 * T * E
        return {"bytes": n, "flops": 4 * T * E}
    G = case["group"]
    if op == "linear4":
        K, N = case["K"], case["N"]
        xb, yb = (4 if case["x"] == F32 else 2), (4 if case["y"] == F32 else 2)
        return {"bytes": T * K * xb + N * (K // 2 + 2 * -(-K // G) + 1) + T * N * yb, "flops": 2 * T * N * K}
    H, I, E, k = case["H"], case["I"], case["E"], case["k"]
    used = min(E, T * k) if T == 1 else E * (1 - (1 - k / E) ** T)       # experts that some token uses
    blob = 2 * I * (H // 2 + 2 * -(-H // G) + 1) + H * (I // 2 + 2 * -(-I // G) + 1)
    rows = T * k + T * case["shared"]
    return {"bytes": int((used + case["shared"]) * blob) + 2 * T * H + 2 * rows * H + 4 * T * k,
            "flops": 6 * rows * H * I}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _route_inputs(case, seed):
    """Logits of unit size with a few popular experts, a bias as balancing leaves it, and gradients."""
    gen = _generator(seed)
    T, E, k = case["T"], case["E"], case["k"]
    liked = torch.randn((1, E), generator=gen, device="cuda")
    logits = 1.5 * torch.randn((T, E), generator=gen, device="cuda") + 0.5 * liked
    bias = 0.1 * torch.randn(E, generator=gen, device="cuda") if case["bias"] else None
    dw = 0.1 * torch.randn((T, k), generator=gen, device="cuda") if case["op"] == "train" else None
    return logits, bias, dw


def _linear_inputs(case, seed):
    """x as a view of rows that may be wider than K, with a few channels ten times as large as the
    rest (as activations have), and W."""
    gen = _generator(seed)
    T, K, N = case["T"], case["K"], case["N"]
    x = torch.randn((T, K + case["pad"]), generator=gen, device="cuda")
    loud = torch.randint(0, K, (max(1, K // 512),), generator=gen, device="cuda")
    x[:, loud] *= 10.0
    w = (torch.randn((N, K), generator=gen, device="cuda") * 0.02).to(torch.bfloat16)
    return x.to(TORCH[case["x"]])[:, :K], w


def _expert_inputs(case, seed):
    """Tokens, their experts (some more popular than others) grouped by expert, and the generator
    that draws the weights expert by expert."""
    gen = _generator(seed)
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    x = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    liked = 0.5 * torch.randn((1, E), generator=gen, device="cuda")
    ids = (torch.randn((T, E), generator=gen, device="cuda") + liked).sort(1, descending=True).indices[:, :k]
    flat = ids.reshape(-1)
    perm = flat.sort(stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = (flat[:, None] == torch.arange(E, device="cuda")).sum(0).cumsum(0)
    return x, ids, perm, offsets, gen


def _expert_weights(case, gen):
    H, I = case["H"], case["I"]
    return [(torch.randn(s, generator=gen, device="cuda") * 0.02).to(torch.bfloat16) for s in ((I, H), (I, H), (H, I))]


class _Handle:
    """A library context, freed with the state that holds it."""

    def __init__(self, B, H=64, I=32, E=1, k=1, shared=0):
        self.B, self.cfg = B, B.make_config(H, I, E, k, shared, w_dtype=B.MOE_W_BF16)
        self.ctx = B.moe_create(self.cfg)

    def __del__(self):
        self.B.moe_destroy(self.ctx)


def _stream():
    return torch.cuda.current_stream()


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def _whole(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    st = {"case": case}
    T, op = case["T"], case["op"]
    if own:
        from expert_cached_moe_amd import binding as B
        st["B"] = B
    if op in ("route", "train"):
        st["logits"], st["bias"], st["dw"] = _route_inputs(case, seed)
        if not own:
            return st
        E, k = case["E"], case["k"]
        h = st["h"] = _Handle(B, E=E, k=k)
        st["rule"] = B.make_route_rule(B.MOE_SCORE_SIGMOID if case["score"] == "sigmoid" else B.MOE_SCORE_SOFTMAX,
                                       case["groups"], case["keep"], case["top"], case["renorm"], case["scale"])
        st["ids"], st["w"] = _whole(T, k), torch.empty((T, k), device="cuda")
        st["counts"], st["offsets"], st["perm"], st["inv"] = _whole(E), _whole(E + 1), _whole(T * k), _whole(T * k)
        st["work"] = _bytes(B.moe_workspace_bytes(h.cfg, T))
        if op == "train":
            st["dlogits"] = torch.empty((T, E), device="cuda")
        return st
    G, zero = case["group"], case["zero"]
    if op == "linear4":
        x, w = _linear_inputs(case, seed)
        st["x"] = x
        if not own:
            st["w"] = _quantise(w, G, zero)
            return st
        N, K = w.shape
        h = st["h"] = _Handle(B)
        st["codes"], st["scale"] = _bytes(N * K // 2), _bytes(N)
        st["words"] = torch.empty((N, -(-K // G)), dtype=torch.int16, device="cuda")
        B.moe_i4_quantize(h.ctx, w, BF16, K, N, K, G, zero, st["codes"], st["words"], st["scale"], _stream())
        st["y"] = torch.empty((T, N), dtype=TORCH[case["y"]], device="cuda")
        st["work"] = _bytes(B.moe_i4_workspace_bytes(T, N, K))
        return st
    x, ids, perm, offsets, gen = _expert_inputs(case, seed)
    H, I, E, k, shared = case["H"], case["I"], case["E"], case["k"], case["shared"]
    on_host = offsets.tolist()
    used = [e for e in range(E) if on_host[e + 1] > on_host[e]]
    st["x"], st["used"] = x, used
    if not own:
        st["perm"], st["on_host"] = perm, on_host
        st["w"] = [[_quantise(w, G, zero) for w in _expert_weights(case, gen)] for _ in range(len(used) + shared)]
        return st
    h = st["h"] = _Handle(B, H, I, E, k, shared)
    size = B.moe_i4_blob_bytes(h.cfg, G)
    st["pool"] = _bytes((len(used) + shared) * size)
    blob = torch.zeros(B.moe_expert_bytes(h.cfg), dtype=torch.uint8, device="cuda").view(torch.bfloat16)
    down = -(-4 * I * H // 256) * 128                                  # where the down projection begins
    for i in range(len(used) + shared):
        wg, wu, wd = _expert_weights(case, gen)
        blob[:2 * I * H] = torch.stack([wg.view(I // 16, 16, H), wu.view(I // 16, 16, H)], 1).reshape(-1)
        blob[down:down + H * I] = wd.reshape(-1)
        B.moe_i4_pack(h.ctx, blob, G, zero, st["pool"][i * size:], _stream())
    st["shared"] = st["pool"][len(used) * size:] if shared else None
    st["perm"], st["offsets"] = perm.to(torch.int32), offsets.to(torch.int32)
    st["o"] = torch.empty((T * k + T * shared, H), dtype=torch.bfloat16, device="cuda")
    st["work"] = _bytes(B.moe_i4_expert_workspace_bytes(h.cfg, T))
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    if not own:
        return _plain_pass(st)
    case, B, ctx, s = st["case"], st["B"], st["h"].ctx, _stream()
    T, op = case["T"], case["op"]
    if op in ("route", "train"):
        B.moe_route_scored(ctx, st["logits"], st["bias"], T, st["rule"], st["ids"], st["w"], st["counts"], st["offsets"],
                           st["perm"], st["inv"], st["work"], s)
        out = {n: st[n] for n in ("ids", "w", "counts", "offsets", "perm", "inv")}
        if op == "train":
            B.moe_route_scored_backward(ctx, st["logits"], T, st["rule"], st["ids"], st["dw"], st["dlogits"], s)
            out["dlogits"] = st["dlogits"]
        return out
    if op == "linear4":
        x, N, K = st["x"], case["N"], case["K"]
        B.moe_i4_matmul(ctx, x, case["x"], x.stride(0), T, st["codes"], st["words"], st["scale"], N, K, case["group"],
                        st["y"], case["y"], N, st["work"], s)
        return st["y"]
    used = st["used"]
    B.moe_i4_expert_ffn(ctx, st["x"], T, st["offsets"], st["perm"], st["pool"], used, list(range(len(used))), len(used),
                        st["shared"], case["shared"], case["group"], st["o"], st["work"], s)
    return st["o"]


# ---------------------------------------------------------------- plain form

def _quantise(w, G, zero):
    """(two codes a byte, group scales, zero points, row scales) of rows: a row's scale is the least power
    of two that leaves its group scales at 448 or less; group scales are e4m3 numbers, to nearest even, or
    up where there are zero points, so that the range fits 15 steps; codes from quotients in 64 bits, half
    to even."""
    N, K = w.shape
    Kg = -(-K // G)
    v = torch.zeros((N, Kg * G), dtype=torch.float64, device=w.device)
    v[:, :K] = w
    v = v.view(N, Kg, G)
    if zero:
        lo, hi, steps = v.amin(2).clamp(max=0), v.amax(2).clamp(min=0), 15.0
        span = hi - lo
    else:
        span, steps = v.abs().amax(2), 7.0
    t = span / steps
    m, e = torch.frexp(t.amax(1) / 448.0)
    S = torch.exp2((e - (m == 0.5).int()).double())
    S = torch.where((m > 0) & (S >= 2.0 ** -100), S, 0.0)
    d = S[:, None]
    u = torch.where(d > 0, t / torch.where(d > 0, d, 1.0), 0.0)
    e = torch.frexp(u).exponent.clamp(min=-5)                          # 2^(e - 1) <= u < 2^e, or subnormal
    unit = torch.exp2(e.double() - 4)
    s = ((u / unit).ceil() if zero else (u / unit).round()) * unit
    s = s.clamp(max=448.0)
    d = (d * s)[:, :, None]
    safe = torch.where(d > 0, d, 1.0)
    z = (-lo[:, :, None] / safe).round().clamp(0, 15) if zero else torch.full_like(d, 8.0)
    z = torch.where(d > 0, z, 8.0)
    c = torch.where(d > 0, ((v / safe).round() + z).clamp(0, 15), 8.0)
    c = c.view(N, Kg * G)[:, :K].to(torch.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4), s.float(), z[:, :, 0].float(), S.float()


def _weights(q, G):
    """The numbers that rows of codes stand for."""
    codes, s, z, S = q
    N, K = codes.shape[0], 2 * codes.shape[1]
    c = torch.stack([codes & 15, codes >> 4], 2).view(N, K).float()
    spread = torch.arange(K, device=c.device) // G
    return (c - z[:, spread]) * s[:, spread] * S[:, None]


def _choice(case, logits, bias):
    """Scores in 64 bits (the choice is decided on them), and the ids that they choose."""
    x = logits.double()
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        s = e / e.sum(1, keepdim=True)
    T, E = x.shape
    rank = s + bias.double() if bias is not None else x
    value = s + bias.double() if bias is not None else s
    groups = case["groups"]
    if groups > 1:
        best = value.view(T, groups, E // groups).sort(2, descending=True).values[:, :, :case["top"]].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :case["keep"]]
        out = torch.ones((T, groups), dtype=torch.bool, device=x.device)
        out[torch.arange(T, device=x.device)[:, None], kept] = False
        rank = torch.where(out[:, torch.arange(E, device=x.device) // (E // groups)], -float("inf"), rank)
    return s, rank.sort(dim=1, descending=True, stable=True).indices[:, :case["k"]]


def _plain_route(st, case):
    s, ids = _choice(case, st["logits"], st["bias"])
    T, E = s.shape
    at = torch.arange(T, device=s.device)[:, None]
    picked = s[at, ids]
    total = picked.sum(1, keepdim=True)
    w = picked / total if case["renorm"] else picked
    flat = ids.reshape(-1)
    perm = flat.sort(stable=True).indices
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(perm.numel(), device=perm.device)
    counts = torch.zeros(E, dtype=torch.int64, device=s.device)
    counts.index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=s.device)
    offsets[1:] = counts.cumsum(0)
    whole = torch.int32
    out = {"ids": ids.to(whole), "w": (w * case["scale"]).float(), "counts": counts.to(whole),
           "offsets": offsets.to(whole), "perm": perm.to(whole), "inv": inv.to(whole)}
    if case["op"] == "train":
        dw = st["dw"].double() * case["scale"]
        if case["renorm"]:
            ds = (dw - (dw * w).sum(1, keepdim=True)) / total
        else:
            ds = dw
        full = torch.zeros_like(s)
        full[at, ids] = ds
        if case["score"] == "sigmoid":
            d = full * s * (1 - s)
        else:
            d = s * (full - (ds * picked).sum(1, keepdim=True))
        out["dlogits"] = d.float()
    return out


def _plain_pass(st):
    case = st["case"]
    if case["op"] in ("route", "train"):
        return _plain_route(st, case)
    G = case["group"]
    if case["op"] == "linear4":
        return (st["x"].float() @ _weights(st["w"], G).T).to(TORCH[case["y"]])
    T, H, k = case["T"], case["H"], case["k"]
    o = torch.empty((T * k + T * case["shared"], H), dtype=torch.bfloat16, device="cuda")

    def block(x, w):
        wg, wu, wd = (_weights(q, G) for q in w)
        g, u = x @ wg.T, x @ wu.T
        return ((g / (1 + torch.exp(-g)) * u) @ wd.T).to(torch.bfloat16)

    x = st["x"].float()
    for e, w in zip(st["used"], st["w"]):
        pairs = st["perm"][st["on_host"][e]:st["on_host"][e + 1]]
        o[pairs] = block(x[pairs // k], w)
    if case["shared"]:
        o[T * k:] = block(x, st["w"][-1])
    return o


# ---------------------------------------------------------------- exact values

def _nearest_weights(w, G, zero):
    """W as its 4-bit form holds it, from the form's definition, group by group."""
    w = w.to(torch.float64)
    N, K = w.shape
    out = torch.empty_like(w)
    parts = [w[:, a:a + G] for a in range(0, K, G)]
    top = [torch.max(p.max(1).values, torch.zeros(N, dtype=w.dtype, device=w.device)) for p in parts]
    low = [torch.min(p.min(1).values, torch.zeros(N, dtype=w.dtype, device=w.device)) for p in parts]
    if zero:
        width, n = [a - b for a, b in zip(top, low)], 15
    else:
        width, n = [torch.max(a, -b) for a, b in zip(top, low)], 7
    widest = torch.stack(width).max(0).values
    row = torch.pow(2.0, torch.ceil(torch.log2(widest.div(n) / 448)))
    row = torch.where((widest > 0) & (row >= 2.0 ** -100), row, 0.0)
    for i, p in enumerate(parts):
        t = torch.where(row > 0, width[i] / n / torch.where(row > 0, row, 1.0), 0.0)
        quantum = torch.ldexp(torch.ones_like(t), torch.floor(torch.log2(t.clamp(min=2.0 ** -6))).to(torch.int32) - 3)
        t = (torch.ceil(t / quantum) if zero else torch.round(t / quantum)).mul(quantum).clamp(max=448)
        step = (row * t)[:, None]
        live = step > 0
        div = torch.where(live, step, 1.0)
        if zero:
            origin = torch.round(-low[i][:, None] / div).clamp(0, 15)
            code = (torch.round(p / div) + origin).clamp(0, 15) - origin
        else:
            code = torch.round(p / div).clamp(-8, 7)
        out[:, i * G:i * G + p.shape[1]] = torch.where(live, code * step, 0.0)
    return out


def _exact_route(case, seed):
    logits, bias, dw = _route_inputs(case, seed)
    z = logits.to(torch.float64)
    T, E = z.shape
    p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, 1)
    by = z if bias is None else p + bias.to(torch.float64)
    mark = p if bias is None else by
    allowed = torch.ones((T, E), dtype=torch.bool, device=z.device)
    if case["groups"] > 1:
        n = E // case["groups"]
        score = torch.stack([mark[:, g * n:(g + 1) * n].topk(min(case["top"], n), 1).values.sum(1)
                             for g in range(case["groups"])], 1)
        # a group stays if fewer than `keep` come before it (larger, or equal with a lower index)
        lower = torch.arange(case["groups"], device=z.device)
        before = (score[:, None, :] > score[:, :, None]) | ((score[:, None, :] == score[:, :, None]) &
                                                           (lower[None, None, :] < lower[None, :, None]))
        allowed = (before.sum(2) < case["keep"]).repeat_interleave(n, 1)
    by = by.masked_fill(~allowed, -float("inf"))
    cols, left = [], by.clone()
    number = torch.arange(E, device=z.device)
    for _ in range(case["k"]):
        best = left.max(1, keepdim=True).values
        pick = torch.where(left == best, number, E).min(1, keepdim=True).values
        cols.append(pick)
        left.scatter_(1, pick, -float("inf"))
    ids = torch.cat(cols, 1)
    chosen = p.gather(1, ids)
    norm = chosen.sum(1, keepdim=True) if case["renorm"] else torch.ones((T, 1), dtype=p.dtype, device=p.device)
    gates = case["scale"] * chosen / norm
    order = torch.argsort(ids.reshape(-1) * (T * case["k"]) + torch.arange(T * case["k"], device=z.device))
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    ends = torch.cat([torch.zeros(1, dtype=counts.dtype, device=z.device), counts.cumsum(0)])
    out = {"ids": ids, "w": gates, "counts": counts, "offsets": ends, "perm": order, "inv": torch.argsort(order)}
    if case["op"] == "train":
        # d gates / d scores, then the scores' own derivative
        g = dw.to(torch.float64)
        back = case["scale"] / norm * g
        if case["renorm"]:
            back = back - (g * gates).sum(1, keepdim=True) / norm
        if case["score"] == "sigmoid":
            d = torch.zeros_like(p).scatter_(1, ids, back * chosen * (1 - chosen))
        else:
            d = -p * (back * chosen).sum(1, keepdim=True)
            d.scatter_add_(1, ids, chosen * back)
        out["dlogits"] = d
    return {n: v if v.is_floating_point() else v.to(torch.int32) for n, v in out.items()}


def exact(case, seed):
    """The operators' definitions in 64 bits (codes and scales of the 4-bit weights are part of the
    definition, as is the choice of experts)."""
    if case["op"] in ("route", "train"):
        return _exact_route(case, seed)
    G, zero = case["group"], case["zero"]
    if case["op"] == "linear4":
        x, w = _linear_inputs(case, seed)
        return torch.mm(x.to(torch.float64), _nearest_weights(w, G, zero).t())
    x, ids, _, _, gen = _expert_inputs(case, seed)
    T, H, k = case["T"], case["H"], case["k"]
    x = x.to(torch.float64)
    out = torch.empty((T * k + T * case["shared"], H), dtype=torch.float64, device="cuda")

    def expert(rows):
        gate, up, down = (_nearest_weights(w, G, zero) for w in _expert_weights(case, gen))
        a = torch.mm(rows, gate.t())
        return torch.mm(a * torch.sigmoid(a) * torch.mm(rows, up.t()), down.t())

    flat = ids.reshape(-1)
    for e in torch.unique(flat).tolist():
        at = torch.nonzero(flat == e)[:, 0]
        out[at] = expert(x[torch.div(at, k, rounding_mode="floor")])
    if case["shared"]:
        out[T * k:] = expert(x)
    return out
