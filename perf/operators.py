"""Workloads of the dense feed-forward operators: cases, inputs, plain forms and exact values.

Three operators stand beside the MoE layer, for the dense parts of a model that holds it:

  linear  y = x . W^T with W held in 8-bit integers, one scale per output channel, and x
          quantised to 8-bit integers with one scale per token on the way
          (``moe_i8_matmul``; the weights are quantised once by ``moe_i8_quantize``);
  ffn     the gated feed-forward block y = Wd (silu(Wg x) * (Wu x)) on an expert blob, for
          serving, and for training with its backward pass (``moe_dense_ffn``,
          ``moe_dense_ffn_backward``);
  ffn8    the same block served from 8-bit weights, both products in integers
          (``moe_i8_pack``, ``moe_i8_ffn``).

``own`` chooses between the plain form (elementary torch operations) and the library.
Eight-bit quantisation of a row: s = fp32(max|row| / 127), code = round_half_even(row / s).
A blob's gate and up rows are interleaved in blocks of 16: gate 0-15, up 0-15, gate 16-31, ...
"""
import torch

own = False

F32, BF16 = 0, 1                      # element types of the C interface
TORCH = {F32: torch.float32, BF16: torch.bfloat16}
LARGEST = 8192 * 4096 * 12288         # tokens * width * inner width of the largest block


def listed():
    return [
        # one token through a square projection at hidden width 2048: the latency of a call
        dict(name="linear_decode_1", op="linear", T=1, K=2048, N=2048, x=BF16, y=BF16, pad=0),
        # a decode batch of 8 through an output head with an odd number of rows: the weight stream
        dict(name="linear_head_8", op="linear", T=8, K=4096, N=100003, x=BF16, y=F32, pad=0),
        # an 8,192-token prefill chunk through a wide projection: the matrix rate
        dict(name="linear_prefill_8k", op="linear", T=8192, K=4096, N=8192, x=BF16, y=BF16, pad=0),
        # a short prompt, fp32 activations cut out of wider rows, no size a multiple of a tile
        dict(name="linear_ragged", op="linear", T=777, K=1552, N=2051, x=F32, y=F32, pad=48),
        # a training step of a block with the sizes of the 2048 x 768 layer's expert
        dict(name="train_2048x768", op="train", T=4096, H=2048, I=768, w=BF16),
        # a training step of a wide dense block on a full chunk: the largest case
        dict(name="train_4096x12288", op="train", T=8192, H=4096, I=12288, w=BF16),
        # a training step in fp32, ragged token count
        dict(name="train_fp32", op="train", T=515, H=1024, I=1120, w=F32),
        # a training step on the few tokens of a small micro-batch: the weights dominate
        dict(name="train_few_tokens", op="train", T=37, H=4096, I=1536, w=BF16),
        # one token through a wide dense block: the weight stream in bf16
        dict(name="serve_1", op="serve", T=1, H=4096, I=12288, w=BF16),
        # one token through a block of the 4096 x 1536 layer's size, 8-bit weights
        dict(name="serve8_1", op="ffn8", T=1, H=4096, I=1536),
        # a decode batch of 8 through the wide block, 8-bit weights
        dict(name="serve8_8", op="ffn8", T=8, H=4096, I=12288),
        # a prefill chunk through the wide block, 8-bit weights
        dict(name="serve8_prefill_8k", op="ffn8", T=8192, H=4096, I=12288),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], uniform over the logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return min(hi // step * step, max(step, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["linear", "linear", "train", "train", "serve", "ffn8", "ffn8"])
    if op == "linear":
        while True:
            T, K, N = _log_int(rng, 1, 8192), _log_int(rng, 256, 12288, 16), _log_int(rng, 128, 100003)
            if T * K * N <= 8192 * 4096 * 8192:
                break
        return dict(op=op, T=T, K=K, N=N, x=rng.choice([BF16, BF16, F32]), y=rng.choice([BF16, F32]),
                    pad=rng.choice([0, 0, 16, 64]))
    w = F32 if op in ("train", "serve") and rng.random() < 0.25 else BF16
    while True:
        T = _log_int(rng, 1, 1024 if w == F32 else 8192)
        H = _log_int(rng, 256, 2048 if w == F32 else 8192, 64)
        I = _log_int(rng, 128, 4096 if w == F32 else 16384, 32)
        if T * H * I <= LARGEST:
            break
    c = dict(op=op, T=T, H=H, I=I)
    if op != "ffn8":
        c["w"] = w
    return c


def work(case):
    T = case["T"]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        xb, yb = (4 if case["x"] == F32 else 2), (4 if case["y"] == F32 else 2)
        return {"bytes": T * K * xb + N * K + 4 * N + T * N * yb, "flops": 2 * T * N * K}
    H, I = case["H"], case["I"]
    if case["op"] == "ffn8":                     # x, codes, scales, y
        return {"bytes": 2 * T * H * 2 + 3 * H * I + 4 * (2 * I + H), "flops": 6 * T * H * I}
    b = 4 if case["w"] == F32 else 2
    if case["op"] == "serve":
        return {"bytes": b * (2 * T * H + 3 * H * I), "flops": 6 * T * H * I}
    # x, dy in; y, dx out; weights in, their gradient out
    return {"bytes": b * (4 * T * H + 6 * H * I), "flops": 18 * T * H * I}


# ---------------------------------------------------------------- inputs

def _randn(gen, shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _linear_inputs(case, seed):
    """x as a view of rows that may be wider than K, with a few channels ten times as large as
    the rest (as activations have), and W's codes and scales."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, K, N = case["T"], case["K"], case["N"]
    x = torch.randn((T, K + case["pad"]), generator=gen, device="cuda")
    loud = torch.randint(0, K, (max(1, K // 512),), generator=gen, device="cuda")
    x[:, loud] *= 10.0
    x = x.to(TORCH[case["x"]])[:, :K]
    w = _randn(gen, (N, K), 0.02, torch.bfloat16)
    return x, w


def _ffn_inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, H, I = case["T"], case["H"], case["I"]
    dt = TORCH[case.get("w", BF16)]
    x = _randn(gen, (T, H), 1.0, dt)
    dy = _randn(gen, (T, H), 0.01, dt) if case["op"] == "train" else None
    wg, wu, wd = (_randn(gen, (I, H), 0.02, dt), _randn(gen, (I, H), 0.02, dt), _randn(gen, (H, I), 0.02, dt))
    return x, dy, wg, wu, wd


def _interleave(g, u):
    """Gate and up rows [I][H] to the blob's [2I][H]."""
    I, H = g.shape
    return torch.stack([g.view(I // 16, 16, H), u.view(I // 16, 16, H)], 1).reshape(2 * I, H)


class _Handle:
    """A library context, freed with the state that holds it."""

    def __init__(self, B, H, I, w_dtype):
        self.B, self.cfg = B, B.make_config(H, I, 1, 1, w_dtype=w_dtype)
        self.ctx = B.moe_create(self.cfg)

    def __del__(self):
        self.B.moe_destroy(self.ctx)


def prepare(case, seed):
    T = case["T"]
    st = {"case": case}
    if case["op"] == "linear":
        x, w = _linear_inputs(case, seed)
        N, K = w.shape
        st["x"] = x
        if not own:
            st["wq"], st["ws"] = _quantise(w)
            return st
        from expert_cached_moe_amd import binding as B
        h = st["h"] = _Handle(B, 64, 32, B.MOE_W_BF16)
        st["wq"] = torch.empty((N, K), dtype=torch.int8, device="cuda")
        st["ws"] = torch.empty(N, dtype=torch.float32, device="cuda")
        B.moe_i8_quantize(h.ctx, w, BF16, K, N, K, st["wq"], st["ws"])
        st["y"] = torch.empty((T, N), dtype=TORCH[case["y"]], device="cuda")
        st["work"] = torch.empty(B.moe_i8_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
        return st
    x, dy, wg, wu, wd = _ffn_inputs(case, seed)
    H, I = case["H"], case["I"]
    st["x"], st["dy"] = x, dy
    if not own:
        if case["op"] == "ffn8":
            for name, w in (("g", wg), ("u", wu), ("d", wd)):
                st["q" + name], st["s" + name] = _quantise(w)
        else:
            st["wg"], st["wu"], st["wd"] = wg, wu, wd
        return st
    from expert_cached_moe_amd import binding as B
    w_dtype = case.get("w", BF16)
    h = st["h"] = _Handle(B, H, I, w_dtype)
    nb = B.moe_expert_bytes(h.cfg)

    def blob_views(blob):
        flat = blob.view(TORCH[w_dtype])
        d0 = (2 * I * H * flat.element_size() + 255) // 256 * 256 // flat.element_size()
        return flat[: 2 * I * H].view(2 * I, H), flat[d0: d0 + H * I].view(H, I)

    blob = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    gu, d = blob_views(blob)
    gu.copy_(_interleave(wg, wu))
    d.copy_(wd)
    st["y"] = torch.empty_like(x)
    st["work"] = torch.empty(B.moe_dense_workspace_bytes(h.cfg, T), dtype=torch.uint8, device="cuda")
    if case["op"] == "ffn8":
        st["blob8"] = torch.empty(B.moe_i8_blob_bytes(h.cfg), dtype=torch.uint8, device="cuda")
        B.moe_i8_pack(h.ctx, blob, st["blob8"])
        return st
    st["blob"] = blob
    if case["op"] == "train":
        st["save"] = torch.empty(B.moe_dense_save_bytes(h.cfg, T), dtype=torch.uint8, device="cuda")
        st["dx"] = torch.empty_like(x)
        st["dblob"] = torch.empty(nb, dtype=torch.uint8, device="cuda")
        st["dgu"], st["dd"] = blob_views(st["dblob"])
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return _own_pass(st) if own else _plain_pass(st)


def _own_pass(st):
    from expert_cached_moe_amd import binding as B
    case, T, s = st["case"], st["case"]["T"], torch.cuda.current_stream()
    ctx = st["h"].ctx
    if case["op"] == "linear":
        B.moe_i8_matmul(ctx, st["x"], case["x"], st["x"].stride(0), None, T, st["wq"], st["ws"], case["N"], case["K"],
                        st["y"], case["y"], case["N"], st["work"], s)
        return st["y"]
    if case["op"] == "ffn8":
        B.moe_i8_ffn(ctx, st["x"], T, st["blob8"], st["y"], st["work"], s)
        return st["y"]
    if case["op"] == "serve":
        B.moe_dense_ffn(ctx, st["x"], T, st["blob"], None, st["y"], st["work"], s)
        return st["y"]
    B.moe_dense_ffn(ctx, st["x"], T, st["blob"], st["save"], st["y"], st["work"], s)
    B.moe_dense_ffn_backward(ctx, st["dy"], st["x"], T, st["blob"], st["save"], st["dx"], st["dblob"], st["work"], s)
    return {"y": st["y"], "dx": st["dx"], "dgu": st["dgu"], "dd": st["dd"]}


def _quantise(x):
    """Codes (int8) and scales (fp32) of the rows of x.  The quotients are taken in 64 bits: a
    code next to a border must not depend on how a division rounds."""
    s = (x.float().abs().amax(-1).double() / 127).float()
    q = torch.round(x.double() / torch.where(s > 0, s, torch.ones_like(s)).double()[..., None])
    return q.to(torch.int8), s


def _product8(q, s, wq, ws):
    return (q.float() @ wq.float().T) * s[:, None] * ws


def _plain_pass(st):
    case = st["case"]
    if case["op"] == "linear":
        q, s = _quantise(st["x"])
        return _product8(q, s, st["wq"], st["ws"]).to(TORCH[case["y"]])
    if case["op"] == "ffn8":
        q, s = _quantise(st["x"])
        g = _product8(q, s, st["qg"], st["sg"])
        u = _product8(q, s, st["qu"], st["su"])
        q, s = _quantise(g / (1 + torch.exp(-g)) * u)
        return _product8(q, s, st["qd"], st["sd"]).to(torch.bfloat16)
    x, wg, wu, wd = (st[k].float() for k in ("x", "wg", "wu", "wd"))
    dt = st["x"].dtype
    g, u = x @ wg.T, x @ wu.T
    sig = 1 / (1 + torch.exp(-g))
    a = g * sig
    h = a * u
    y = (h @ wd.T).to(dt)
    if case["op"] == "serve":
        return y
    dy = st["dy"].float()
    dh = dy @ wd
    dd = dy.T @ h
    du = dh * a
    dg = dh * u * (sig * (1 + g * (1 - sig)))
    dx = dg @ wg + du @ wu
    dgu = _interleave((dg.T @ x).to(dt), (du.T @ x).to(dt))
    return {"y": y, "dx": dx.to(dt), "dgu": dgu, "dd": dd.to(dt)}


# ---------------------------------------------------------------- exact values

def exact(case, seed):
    """The operators' definitions in 64 bits (codes and scales of the 8-bit operators are part
    of the definition: scales are fp32 numbers, codes whole ones)."""
    def codes(m):
        m = m.to(torch.float64)
        top = m.abs().max(dim=1, keepdim=True).values
        step = torch.div(top, 127.0).to(torch.float32).to(torch.float64)
        return torch.where(step > 0, torch.round(m / torch.where(step > 0, step, 1.0)), 0.0), step

    def mul8(a, b):
        (ca, sa), (cb, sb) = a, b
        return torch.mm(ca, cb.t().contiguous()) * (sa * sb.t())

    if case["op"] == "linear":
        x, w = _linear_inputs(case, seed)
        return mul8(codes(x), codes(w))
    x, dy, wg, wu, wd = _ffn_inputs(case, seed)
    if case["op"] == "ffn8":
        cx = codes(x)
        gate, up = mul8(cx, codes(wg)), mul8(cx, codes(wu))
        return mul8(codes(gate * torch.sigmoid(gate) * up), codes(wd))
    x, wg, wu, wd = (t.to(torch.float64) for t in (x, wg, wu, wd))
    gate, up = torch.mm(x, wg.t()), torch.mm(x, wu.t())
    s = torch.sigmoid(gate)
    hidden = gate * s * up
    y = torch.mm(hidden, wd.t())
    if case["op"] == "serve":
        return y
    dy = dy.to(torch.float64)
    dhid = torch.mm(dy, wd)
    d_up = dhid * gate * s
    d_gate = dhid * up * (s + gate * s * (1 - s))
    I, H = wg.shape
    both = torch.empty((I // 16, 2, 16, H), dtype=torch.float64, device=x.device)
    both[:, 0] = torch.mm(d_gate.t(), x).view(I // 16, 16, H)
    both[:, 1] = torch.mm(d_up.t(), x).view(I // 16, 16, H)
    return {"y": y, "dx": torch.mm(d_gate, wg) + torch.mm(d_up, wu), "dgu": both.view(2 * I, H),
            "dd": torch.mm(dy.t(), hidden)}
