"""What is measured of the 8-bit operators: their cases, inputs and plain forms.

The 8-bit (e4m3) form of one sparse-MoE layer, a scale for each 128 values of a token and for each 128 x 128 block of a
weight:
  norm      moe_norm_quantize      r = x + residual; y = RMSNorm(r) * weight; y in 8 bits (and in bf16, for the router)
  quantize  moe_block_quantize     tokens in 8 bits
  linear    moe_block_linear       y = x W^T + bias, tokens and weights in 8 bits
  ffn       moe_block_expert_ffn   the routed experts, their products grouped by expert:
                                 y_t = sum_j w_tj W_down,e h_tj with h_tj = SiLU(W_gate,e x_t) * (W_up,e x_t) in 8 bits

With `own` false, run() computes them with elementary torch operations; with `own` true it calls the library.
"""

import math

import torch

own = False

DEV = "cuda"
BLOCK = 128                       # values that share a scale
TOP = 448.0                       # the largest e4m3 value
SMALL = 2.0 ** -126               # the smallest scale
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases

def _norm(name, T, H, stream, offset, hidden):
    return {"name": name, "op": "norm", "T": T, "H": H, "stream": stream, "offset": offset, "hidden": hidden}


def _quantize(name, T, K):
    return {"name": name, "op": "quantize", "T": T, "K": K}


def _linear(name, T, N, K, bias):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "bias": bias}


def _ffn(name, T, H, I, E, k, skew):
    return {"name": name, "op": "ffn", "T": T, "H": H, "I": I, "E": E, "k": k, "skew": skew}


def listed():
    return [
        # one token of a decode loop in front of a layer: latency
        _norm("norm_t1_2048", 1, 2048, "bf16", 0.0, True),
        # a prefill chunk on an fp32 residual stream, weights stored as their distance from one
        _norm("norm_t4096_2560_f32", 4096, 2560, "fp32", 1.0, True),
        # a ragged batch whose rows end inside a block
        _quantize("quantize_t33_720", 33, 720),
        # a long prefill's activations in front of a projection
        _quantize("quantize_t8192_4096", 8192, 4096),
        # one token through one projection: latency and weight bytes
        _linear("linear_t1_2048x2048", 1, 2048, 2048, False),
        # a batch of 32 decoding requests, an odd number of outputs
        _linear("linear_t32_9999x4096", 32, 9999, 4096, False),
        # an odd batch, a reduction that ends inside a block, a bias
        _linear("linear_t333_2560x5200", 333, 2560, 5200, True),
        # a prefill chunk: bound by the matrix cores
        _linear("linear_t4096_4096x4096", 4096, 4096, 4096, False),
        # the repository's decode batch: 4 tokens, 512 experts, top-10, H = 2048, I = 512
        _ffn("ffn_t4_2048x512_e512", 4, 2048, 512, 512, 10, 0.0),
        # a ragged verify batch at H = 2560, I = 640
        _ffn("ffn_t100_2560x640_e512", 100, 2560, 640, 512, 10, 0.0),
        # few large experts, unevenly chosen
        _ffn("ffn_t2000_4096x2048_e16", 2000, 4096, 2048, 16, 2, 0.7),
        # the repository's prefill chunk
        _ffn("ffn_t4096_2048x512_e512", 4096, 2048, 512, 512, 10, 0.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "linear", "ffn", "ffn"])
    if op == "norm":
        H = 16 * _log(rng, 2, 1024)
        c = _norm("", _log(rng, 1, min(16384, (1 << 25) // H)), H, rng.choice(["none", "bf16", "fp32"]),
                  rng.choice([0.0, 1.0]), rng.random() < 0.5)
    elif op == "quantize":
        K = 16 * _log(rng, 2, 1024)
        c = _quantize("", _log(rng, 1, min(16384, (1 << 25) // K)), K)
    elif op == "linear":
        K = 16 * _log(rng, 4, 512)
        N = _log(rng, 16, 16384)
        c = _linear("", _log(rng, 1, max(1, min(8192, int(6.8e10 / (K * N))))), N, K, rng.random() < 0.5)
    else:
        E = _log(rng, 2, 512)
        H = 16 * _log(rng, 8, 256)
        I = 16 * _log(rng, 4, max(4, min(128, int(5e8 / (16 * E * H)))))  # noqa: E741
        k = rng.randint(1, min(E, 10))
        c = _ffn("", _log(rng, 1, max(1, min(4096, int(4e10 / (k * H * I))))), H, I, E, k, rng.choice([0.0, 0.7]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _blocks(n):
    return -(-n // BLOCK)


def _encode(w):
    """fp32 [..., N, K] -> e4m3 codes [..., N, K] and fp32 scales [..., N/128, K/128], both rounded up."""
    *lead, N, K = w.shape
    nb, kb = _blocks(N), _blocks(K)
    p = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(*lead, nb, BLOCK, kb, BLOCK)
    scale = (p.abs().amax(dim=(-3, -1)) / TOP).clamp(min=SMALL)
    q = (p / scale[..., :, None, :, None]).to(E4M3).view(*lead, nb * BLOCK, kb * BLOCK)
    return q[..., :N, :K].contiguous(), scale


def _tokens(x):
    """fp32 [T, K] -> e4m3 codes [T, K] and fp32 scales [T, K/128], rounded up."""
    T, K = x.shape
    p = torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K)).view(T, _blocks(K), BLOCK)
    scale = (p.abs().amax(dim=2) / TOP).clamp(min=SMALL)
    return (p / scale.unsqueeze(2)).to(E4M3).view(T, -1)[:, :K].contiguous(), scale


def _activations(gen, T, K):
    """Activations with a few channels ten times the size of the others, as a layer's inputs have."""
    x = torch.randn((T, K), generator=gen, device=DEV)
    loud = torch.rand((K,), generator=gen, device=DEV) < 0.01
    return x * torch.where(loud, 10.0, 1.0)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 2 + 1)
    rand = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    op, T = case["op"], case["T"]
    s = {"case": case}
    if op in ("norm", "quantize"):
        K = case["H"] if op == "norm" else case["K"]
        s["x"] = _activations(gen, T, K).bfloat16()
        s["q"] = torch.empty((T, K), dtype=E4M3, device=DEV)
        s["scale"] = torch.empty((T, _blocks(K)), device=DEV)
        if op == "norm":
            dtype = {"none": None, "bf16": torch.bfloat16, "fp32": torch.float32}[case["stream"]]
            s["weight"] = (1.0 - case["offset"] + 0.1 * rand(K)).bfloat16()
            s["residual"] = None if dtype is None else (4.0 * rand(T, K)).to(dtype)
            s["residual_out"] = None if dtype is None else torch.empty((T, K), dtype=dtype, device=DEV)
            s["y"] = torch.empty((T, K), dtype=torch.bfloat16, device=DEV) if case["hidden"] else None
        if own:
            import sparse_moe_expert_amd as sme
            s["out"] = sme.Fp8Tokens(s["q"], s["scale"])
        return s
    if op == "linear":
        N, K = case["N"], case["K"]
        s["x"] = _tokens(_activations(gen, T, K))
        s["w"] = _encode(rand(N, K) / math.sqrt(K))
        s["bias"] = (0.1 * rand(N)).bfloat16() if case["bias"] else None
        s["y"] = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
        if own:
            import sparse_moe_expert_amd as sme
            s["x"], s["w"] = sme.Fp8Tokens(*s["x"]), sme.Fp8Weight(*s["w"])
            s["ws"] = sme.make_block_linear_workspace(DEV)
        return s
    H, I, E, k = case["H"], case["I"], case["E"], case["k"]
    s["x"] = _tokens(_activations(gen, T, H))
    s["gate"] = _encode(rand(E, I, H) / math.sqrt(H))
    s["up"] = _encode(rand(E, I, H) / math.sqrt(H))
    s["down"] = _encode(rand(E, H, I) / math.sqrt(I))
    top = torch.topk(rand(T, E) + case["skew"] * rand(E), k, dim=1)
    s["idx"], s["w"] = top.indices.int(), torch.softmax(top.values, dim=1)
    flat = s["idx"].reshape(-1).long()
    count = torch.zeros(E, dtype=torch.int64, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
    offset = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(count, 0)])
    src = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(src).scatter_(0, src, torch.arange(T * k, device=DEV))
    s["active"] = torch.nonzero(count).squeeze(1)
    s["count"], s["offset"], s["src"], s["pos"] = count[s["active"]], offset[s["active"]], src, pos
    s["most"] = int(count.max())
    s["y"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    if own:
        import sparse_moe_expert_amd as sme
        s["x"] = sme.Fp8Tokens(*s["x"])
        s["experts"] = sme.Fp8Experts(*s["gate"], *s["up"], *s["down"])
        s["buckets"] = sme.moe_bucket_routes(s["idx"], E)
        s["ws"] = sme.make_block_ffn_workspace(T, H, I, E, k, DEV)
    return s


# ------------------------------------------------------------------ plain forms

def _wide(enc):
    """A weight as fp32 from its codes and scales."""
    q, scale = enc
    N, K = q.shape[-2:]
    s = scale.repeat_interleave(BLOCK, dim=-2)[..., :N, :].repeat_interleave(BLOCK, dim=-1)[..., :K]
    return q.float() * s


def _wide_tokens(enc):
    q, scale = enc
    return q.float() * scale.repeat_interleave(BLOCK, dim=-1)[..., : q.shape[-1]]


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    r, out = x, None
    if s["residual"] is not None:
        out = (x + s["residual"].float()).to(s["residual"].dtype)
        r = out.float()
    y = r / torch.sqrt((r * r).mean(dim=1, keepdim=True) + 1e-6) * (s["weight"].float() + c["offset"])
    q, scale = _tokens(y)
    return q, scale, out, y.bfloat16() if c["hidden"] else None


def _plain_linear(s):
    y = _wide_tokens(s["x"]) @ _wide(s["w"]).t()
    return (y if s["bias"] is None else y + s["bias"].float()).bfloat16()


def _plain_ffn(s):
    c = s["case"]
    T, k, active = c["T"], c["k"], s["active"]
    gate, up, down = (_wide((q[active], scale[active])) for q, scale in (s["gate"], s["up"], s["down"]))
    # each chosen expert's routes as rows of one padded array; row T of x is zero
    row = torch.arange(s["most"], device=DEV)
    at = s["offset"][:, None] + row
    live = row < s["count"][:, None]
    token = torch.where(live, s["src"][at.clamp(max=T * k - 1)] // k, T)
    x = torch.cat([_wide_tokens(s["x"]), torch.zeros((1, c["H"]), device=DEV)])[token]
    g = torch.bmm(x, gate.transpose(1, 2).contiguous())
    u = torch.bmm(x, up.transpose(1, 2).contiguous())
    h = g / (1.0 + torch.exp(-g)) * u
    h = _wide_tokens(_tokens(h.view(-1, c["I"]))).view(active.numel(), -1, c["I"])
    o = torch.bmm(h, down.transpose(1, 2).contiguous())
    expert = torch.bucketize(s["pos"], s["offset"], right=True) - 1
    routes = o[expert, s["pos"] - s["offset"][expert]].view(T, k, -1)
    return (routes * s["w"].unsqueeze(2)).sum(dim=1).bfloat16()


def _own_run(s):
    import sparse_moe_expert_amd as sme
    c = s["case"]
    if c["op"] == "norm":
        tokens, r = sme.moe_norm_quantize(s["x"], s["weight"], s["residual"], eps=1e-6, weight_offset=c["offset"], out=s["out"],
                                     residual_out=s["residual_out"], y=s["y"])
        return tokens.q, tokens.scale, r, s["y"]
    if c["op"] == "quantize":
        return tuple(sme.moe_block_quantize(s["x"], s["out"]))
    if c["op"] == "linear":
        return sme.moe_block_linear(s["x"], s["w"], s["bias"], s["y"], s["ws"])
    return sme.moe_block_expert_ffn(s["x"], s["experts"], s["w"], s["buckets"], s["ws"], s["y"])


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "quantize":
        return _tokens(state["x"].float())
    return {"norm": _plain_norm, "linear": _plain_linear, "ffn": _plain_ffn}[op](state)


# ------------------------------------------------------------------ work and exact values

def _touched(case):
    """Experts with a route, expected under even routing: E (1 - (1 - k/E)^T)."""
    E = case["E"]
    return E * (1.0 - (1.0 - case["k"] / E) ** case["T"])


def work(case):
    op, T = case["op"], case["T"]
    if op in ("norm", "quantize"):
        K = case["H"] if op == "norm" else case["K"]
        n = T * K * 3 + 4 * T * _blocks(K)                       # bf16 in, e4m3 and scales out
        if op == "norm":
            n += T * K * ({"none": 0, "bf16": 4, "fp32": 8}[case["stream"]] + (2 if case["hidden"] else 0)) + 2 * K
        return {"bytes": n, "flops": T * K * (8 if op == "norm" else 4)}
    token = lambda K: K + 4 * _blocks(K)  # noqa: E731
    weight = lambda N, K: N * K + 4 * _blocks(N) * _blocks(K)  # noqa: E731
    if op == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": weight(N, K) + T * token(K) + 2 * T * N + (2 * N if case["bias"] else 0), "flops": 2 * T * N * K}
    H, I, k = case["H"], case["I"], case["k"]
    experts = 2 * weight(I, H) + weight(H, I)
    return {"bytes": int(_touched(case) * experts) + T * token(H) + 2 * T * H + 12 * T * k, "flops": 6 * T * k * H * I}


def _exact_encode(v):
    """float64 [n, K] -> code values before their rounding, and scales: amax / 448 of each 128."""
    n, K = v.shape
    parts = [(v[:, a:a + BLOCK], v[:, a:a + BLOCK].abs().amax(dim=1, keepdim=True) / TOP) for a in range(0, K, BLOCK)]
    scale = torch.cat([s.clamp(min=SMALL) for _, s in parts], dim=1)
    return torch.cat([p / s.clamp(min=SMALL) for p, s in parts], dim=1), scale


def _exact_e4m3(v):
    """The nearest e4m3 value, ties to even: steps of 2^(e-3), e at least -6."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp(min=-9))
    return torch.round(v / step) * step


def _exact_times(x, x_scale, q, scale):
    """x q^T with the scales of x's blocks of 128 columns and of q's blocks of 128 x 128."""
    y = torch.zeros((x.shape[0], q.shape[0]), dtype=torch.float64, device=x.device)
    rows = torch.arange(q.shape[0], device=x.device) // BLOCK
    for b in range(scale.shape[1]):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        part = torch.mm(x[:, at].contiguous(), q[:, at].double().t().contiguous())
        y += part * x_scale[:, b:b + 1] * scale[rows, b].double()
    return y


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "quantize":
        return _exact_encode(s["x"].double())
    if op == "norm":
        r, total = s["x"].double(), None
        if s["residual"] is not None:
            total = r + s["residual"].double()
            r = total.to(s["residual"].dtype).double()
        y = r * torch.rsqrt((r * r).sum(dim=1, keepdim=True) / case["H"] + 1e-6) * (s["weight"].double() + case["offset"])
        return *_exact_encode(y), total, y if case["hidden"] else None
    if op == "linear":
        y = _exact_times(s["x"][0].double(), s["x"][1].double(), *s["w"])
        return y if s["bias"] is None else y + s["bias"].double()
    T, k = case["T"], case["k"]
    y = torch.zeros((T, case["H"]), dtype=torch.float64, device=DEV)
    idx = s["idx"].long()
    for e in torch.unique(idx).tolist():
        t, j = torch.nonzero(idx == e, as_tuple=True)
        x, xs = s["x"][0][t].double(), s["x"][1][t].double()
        g = _exact_times(x, xs, s["gate"][0][e], s["gate"][1][e])
        h = g * torch.sigmoid(g) * _exact_times(x, xs, s["up"][0][e], s["up"][1][e])
        v, hs = _exact_encode(h)
        o = _exact_times(_exact_e4m3(v), hs, s["down"][0][e], s["down"][1][e])
        y.index_add_(0, t, o * s["w"][t, j].double().unsqueeze(1))
    return y
