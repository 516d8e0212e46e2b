"""What is measured of the routing and 4-bit dense operators: their cases, inputs and plain forms.

Three operators of one sparse-MoE layer:
  route   moe_route_grouped_bucket   router scores (softmax or sigmoid), a balance bias in the selection only,
                                     groups of experts, top-k, gate weights, and the routes' buckets
  linear  moe_quant_linear           y = x W^T + bias, W in 4 bits with a scale per group (NVFP4, MXFP4)
  shared  moe_quant_shared_expert    y = add + sigmoid(x . v) * W_down (SiLU(W_gate x) * (W_up x)), 4-bit weights

With `own` false, run() computes them with elementary torch operations; with `own` true it calls the library.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
LOWEST = -3.3e38              # a logit or bias at or below this, or NaN, masks its expert
FLT_MAX = 3.4028234663852886e38
GROUP = {"nvfp4": 16, "mxfp4": 32}      # weights that share a scale


# ------------------------------------------------------------------ cases

def _route(name, T, E, k, groups, kept, group_top, score, renorm, scale, dtype, masked):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "groups": groups, "kept": kept,
            "group_top": group_top, "score": score, "renorm": renorm, "scale": scale, "dtype": dtype, "masked": masked}


def _linear(name, T, N, K, fmt, bias):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "fmt": fmt, "bias": bias}


def _shared(name, T, H, Is, fmt, gated, add):
    return {"name": name, "op": "shared", "T": T, "H": H, "Is": Is, "fmt": fmt, "gated": gated, "add": add}


def listed():
    return [
        # one token of a decode loop: the latency of the routing alone
        _route("route_t1_e256_g8", 1, 256, 8, 8, 4, 2, "sigmoid", True, 2.5, "fp32", False),
        # the repository's decode batch (4 tokens, 512 experts, top-10), without groups
        _route("route_t4_e512", 4, 512, 10, 1, 1, 1, "softmax", True, 1.0, "fp32", False),
        # a ragged batch with bf16 logits (ties), few experts per group, weights left unnormalised
        _route("route_t333_e160_g8", 333, 160, 6, 8, 3, 1, "softmax", False, 16.0, "bf16", False),
        # a prefill chunk (4096 tokens, 512 experts) with some experts masked out
        _route("route_t4096_e512_g16", 4096, 512, 10, 16, 8, 2, "sigmoid", True, 1.0, "fp32", True),
        # one token through one projection: latency and weight bytes
        _linear("linear_t1_2048x2048", 1, 2048, 2048, "nvfp4", False),
        # four speculative tokens, a wide projection with a bias
        _linear("linear_t4_10240x2560_mx", 4, 10240, 2560, "mxfp4", True),
        # a batch of 32 decoding requests, an odd number of outputs
        _linear("linear_t32_9999x4096", 32, 9999, 4096, "nvfp4", False),
        # a prefill chunk: bound by the matrix cores
        _linear("linear_t4096_4096x4096", 4096, 4096, 4096, "nvfp4", False),
        # the repository's decode layer: 4 tokens, H = 2048, Is = 512, summed onto the routed output
        _shared("shared_t4_2048x512", 4, 2048, 512, "nvfp4", True, True),
        # one token through a large dense FFN: weight bytes
        _shared("shared_t1_4096x12288_mx", 1, 4096, 12288, "mxfp4", False, False),
        # a ragged verify batch at H = 2560, Is = 640
        _shared("shared_t100_2560x640", 100, 2560, 640, "nvfp4", True, True),
        # a prefill chunk, gated and summed
        _shared("shared_t4096_2048x2048", 4096, 2048, 2048, "nvfp4", True, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "linear", "shared"])
    fmt = rng.choice(["nvfp4", "mxfp4"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16, 32])
        size = _log(rng, 2 if groups > 1 else 8, 1024 // groups)
        E = groups * size
        kept = rng.randint(1, groups)
        k = _log(rng, 1, min(32, kept * size))
        c = _route("", _log(rng, 1, 8192), E, k, groups, kept, rng.choice([1, 2]), rng.choice(["softmax", "sigmoid"]),
                   rng.random() < 0.6, rng.choice([1.0, 1.0, 2.5, 16.0]), rng.choice(["fp32", "bf16"]), rng.random() < 0.3)
    elif op == "linear":
        K = 32 * _log(rng, 2, 256)
        N = _log(rng, 16, 16384)
        T = _log(rng, 1, max(1, min(8192, int(6.8e10 / (K * N)))))
        c = _linear("", T, N, K, fmt, rng.random() < 0.5)
    else:
        H = 32 * _log(rng, 4, 128)
        Is = 32 * _log(rng, 2, 384)
        T = _log(rng, 1, max(1, min(8192, int(2.2e10 / (H * Is)))))
        c = _shared("", T, H, Is, fmt, rng.random() < 0.5, rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _bf16(t):
    return t.to(torch.bfloat16)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode(w, fmt):
    """fp32 [N,K] -> codes uint8 [N,K/2] (element 2i in the low nibble of byte i), scales uint8 [N,K/G], global fp32 [1]."""
    N, K = w.shape
    G = GROUP[fmt]
    blocks = w.view(N, K // G, G)
    amax = blocks.abs().amax(dim=2)
    if fmt == "nvfp4":
        g = (w.abs().max() / (6.0 * 448.0)).reshape(1)
        s8 = (amax / (6.0 * g)).to(torch.float8_e4m3fn)
        scales = s8.view(torch.uint8)
        step = s8.float() * g
    else:
        g = None
        e = torch.floor(torch.log2(amax.clamp(min=1e-30))) - 2.0          # e2m1's largest exponent is 2
        scales = (e + 127.0).to(torch.uint8)
        step = torch.exp2(e)
    v = blocks / step.clamp(min=1e-38).unsqueeze(2)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    codes = torch.bucketize(v.abs(), edges).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    codes = codes.view(N, K)
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous(), scales.contiguous(), g


def _weight(gen, N, K, fmt):
    return _encode(torch.randn((N, K), generator=gen, device=DEV) / math.sqrt(K), fmt)


def _handle(enc, fmt):
    """The library's handle of a weight: the same tensors, nothing laid out anew."""
    import sparse_moe_expert_amd as sme
    return sme.QuantWeight(*enc, fmt)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 2 + 1)
    rand = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    s = {"case": case}
    T = case["T"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        s["logits"] = rand(T, E) * 1.5
        if case["dtype"] == "bf16":
            s["logits"] = _bf16(s["logits"])
        s["bias"] = rand(E) * 0.05
        if case["masked"]:                                  # experts out of service
            s["bias"][torch.rand((E,), generator=gen, device=DEV) < 0.1] = float("-inf")
        i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device=DEV)  # noqa: E731
        s["idx"], s["w"] = i32(T, k), torch.empty((T, k), device=DEV)
        s["buckets"] = (i32(E), i32(E + 1), i32(E), i32(1), i32(T * k), i32(T * k))
        if own:
            import sparse_moe_expert_amd as sme
            s["rule"] = sme.RouteRule(k, case["score"], case["groups"], case["kept"], case["group_top"], case["renorm"],
                                      case["scale"])
            s["buckets"] = sme.Buckets(*s["buckets"])
        return s
    fmt = case["fmt"]
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        s["x"] = _bf16(rand(T, K))
        s["w"] = _weight(gen, N, K, fmt)
        s["bias"] = _bf16(rand(N) * 0.1) if case["bias"] else None
        s["y"] = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
        if own:
            s["w"] = _handle(s["w"], fmt)
        return s
    H, Is = case["H"], case["Is"]
    s["x"] = _bf16(rand(T, H))
    s["gate"], s["up"], s["down"] = _weight(gen, Is, H, fmt), _weight(gen, Is, H, fmt), _weight(gen, H, Is, fmt)
    s["token_gate"] = _bf16(rand(H) / math.sqrt(H)) if case["gated"] else None
    s["add"] = _bf16(rand(T, H) * 0.3) if case["add"] else None
    s["y"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    if own:
        import sparse_moe_expert_amd as sme
        s["gate"], s["up"], s["down"] = (_handle(s[n], fmt) for n in ("gate", "up", "down"))
        s["ws"] = sme.make_quant_shared_workspace(T, H, Is, DEV)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    dev = s["logits"].device
    # in 64 bits: a selection between near-equal scores is not left to an exponential's rounding
    z, b = s["logits"].double(), s["bias"].double()
    off = torch.isnan(z) | (z <= LOWEST)
    z = z.clamp(max=FLT_MAX)
    if c["score"] == "softmax":
        top = torch.where(off, torch.full_like(z, LOWEST), z).amax(dim=1, keepdim=True)
        e = torch.where(off, torch.zeros_like(z), torch.exp(z - top))
        total = e.sum(dim=1, keepdim=True)
        score = torch.where(total > 0, e / total, torch.zeros_like(e))
    else:
        score = torch.where(off, torch.zeros_like(z), 1.0 / (1.0 + torch.exp(-z)))
    off = off | torch.isnan(b) | (b <= LOWEST)
    inf = torch.full_like(z, float("-inf"))
    choice = torch.where(off, inf, score + b)
    grouped = choice.view(T, G, E // G)
    best = torch.sort(grouped, dim=2, descending=True).values[:, :, :c["group_top"]]
    group = torch.where(best == float("-inf"), torch.zeros_like(best), best).sum(dim=2)
    group = torch.where(best[:, :, 0] == float("-inf"), inf[:, :G], group)
    first = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
    kept = torch.zeros((T, G), dtype=torch.bool, device=dev).scatter_(1, first, True)
    kept = kept.unsqueeze(2).expand(T, G, E // G).reshape(T, E)
    key = torch.where(kept, torch.where(off, torch.full_like(z, -1e300), choice), inf)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.where(torch.gather(off, 1, idx), torch.zeros_like(z[:, :k]), torch.gather(score, 1, idx))
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    flat = idx.reshape(-1)
    count = (flat.unsqueeze(0) == torch.arange(E, device=dev).unsqueeze(1)).sum(dim=1) if T * k * E < 1 << 24 else \
        torch.zeros(E, dtype=torch.int64, device=dev).scatter_add_(0, flat, torch.ones_like(flat))
    offset = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(count, 0)])
    empty = count == 0
    order = torch.sort(empty.to(torch.int32), stable=True).indices      # experts with routes first, ascending
    n_active = (~empty).sum().reshape(1)
    active = torch.where(torch.arange(E, device=dev) < n_active, order, torch.full_like(order, -1))
    src = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(src).scatter_(0, src, torch.arange(T * k, device=dev))
    return (idx.int(), (w * c["scale"]).float(), count.int(), offset.int(), active.int(), n_active.int(), src.int(),
            pos.int())


def _dense(enc, fmt):
    """The weights as fp32, but for the global scale, which the product takes once."""
    codes, scales, _ = enc
    N, half = codes.shape
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), dim=2).long()].view(N, -1, GROUP[fmt])
    s = scales.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else torch.exp2(scales.float() - 127.0)
    return (v * s.unsqueeze(2)).view(N, 2 * half)


def _times(x, enc, fmt):
    y = x @ _dense(enc, fmt).t()
    return y if enc[2] is None else y * enc[2]


def _plain_linear(s):
    y = _times(s["x"].float(), s["w"], s["case"]["fmt"])
    return _bf16(y if s["bias"] is None else y + s["bias"].float())


def _plain_shared(s):
    fmt, x = s["case"]["fmt"], s["x"].float()
    g, u = _times(x, s["gate"], fmt), _times(x, s["up"], fmt)
    y = _times(g / (1.0 + torch.exp(-g)) * u, s["down"], fmt)
    if s["token_gate"] is not None:
        y = y / (1.0 + torch.exp(-(x * s["token_gate"].float()).sum(dim=1, keepdim=True)))
    return _bf16(y if s["add"] is None else y + s["add"].float())


def _own_run(s):
    import sparse_moe_expert_amd as sme
    op = s["case"]["op"]
    if op == "route":
        idx, w, buckets = sme.moe_route_grouped_bucket(s["logits"], s["bias"], s["rule"], s["idx"], s["w"], s["buckets"])
        return (idx, w, *buckets)
    if op == "linear":
        return sme.moe_quant_linear(s["x"], s["w"], s["bias"], s["y"])
    return sme.moe_quant_shared_expert(s["x"], s["gate"], s["up"], s["down"], s["token_gate"], s["add"], s["y"], s["ws"])


def run(state):
    if own:
        return _own_run(state)
    return {"route": _plain_route, "linear": _plain_linear, "shared": _plain_shared}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work and exact values

def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        read = T * E * (2 if case["dtype"] == "bf16" else 4) + 4 * E
        # a score of some 30 operations and k comparisons an expert
        return {"bytes": read + 8 * T * k + 4 * (3 * E + 2 + 2 * T * k), "flops": T * E * (30 + k)}
    per = 0.5 + 1.0 / GROUP[case["fmt"]]
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": int(N * K * per) + 2 * T * (N + K) + (2 * N if case["bias"] else 0), "flops": 2 * T * N * K}
    H, Is = case["H"], case["Is"]
    return {"bytes": int(3 * H * Is * per) + 2 * T * H * (3 if case["add"] else 2) + (2 * H if case["gated"] else 0),
            "flops": 6 * T * H * Is + (2 * T * H if case["gated"] else 0)}


def _exact_route(case, s):
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    size = E // G
    z = s["logits"].double().cpu().numpy()
    b = s["bias"].double().cpu().numpy()
    idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        usable = ~(np.isnan(z[t]) | (z[t] <= LOWEST))
        zt = np.where(usable, np.minimum(z[t], FLT_MAX), 0.0)
        p = np.zeros(E)
        if case["score"] == "sigmoid":
            p[usable] = 1.0 / (1.0 + np.exp(-zt[usable]))
        elif usable.any():
            p[usable] = np.exp(zt[usable] - zt[usable].max())
            p /= p.sum()
        usable &= ~(np.isnan(b) | (b <= LOWEST))
        # ordered by (masked, -choice, id): np.lexsort sorts by its last key first
        choice = np.where(usable, p + np.where(usable, b, 0.0), 0.0)
        ids = np.lexsort((np.arange(E), -choice, ~usable))
        total = np.zeros(G)
        taken = np.zeros(G, int)
        for e in ids[:int(usable.sum())]:
            if taken[e // size] < case["group_top"]:
                total[e // size] += choice[e]
                taken[e // size] += 1
        groups = set(np.lexsort((np.arange(G), -total, taken == 0))[:case["kept"]].tolist())
        chosen = [e for e in ids.tolist() if e // size in groups][:k]
        idx[t] = chosen
        w[t] = np.where(usable[chosen], p[chosen], 0.0)
    if case["renorm"]:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    flat = idx.reshape(-1)
    count = np.bincount(flat, minlength=E).astype(np.int32)
    offset = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    active = np.full(E, -1, np.int32)
    used = np.flatnonzero(count)
    active[:used.size] = used
    src = np.argsort(flat, kind="stable").astype(np.int32)
    pos = np.empty_like(src)
    pos[src] = np.arange(src.size)
    return idx, w * case["scale"], count, offset, active, np.array([used.size], np.int32), src, pos


def _exact_weight(enc, fmt):
    codes, scales, g = enc
    low, high = (codes & 15).long(), (codes >> 4).long()
    c = torch.stack((low, high), dim=2).flatten(1)
    e, m = (c >> 1) & 3, c & 1
    v = torch.where(e == 0, m * 0.5, torch.ldexp(1.0 + m.double() * 0.5, e - 1)) * (1.0 - 2.0 * (c >> 3).double())
    b = scales.long()
    if fmt == "nvfp4":
        e, m = (b >> 3) & 15, (b & 7).double()
        s = torch.where(e == 0, m * 2.0 ** -9, torch.ldexp(1.0 + m / 8.0, e - 7)) * float(g)
    else:
        s = torch.ldexp(torch.ones_like(b, dtype=torch.float64), b - 127)
    return v * s.repeat_interleave(GROUP[fmt], dim=1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "route":
        return _exact_route(case, s)
    fmt, x = case["fmt"], s["x"].double()
    if case["op"] == "linear":
        y = torch.mm(x, _exact_weight(s["w"], fmt).t())
        return y if s["bias"] is None else y + s["bias"].double()
    a = torch.mm(x, _exact_weight(s["gate"], fmt).t())
    a = a * torch.sigmoid(a) * torch.mm(x, _exact_weight(s["up"], fmt).t())
    y = torch.mm(a, _exact_weight(s["down"], fmt).t())
    if s["token_gate"] is not None:
        y = y * torch.sigmoid(torch.mv(x, s["token_gate"].double())).unsqueeze(1)
    return y if s["add"] is None else y + s["add"].double()
