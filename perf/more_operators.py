"""Measured cases of the 4-bit products and of the mixture of experts around them: the routing of
tokens to experts, the product of 4-bit weights with group scales, and the experts' feed-forward
blocks on such weights.  `run` computes a case either with elementary torch operations in 32 bits
(own = False) or with the library's entry points (own = True).

Weights (the library's layout): codes [N][K / 2] bytes, column 2j in the low four bits of byte j and
2j + 1 in the high ones; scales [N][S] fp16 and zeros [N][S] bytes, one of each for `group` columns,
S = round_up(K / group, 8).  A code c stands for d * (c - z); without zeros, z is 8.
"""
import math

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # One user's token: latency.  Softmax scores, eight of 64 experts.
        dict(name="route_t1_e64_f32", op="route", tokens=1, spare=0, experts=64, k=8, scoring="softmax", bias=False,
             groups=1, keep=1, renormalize=True, scale=1.0, type="f32"),
        # A batch of prompts: sigmoid scores with a balancing bias, four groups of eight, an odd number of tokens.
        dict(name="route_t8191_e256_f32", op="route", tokens=8191, spare=0, experts=256, k=8, scoring="sigmoid",
             bias=True, groups=8, keep=4, renormalize=True, scale=2.5, type="f32"),
        # One token through a gate projection of Qwen3-8B's sizes, small groups, fp32 as the library's products give.
        dict(name="product_t1_f32", op="product", tokens=1, n=12288, k=4096, group=32, zeros=False, type="f32"),
        # Five drafted tokens through its down projection, with zero points.
        dict(name="product_t5_bf16", op="product", tokens=5, n=4096, k=12288, group=128, zeros=True, type="bf16"),
        # A decode batch of 64 requests through its output projection.
        dict(name="product_t64_bf16", op="product", tokens=64, n=4096, k=4096, group=128, zeros=False, type="bf16"),
        # A prompt of an odd length through a projection of BitNet-2B4T's sizes, fp32.
        dict(name="product_t509_f32", op="product", tokens=509, n=6912, k=2560, group=64, zeros=True, type="f32"),
        # Long prompts through a gate projection.
        dict(name="product_t4096_bf16", op="product", tokens=4096, n=12288, k=4096, group=128, zeros=False, type="bf16"),
        # One user's token through its eight experts.
        dict(name="experts_t1_bf16", op="experts", tokens=1, spare=0, hidden=2048, ffn=1024, experts=64, k=8,
             group=128, zeros=False, type="bf16"),
        # A decode batch, padded to the size of a captured graph: a few tokens per expert, fp32.
        dict(name="experts_t48_f32", op="experts", tokens=48, spare=5, hidden=2048, ffn=1024, experts=64, k=8,
             group=64, zeros=True, type="f32"),
        # A chunk of a prompt, few large experts, odd sizes.
        dict(name="experts_t331_f32", op="experts", tokens=331, spare=0, hidden=2560, ffn=1152, experts=12, k=2,
             group=32, zeros=False, type="f32"),
        # A chunk of a prompt beside decoding requests.
        dict(name="experts_t777_bf16", op="experts", tokens=777, spare=0, hidden=2048, ffn=768, experts=128, k=8,
             group=128, zeros=False, type="bf16"),
        # Long prompts.
        dict(name="experts_t4096_bf16", op="experts", tokens=4096, spare=0, hidden=2048, ffn=1024, experts=64, k=8,
             group=128, zeros=True, type="bf16"),
    ]


MOST_FLOPS = 4.2e11  # a drawn case's, about the largest listed one's


def _spread(rng, lo, hi):
    """A whole number in lo..hi, uniform in its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "product", "product", "experts", "experts"])
    kind = dict(op=op, type=rng.choice(["f32", "bf16"]))
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.choice([4, 8, 9, 16, 32])
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(8, keep * experts // groups))
        tokens = _spread(rng, 1, 8000)
        return kind | dict(tokens=tokens, spare=rng.choice([0, tokens // 9]), experts=experts, k=k,
                           scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                           keep=keep, renormalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
    group = rng.choice([32, 64, 128])
    if op == "product":
        n, k = _spread(rng, 60, 12288), group * _spread(rng, 4, 12288 // group)
        return kind | dict(tokens=min(_spread(rng, 1, 4096), int(MOST_FLOPS / (2 * n * k))), n=n, k=k, group=group,
                           zeros=rng.random() < 0.5)
    hidden, ffn = 128 * rng.randint(4, 20), group * _spread(rng, 256 // group, 1536 // group)
    experts = _spread(rng, 4, 128)
    k = rng.randint(1, min(8, experts))
    tokens = min(_spread(rng, 1, 4096), int(MOST_FLOPS / (6 * hidden * ffn * k)))
    return kind | dict(tokens=tokens, spare=rng.choice([0, 0, tokens // 7]), hidden=hidden, ffn=ffn, experts=experts,
                       k=k, group=group, zeros=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _dtype(case):
    return torch.float32 if case["type"] == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return dict(route=_prepare_route, product=_prepare_product, experts=_prepare_experts)[case["op"]](case, g) | {
        "case": case}


def _prepare_route(case, g):
    T, E, k = case["tokens"], case["experts"], case["k"]
    # Some experts are more popular than others; the balancing bias goes against that.
    popular = 0.7 * torch.randn(E, generator=g, device=DEVICE)
    logits = (1.5 * torch.randn(T, E, generator=g, device=DEVICE) + popular).to(_dtype(case))
    i32 = dict(dtype=torch.int32, device=DEVICE)
    return dict(logits=logits, bias=-0.1 * popular + 0.02 * torch.randn(E, generator=g, device=DEVICE),
                live=torch.tensor([T - case["spare"]], **i32), ids=torch.empty(T, k, **i32),
                weights=torch.empty(T, k, dtype=torch.float32, device=DEVICE), start=torch.empty(E + 1, **i32),
                order=torch.empty(T * k, **i32))


def _matrices(g, count, n, k, group, zeros):
    """count matrices [n][k] of 4-bit weights with about unit gain: (codes, scales, zeros or None)."""
    S = (k // group + 7) // 8 * 8
    codes = torch.randint(0, 256, (count, n, k // 2), generator=g, device=DEVICE, dtype=torch.uint8)
    scales = (0.5 + torch.rand(count, n, S, generator=g, device=DEVICE)) / (4.6 * math.sqrt(k))
    z = torch.randint(5, 11, (count, n, S), generator=g, device=DEVICE, dtype=torch.uint8) if zeros else None
    return codes, scales.half(), z


def _activations(g, tokens, k, dtype):
    """Rows with a few strong columns, as a slice of a wider buffer."""
    strong = 1 + 5 * (torch.rand(k, generator=g, device=DEVICE) < 0.02)
    wide = torch.randn(tokens, k + 64, generator=g, device=DEVICE)
    wide[:, :k] *= strong
    return wide.to(dtype)[:, :k]


def _prepare_product(case, g):
    T, N, K = case["tokens"], case["n"], case["k"]
    codes, scales, zeros = _matrices(g, 1, N, K, case["group"], case["zeros"])
    return dict(codes=codes[0], scales=scales[0], zeros=None if zeros is None else zeros[0],
                x=_activations(g, T, K, _dtype(case)), y=torch.empty(T, N, dtype=_dtype(case), device=DEVICE))


def _prepare_experts(case, g):
    T, E, k, H, F = (case[n] for n in ("tokens", "experts", "k", "hidden", "ffn"))
    up = _matrices(g, E, 2 * F, H, case["group"], case["zeros"])
    down = _matrices(g, E, H, F, case["group"], case["zeros"])
    # What the routing leaves: experts and weights of each token, and the pairs (token, place) by expert.
    score = torch.randn(T, E, generator=g, device=DEVICE) + 0.5 * torch.randn(E, generator=g, device=DEVICE)
    best, ids = score.topk(k, dim=1)
    weights = torch.exp(best - best[:, :1])
    weights = weights / weights.sum(1, keepdim=True)
    idle = torch.arange(T, device=DEVICE)[:, None] >= T - case["spare"]
    ids = torch.where(idle, -1, ids)
    weights = torch.where(idle, 0, weights)
    flat = ids.flatten()
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    order = torch.where(torch.arange(T * k, device=DEVICE) < (T - case["spare"]) * k, order, -1)
    start = torch.zeros(E + 1, dtype=torch.int64, device=DEVICE)
    start[1:] = torch.cumsum(torch.bincount(flat[flat >= 0], minlength=E), 0)
    return dict(x=_activations(g, T, H, _dtype(case)), up=up, down=down, ids=ids.int(), weights=weights,
                start=start.int(), order=order.int(), most=int((start[1:] - start[:-1]).max()),
                y=torch.empty(T, H, dtype=_dtype(case), device=DEVICE))


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return dict(route=_own_route, product=_own_product, experts=_own_experts)[op](state)
    return dict(route=_plain_route, product=_plain_product, experts=_plain_experts)[op](state)


def _library():
    import bit_matvec_lb_gb300 as lb
    return lb


def _workspace(s, nbytes):
    if "workspace" not in s:
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=DEVICE)
    return s["workspace"]


def _own_route(s):
    lb, c = _library(), s["case"]
    T, E = c["tokens"], c["experts"]
    lb.lb_route(s["logits"], lb.OUT_F32 if c["type"] == "f32" else lb.OUT_BF16, s["logits"].stride(0), T, E, c["k"],
                lb.ROUTE_SOFTMAX if c["scoring"] == "softmax" else lb.ROUTE_SIGMOID, s["ids"], s["weights"],
                s["start"], s["order"], _workspace(s, lb.lb_route_workspace_bytes(T, E)),
                bias=s["bias"] if c["bias"] else None, groups=c["groups"], keep_groups=c["keep"],
                group_best=2 if c["bias"] else 1, renormalize=c["renormalize"], scale=c["scale"],
                live=s["live"] if c["spare"] else None)
    return [s["ids"], s["weights"], s["start"], s["order"]]


def _own_product(s):
    lb, c = _library(), s["case"]
    T, N, K = c["tokens"], c["n"], c["k"]
    fmt = lb.OUT_F32 if c["type"] == "f32" else lb.OUT_BF16
    if T <= 8:
        lb.lb_gemv_q4(s["codes"], s["scales"], s["zeros"], c["group"], s["x"], fmt, s["x"].stride(0), s["y"],
                      s["y"].stride(0), N, K, T)
    else:
        lb.lb_gemm_q4(s["codes"], s["scales"], s["zeros"], c["group"], s["x"], fmt, s["x"].stride(0), s["y"],
                      s["y"].stride(0), T, N, K, _workspace(s, lb.lb_gemm_q4_workspace_bytes(T, N, K, fmt)))
    return s["y"]


def _own_experts(s):
    lb, c = _library(), s["case"]
    T, E, k, H, F = (c[n] for n in ("tokens", "experts", "k", "hidden", "ffn"))
    fmt = lb.OUT_F32 if c["type"] == "f32" else lb.OUT_BF16
    lb.lb_experts_q4(s["x"], fmt, s["x"].stride(0), T, E, k, H, F, c["group"], s["up"], s["down"], s["ids"],
                     s["weights"], s["start"], s["order"], s["y"], s["y"].stride(0),
                     _workspace(s, lb.lb_experts_q4_workspace_bytes(T, E, k, H, F, fmt)))
    return s["y"]


def _plain_route(s):
    c = s["case"]
    T, E, k, G = c["tokens"], c["experts"], c["k"], c["groups"]
    # 64 bits: two scores may lie closer together than 32 tell apart
    x = s["logits"].double()
    if c["scoring"] == "softmax":
        score = torch.exp(x - x.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-x))
    key = score + s["bias"].double() if c["bias"] else x
    if G > 1:
        parts = key.view(T, G, E // G)
        best = parts.sort(dim=2, descending=True).values[:, :, :2 if c["bias"] else 1].sum(2)
        first = best.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=DEVICE).scatter_(1, first, True)
        key = torch.where(kept[:, :, None], parts, -math.inf).view(T, E)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    weights = score.gather(1, ids)
    if c["renormalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    live = torch.arange(T, device=DEVICE)[:, None] < s["live"]
    ids = torch.where(live, ids, -1)
    weights = torch.where(live, weights * c["scale"], 0)
    flat = ids.flatten()
    start = torch.zeros(E + 1, dtype=torch.int64, device=DEVICE)
    start[1:] = torch.cumsum((flat[:, None] == torch.arange(E, device=DEVICE)).sum(0), 0)
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    order = torch.where(torch.arange(T * k, device=DEVICE) < start[-1], order, -1)
    return [ids.int(), weights.float(), start.int(), order.int()]


def _weights(matrix, k, group):
    """fp32 weights [..., n, k] of (codes, scales, zeros or None)."""
    codes, scales, zeros = matrix
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (k // group, group)).float()
    z = 8.0 if zeros is None else zeros[..., :k // group, None].float()
    return ((c - z) * scales[..., :k // group, None].float()).flatten(-2)


def _plain_product(s):
    c = s["case"]
    w = _weights((s["codes"], s["scales"], s["zeros"]), c["k"], c["group"])
    return torch.matmul(s["x"].float(), w.t()).to(_dtype(c))


def _plain_experts(s):
    c = s["case"]
    T, E, k, H, F = (c[n] for n in ("tokens", "experts", "k", "hidden", "ffn"))
    # each expert's tokens in rows of one padded batch
    flat, start = s["ids"].flatten().long(), s["start"].long()
    pair = s["order"].long()
    there = pair >= 0
    expert = torch.where(there, flat[pair.clamp(min=0)], 0)
    row = torch.where(there, torch.arange(T * k, device=DEVICE) - start[expert], s["most"])
    x = torch.zeros(E, s["most"] + 1, H, device=DEVICE)
    x[expert, row] = s["x"].float()[pair.clamp(min=0) // k]
    gate, up = torch.bmm(x, _weights(s["up"], H, c["group"]).transpose(1, 2)).split(F, dim=2)
    h = gate / (1 + torch.exp(-gate)) * up
    y = torch.bmm(h, _weights(s["down"], F, c["group"]).transpose(1, 2))
    part = torch.zeros(T * k + 1, H, device=DEVICE)
    part[torch.where(there, pair, T * k)] = y[expert, row]
    return (part[:-1].view(T, k, H) * s["weights"][:, :, None]).sum(1).to(_dtype(c))


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------
def _weight_bytes(n, k, case):
    return n * k / 2 + n * (k // case["group"]) * (3 if case["zeros"] else 2)


def work(case):
    size, T = 4 if case["type"] == "f32" else 2, case["tokens"]
    if case["op"] == "route":
        E, k = case["experts"], case["k"]
        return dict(bytes=(T - case["spare"]) * E * size + T * k * 12 + 4 * (E + 1), flops=T * E * 8)
    if case["op"] == "product":
        N, K = case["n"], case["k"]
        return dict(bytes=_weight_bytes(N, K, case) + T * (N + K) * size, flops=2 * T * N * K)
    E, k, H, F = (case[n] for n in ("experts", "k", "hidden", "ffn"))
    live = T - case["spare"]
    used = E * (1 - (1 - k / E) ** live)  # experts that some token goes to, if all are equally likely
    return dict(bytes=used * (_weight_bytes(2 * F, H, case) + _weight_bytes(H, F, case)) + (live + T) * H * size
                + live * k * 12, flops=6 * live * k * H * F)


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return dict(route=_exact_route, product=_exact_product, experts=_exact_experts)[case["op"]](s)


def _exact_route(s):
    c = s["case"]
    T, E, k, n = c["tokens"], c["experts"], c["k"], c["experts"] // c["groups"]
    weights = torch.zeros(T, k, dtype=torch.float64, device=DEVICE)
    x = s["logits"].to(torch.float64)
    score = torch.softmax(x, 1) if c["scoring"] == "softmax" else torch.sigmoid(x)
    rank = (score + s["bias"].to(torch.float64) if c["bias"] else x).clone()
    if c["groups"] > 1:
        best = torch.stack([rank[:, g * n:(g + 1) * n].topk(2 if c["bias"] else 1, dim=1).values.sum(1)
                            for g in range(c["groups"])], 1)
        for _ in range(c["groups"] - c["keep"]):  # the worst group goes (the later of two equal ones)
            worst = c["groups"] - 1 - best.flip(1).argmin(1)
            best.scatter_(1, worst[:, None], math.inf)
        rank[(best < math.inf).logical_not().repeat_interleave(n, 1)] = -math.inf
    for j in range(k):
        at = rank.argmax(1, keepdim=True)
        weights[:, j] = score.gather(1, at)[:, 0]
        rank.scatter_(1, at, -math.inf)
    if c["renormalize"]:
        weights /= weights.sum(1, keepdim=True)
    weights[T - c["spare"]:] = 0
    return [None, weights * c["scale"], None, None]


def _exact_matrix(codes, scales, zeros, k, group):
    w = torch.empty(codes.shape[0], k, dtype=torch.float64, device=DEVICE)
    w[:, 0::2], w[:, 1::2] = codes.remainder(16).double(), (codes // 16).double()
    per = torch.arange(k, device=DEVICE) // group
    w -= 8 if zeros is None else zeros.double()[:, per]
    return w * scales.double()[:, per]


def _exact_product(s):
    c = s["case"]
    w = _exact_matrix(s["codes"], s["scales"], s["zeros"], c["k"], c["group"])
    return torch.einsum("tk,nk->tn", s["x"].double(), w)


def _exact_experts(s):
    c = s["case"]
    y = torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device=DEVICE)
    for e in range(c["experts"]):
        token, place = (s["ids"] == e).nonzero(as_tuple=True)
        w, v = ([None if m is None else m[e] for m in s[n]] for n in ("up", "down"))
        both = s["x"][token].double() @ _exact_matrix(*w, c["hidden"], c["group"]).t()
        h = torch.nn.functional.silu(both[:, :c["ffn"]]) * both[:, c["ffn"]:]
        part = h @ _exact_matrix(*v, c["ffn"], c["group"]).t()
        y.index_add_(0, token, part * s["weights"][token, place].double()[:, None])
    return y
