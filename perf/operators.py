"""Measured cases of the serving operators that go around the low-bit products: the page plan of a
step, the 4-bit key/value cache (write and read back), attention over that cache, and the
adjustment of logits.  `run` computes a case either with elementary torch operations in 32 bits
(own = False) or with the library's entry points (own = True).

Cache layout (the library's): one byte buffer [pages][kv_heads][page_size / 16] of chunks of 16
tokens; a chunk holds 16 key rows and then 16 value rows of head_dim / 2 bytes (dimension 2j in
the low four bits of byte j, 2j + 1 in the high ones), then 16 {d, z} pairs of fp16 for the keys
and 16 for the values.  A code c stands for d * (c - z), z a whole number in 0..15.
"""
import math

import torch

own = False

CHUNK = 16
DEVICE = "cuda"


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # A decode step of a small server: every request adds one token.
        dict(name="plan_decode_r8", op="plan", requests=8, page=16, past=900, fresh=1, spare=0),
        # Continuous batching: many requests, most decode one token, some bring a prompt chunk.
        dict(name="plan_mixed_r512", op="plan", requests=512, page=64, past=8000, fresh=1500, spare=64),
        # One decode step's keys and values of a batch (Qwen3-8B's 8 heads of 128), as the
        # projections leave them: slices of one fp32 buffer.
        dict(name="store_decode_t64_f32", op="store", tokens=64, kv_heads=8, dim=128, page=16, type="f32"),
        # A prompt chunk of a batch, bf16.
        dict(name="store_prompt_t8191_bf16", op="store", tokens=8191, kv_heads=8, dim=128, page=64, type="bf16"),
        # One user, a short chat: latency.  fp32 as the library's products give and take.
        dict(name="attend_one_short_f32", op="attend", requests=1, heads=32, kv_heads=8, dim=128, page=16,
             q=1, past=332, ragged=False, window=0, type="f32"),
        # A full decode batch with ragged contexts.
        dict(name="attend_decode_r64_f32", op="attend", requests=64, heads=32, kv_heads=8, dim=128, page=64,
             q=1, past=4096, ragged=True, window=0, type="f32"),
        # One user with a very long context.
        dict(name="attend_long_131k_bf16", op="attend", requests=1, heads=32, kv_heads=8, dim=128, page=128,
             q=1, past=131070, ragged=False, window=0, type="bf16"),
        # Verification of five drafted tokens per request, BitNet-2B4T's 20/5 heads, sliding window.
        dict(name="attend_verify_r33_bf16", op="attend", requests=33, heads=20, kv_heads=5, dim=128, page=16,
             q=5, past=2500, ragged=True, window=1000, type="bf16"),
        # Ragged prompt chunks behind cached prefixes, fp32.
        dict(name="attend_chunk_r3_f32", op="attend", requests=3, heads=32, kv_heads=8, dim=128, page=64,
             q=1021, past=3000, ragged=True, window=0, type="f32"),
        # A long prompt at once, bf16.
        dict(name="attend_prompt_8k_bf16", op="attend", requests=1, heads=32, kv_heads=8, dim=128, page=64,
             q=8192, past=0, ragged=False, window=0, type="bf16"),
        # One user's logits (BitNet-2B4T vocabulary) under penalties, biases and a grammar.
        dict(name="logits_b1_f32", op="logits", rows=1, vocab=128256, prompt=700, output=200, biases=16,
             grammar=True, type="f32"),
        # A batch (Qwen3-8B vocabulary, an odd row length), long histories.
        dict(name="logits_b96_f32", op="logits", rows=96, vocab=151669, prompt=6000, output=2000, biases=100,
             grammar=True, type="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, uniform in its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "plan", "store", "logits"])
    if op == "plan":
        return dict(op=op, requests=_spread(rng, 1, 600), page=rng.choice([16, 32, 64, 128]),
                    past=_spread(rng, 1, 9000), fresh=rng.choice([1, 1, _spread(rng, 2, 1200)]),
                    spare=rng.choice([0, 7, 64]))
    if op == "store":
        return dict(op=op, tokens=_spread(rng, 1, 6000), kv_heads=rng.choice([1, 2, 5, 8]),
                    dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                    type=rng.choice(["f32", "bf16"]))
    if op == "logits":
        return dict(op=op, rows=_spread(rng, 1, 64), vocab=_spread(rng, 1000, 152000),
                    prompt=_spread(rng, 1, 8000), output=_spread(rng, 1, 2000),
                    biases=rng.choice([0, 3, 100]), grammar=rng.random() < 0.7,
                    type=rng.choice(["f32", "bf16"]))
    kv_heads = rng.choice([1, 2, 5, 8])
    group = rng.choice([1, 2, 4, 4, 5, 7, 8])
    kind = rng.choice(["decode", "decode", "verify", "prompt"])
    if kind == "decode":
        q, requests = 1, _spread(rng, 1, 96)
        past = _spread(rng, 1, max(2, 200000 // requests))
    elif kind == "verify":
        q, requests = rng.randint(2, 9), _spread(rng, 1, 32)
        past = _spread(rng, 1, max(2, 100000 // requests))
    else:
        q, requests = _spread(rng, 17, 2000), rng.randint(1, 3)
        past = rng.choice([0, _spread(rng, 1, 3000)])
    return dict(op=op, requests=requests, heads=kv_heads * group, kv_heads=kv_heads,
                dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]), q=q, past=past,
                ragged=rng.random() < 0.7, window=rng.choice([0, 0, 0, _spread(rng, 1, 2000)]),
                type=rng.choice(["f32", "bf16"]))


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _dtype(case):
    return torch.float32 if case["type"] == "f32" else torch.bfloat16


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEVICE)


def _spaced(lo, hi, n):
    """n whole numbers from hi down to lo at even distances: a ragged batch's lengths."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _shuffled(g, values):
    v = torch.tensor(values, device=DEVICE)
    return v[torch.randperm(v.numel(), generator=g, device=DEVICE)]


def _lengths(case):
    """The cached and the new tokens of an attend case's requests, each in falling order (the
    seed shuffles both; ragged requests end at different places)."""
    R, q, past = case["requests"], case["q"], case["past"]
    if not case["ragged"]:
        return [past] * R, [q] * R
    return _spaced(past // 4, past, R), _spaced((q + 1) // 2, q, R)


def _fresh(case):
    """The new tokens of a plan case's requests: one each, or (continuous batching) a chunk of a
    prompt in one request of eight, none in one of sixteen, and one each in the others."""
    R = case["requests"]
    if case["fresh"] == 1:
        return [1] * R
    return _spaced(1, case["fresh"], R // 8) + [0] * (R // 16) + [1] * (R - R // 8 - R // 16)


def _table(g, need, width, pages):
    """A block table [R][width]: need[r] different pages of 0..pages-1 in any order, then -1."""
    order = torch.randperm(pages, generator=g, device=DEVICE)
    start = torch.cumsum(need, 0) - need
    col = torch.arange(width, device=DEVICE)
    at = (start[:, None] + col).clamp(max=pages - 1)
    return torch.where(col < need[:, None], order[at], -1).to(torch.int32), order


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return dict(plan=_prepare_plan, store=_prepare_store, attend=_prepare_attend,
                logits=_prepare_logits)[case["op"]](case, g) | {"case": case}


def _prepare_plan(case, g):
    R, page = case["requests"], case["page"]
    past = _ints(g, 0, case["past"], R)
    fresh = _shuffled(g, _fresh(case))
    have = (past + page - 1) // page
    take = (past + fresh + page - 1) // page - have
    width = (case["past"] + case["fresh"] + page - 1) // page
    pages = int((have + take).sum()) + 16
    table, order = _table(g, have, width, pages)
    free = order[int(have.sum()):].to(torch.int32).contiguous()
    T = int(fresh.sum()) + case["spare"]
    i32 = dict(dtype=torch.int32, device=DEVICE)
    return dict(past=past.int(), fresh=fresh.int(), table=table, free=free, tokens=T, width=width,
                q_start=torch.empty(R + 1, **i32), kv_len=torch.empty(R, **i32),
                position=torch.empty(T, **i32), slot=torch.empty(T, dtype=torch.int64, device=DEVICE),
                counts=torch.empty(2, **i32))


def _prepare_store(case, g):
    T, H, D, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
    pages = (T + page - 1) // page + 3
    # The products leave q, k and v side by side; keys have a few strong dimensions.
    qkv = torch.randn(T, 6 * H * D, generator=g, device=DEVICE)
    strong = 1 + 3 * (torch.rand(H * D, generator=g, device=DEVICE) < 0.05)
    qkv[:, 4 * H * D:5 * H * D] *= strong
    qkv = qkv.to(_dtype(case))
    slot = torch.randperm(pages * page, generator=g, device=DEVICE)[:T]
    if T >= 64:  # a prompt's tokens lie page by page
        order = torch.randperm(pages, generator=g, device=DEVICE)
        at = torch.arange(T, device=DEVICE)
        slot = order[at // page] * page + at % page
    return dict(k=qkv[:, 4 * H * D:5 * H * D].unflatten(1, (H, D)), v=qkv[:, 5 * H * D:].unflatten(1, (H, D)),
                slot=slot, pages=pages,
                cache=torch.zeros(pages * H * page * (D + 8), dtype=torch.uint8, device=DEVICE),
                k_back=torch.empty(T, H, D, dtype=_dtype(case), device=DEVICE),
                v_back=torch.empty(T, H, D, dtype=_dtype(case), device=DEVICE))


def _prepare_attend(case, g):
    R, H, D, page = case["requests"], case["kv_heads"], case["dim"], case["page"]
    past, fresh = (_shuffled(g, v) for v in _lengths(case))
    kv_len = past + fresh
    need = (kv_len + page - 1) // page
    width = int(need.max())
    pages = int(need.sum()) + 1
    table, _ = _table(g, need, width, pages)
    T = int(fresh.sum())
    cache = torch.empty(pages, H, page * (D + 8), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 26) // (H * page * D))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        cache[at:at + n] = _pack(torch.randn(2, n, H, page, D, generator=g, device=DEVICE))
    q_start = torch.zeros(R + 1, dtype=torch.int32, device=DEVICE)
    q_start[1:] = torch.cumsum(fresh, 0)
    q = torch.randn(T, case["heads"], D, generator=g, device=DEVICE).to(_dtype(case))
    return dict(q=q, cache=cache.view(-1), pages=pages, table=table, q_start=q_start, kv_len=kv_len.int(),
                max_q=int(fresh.max()), scale=1 / math.sqrt(D), out=torch.empty_like(q))


def _prepare_logits(case, g):
    B, V = case["rows"], case["vocab"]
    x = (3 * torch.randn(B, V, generator=g, device=DEVICE) - 2).to(_dtype(case))

    def rows(most, floor):
        n = _ints(g, min(floor, most), most, B)
        start = torch.zeros(B + 1, dtype=torch.int32, device=DEVICE)
        start[1:] = torch.cumsum(n, 0)
        # A text's token numbers: small ones often, large ones seldom.
        ids = (V * torch.rand(int(n.sum()), generator=g, device=DEVICE) ** 4).int().clamp(max=V - 1)
        return ids, start

    prompt, output, bias = rows(case["prompt"], 1), rows(case["output"], 0), rows(case["biases"], 0)
    words = (V + 31) // 32
    mask = torch.randint(-2 ** 31, 2 ** 31, (B, words), generator=g, device=DEVICE, dtype=torch.int64).int()
    mask_row = torch.arange(B, device=DEVICE, dtype=torch.int32)
    mask_row[1::4] = -1  # requests without a grammar
    u = torch.rand(3, B, generator=g, device=DEVICE)
    return dict(x=x, prompt=prompt, output=output, bias=bias,
                bias_value=2 * torch.randn(bias[0].numel(), generator=g, device=DEVICE), mask=mask,
                mask_row=mask_row, repetition=1 + 0.3 * u[0], presence=u[1] - 0.25, frequency=u[2] - 0.25,
                out=torch.empty_like(x))


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return dict(plan=_own_plan, store=_own_store, attend=_own_attend, logits=_own_logits)[op](state)
    return dict(plan=_plain_plan, store=_plain_store, attend=_plain_attend, logits=_plain_logits)[op](state)


def _library():
    import bit_matvec_lb_gb300 as lb
    return lb


def _own_plan(s):
    lb, c = _library(), s["case"]
    lb.lb_kv_plan(s["past"], s["fresh"], c["requests"], s["free"], s["free"].numel(), None, c["page"],
                  s["table"], s["width"], s["tokens"], s["q_start"], s["kv_len"], s["position"], s["slot"],
                  s["counts"])
    return [s["table"], s["q_start"], s["kv_len"], s["position"], s["slot"], s["counts"]]


def _own_store(s):
    lb, c = _library(), s["case"]
    fmt = lb.OUT_F32 if c["type"] == "f32" else lb.OUT_BF16
    lb.lb_kv4_append(s["k"], s["v"], fmt, s["k"].stride(0), s["v"].stride(0), s["slot"], c["tokens"],
                     s["cache"], s["pages"], c["page"], c["kv_heads"], c["dim"])
    lb.lb_dequantize_kv4(s["cache"], s["pages"], c["page"], c["kv_heads"], c["dim"], s["slot"], c["tokens"],
                         fmt, s["k_back"], s["v_back"])
    return [s["k_back"], s["v_back"]]


def _own_attend(s):
    lb, c = _library(), s["case"]
    if "workspace" not in s:
        n = lb.lb_attn_kv4_workspace_bytes(c["heads"], c["kv_heads"], c["dim"], s["max_q"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEVICE)
    lb.lb_attn_kv4(s["q"], lb.OUT_F32 if c["type"] == "f32" else lb.OUT_BF16, s["q"].stride(0), s["cache"],
                   s["pages"], c["page"], c["heads"], c["kv_heads"], c["dim"], s["table"], s["table"].shape[1],
                   s["q_start"], s["kv_len"], c["requests"], s["q"].shape[0], s["max_q"], s["scale"], True,
                   c["window"], s["out"], s["out"].stride(0), None, s["workspace"])
    return s["out"]


def _own_logits(s):
    lb, c = _library(), s["case"]
    lb.lb_logits_adjust(s["x"], lb.OUT_F32 if c["type"] == "f32" else lb.OUT_BF16, s["x"].stride(0), s["out"],
                        s["out"].stride(0), c["rows"], c["vocab"], prompt_ids=s["prompt"][0],
                        prompt_start=s["prompt"][1], output_ids=s["output"][0], output_start=s["output"][1],
                        repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                        bias_ids=s["bias"][0], bias_values=s["bias_value"], bias_start=s["bias"][1],
                        mask=s["mask"] if c["grammar"] else None, mask_stride=s["mask"].shape[1],
                        mask_row=s["mask_row"] if c["grammar"] else None)
    return s["out"]


def _plain_plan(s):
    page, T, table = s["case"]["page"], s["tokens"], s["table"]
    past, fresh = s["past"].long(), s["fresh"].long()
    have = (past + page - 1) // page
    take = (past + fresh + page - 1) // page - have
    first = torch.cumsum(take, 0) - take
    q_start = torch.zeros(past.numel() + 1, dtype=torch.int64, device=DEVICE)
    q_start[1:] = torch.cumsum(fresh, 0)
    col = torch.arange(s["width"], device=DEVICE)
    new = col - have[:, None]
    at = (first[:, None] + new).clamp(0, s["free"].numel() - 1)
    table = torch.where((new >= 0) & (new < take[:, None]), s["free"][at], table)
    t = torch.arange(T, device=DEVICE)
    r = torch.searchsorted(q_start[1:], t, right=True).clamp(max=past.numel() - 1)
    live = t < q_start[-1]
    position = torch.where(live, past[r] + t - q_start[r], -1)
    slot = torch.where(live, table[r, (position // page).clamp(min=0)].long() * page + position % page, -1)
    counts = torch.stack([q_start[-1], take.sum()])
    return [table, q_start.int(), (past + fresh).int(), position.int(), slot, counts.int()]


def _codes(x):
    """4-bit codes of fp32 rows: (codes as fp32, d as fp16, z as fp32), one d and z per row."""
    lo, hi = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
    d = ((hi - lo) / torch.full_like(hi, 15)).clamp(max=65504).half()
    some = d > 0
    inv = torch.where(some, torch.ones_like(hi) / torch.where(some, d.float(), 1), 0)
    z = torch.round(-lo * inv).clamp(0, 15)
    return (torch.round(x * inv) + z).clamp(0, 15), d, z


def _pack(kv):
    """Cache pages [n][H][page * (D + 8)] of keys and values kv [2][n][H][page][D]."""
    _, n, H, page, D = kv.shape
    c, d, z = _codes(kv)
    c = c.to(torch.uint8).view(2, n, H, page // CHUNK, CHUNK, D // 2, 2)
    rows = (c[..., 0] | (c[..., 1] << 4)).flatten(4)
    pairs = torch.cat([d, z.half()], -1).contiguous().view(torch.uint8)
    pairs = pairs.view(2, n, H, page // CHUNK, CHUNK * 4)
    return torch.cat([rows[0], rows[1], pairs[0], pairs[1]], -1).flatten(2)


def _unpack(chunks, D):
    """fp32 keys and values [..., 16, D] of whole chunks [..., 16 * (D + 8)]."""
    n = CHUNK * D // 2
    out = []
    for at, pair in ((0, 2 * n), (n, 2 * n + 4 * CHUNK)):
        b = chunks[..., at:at + n].unflatten(-1, (CHUNK, D // 2))
        c = torch.stack([b & 15, b >> 4], -1).flatten(-2).float()
        dz = chunks[..., pair:pair + 4 * CHUNK].contiguous().view(torch.float16).unflatten(-1, (CHUNK, 2)).float()
        out.append((c - dz[..., 1:]) * dz[..., :1])
    return out


def _plain_store(s):
    c = s["case"]
    T, H, D, page = c["tokens"], c["kv_heads"], c["dim"], c["page"]
    cache = s["cache"].view(s["pages"], H, page // CHUNK, CHUNK * (D + 8))
    codes, d, z = _codes(torch.stack([s["k"].float(), s["v"].float()]))
    codes = codes.to(torch.uint8)
    rows = codes[..., 0::2] | (codes[..., 1::2] << 4)
    pairs = torch.cat([d, z.half()], -1).contiguous().view(torch.uint8)
    p, chunk, i = s["slot"] // page, s["slot"] % page // CHUNK, s["slot"] % CHUNK
    n = CHUNK * D // 2
    h = torch.arange(H, device=DEVICE)
    at = (p[:, None, None], h[None, :, None], chunk[:, None, None])
    j, j4 = torch.arange(D // 2, device=DEVICE), torch.arange(4, device=DEVICE)
    cache[at + (i[:, None, None] * (D // 2) + j,)] = rows[0]
    cache[at + (n + i[:, None, None] * (D // 2) + j,)] = rows[1]
    cache[at + (2 * n + i[:, None, None] * 4 + j4,)] = pairs[0]
    cache[at + (2 * n + 4 * CHUNK + i[:, None, None] * 4 + j4,)] = pairs[1]
    k, v = _unpack(cache[p, :, chunk], D)
    t = torch.arange(T, device=DEVICE)
    return [k[t, :, i].to(_dtype(c)), v[t, :, i].to(_dtype(c))]


def _plain_attend(s):
    c = s["case"]
    R, H, D, page, q = c["requests"], c["kv_heads"], c["dim"], c["page"], s["q"]
    G = c["heads"] // H
    kv_len, start = s["kv_len"].long(), s["q_start"].long()
    fresh = start[1:] - start[:-1]
    mq, width = s["max_q"], s["table"].shape[1]
    cache = s["cache"].view(s["pages"], H, page // CHUNK, CHUNK * (D + 8))
    k, v = _unpack(cache[s["table"].long().clamp(min=0)], D)  # [R][width][H][chunks][16][D]
    k = k.permute(0, 2, 1, 3, 4, 5).reshape(R, H, width * page, D)
    v = v.permute(0, 2, 1, 3, 4, 5).reshape(R, H, width * page, D)
    i = torch.arange(mq, device=DEVICE)
    row = (start[:-1, None] + i).clamp(max=q.shape[0] - 1)
    qr = q[row].float().view(R, mq, H, G, D).permute(0, 2, 3, 1, 4).reshape(R, H, G * mq, D)
    sc = torch.matmul(qr, k.transpose(2, 3)).view(R, H, G, mq, -1) * s["scale"]
    pos = (kv_len - fresh)[:, None] + i
    j = torch.arange(width * page, device=DEVICE)
    see = (j <= pos[:, :, None]) & (j < kv_len[:, None, None])
    if c["window"]:
        see &= j > pos[:, :, None] - c["window"]
    sc.masked_fill_(~see[:, None, None], -math.inf)
    sc -= sc.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    sc.exp_()
    total = sc.sum(-1, keepdim=True)
    o = torch.matmul(sc.view(R, H, G * mq, -1), v).view(R, H, G, mq, D)
    o = torch.where(total > 0, o / total, 0).permute(0, 3, 1, 2, 4).reshape(R, mq, H * G, D)
    return o[i < fresh[:, None]].to(q.dtype)


def _plain_logits(s):
    c = s["case"]
    B, V = c["rows"], c["vocab"]
    x = s["x"].float()

    def row_of(start):
        return torch.repeat_interleave(torch.arange(B, device=DEVICE), (start[1:] - start[:-1]).long())

    def count(ids, start):
        n = torch.zeros(B, V, dtype=torch.int32, device=DEVICE)
        return n.index_put_((row_of(start), ids.long()), torch.ones_like(ids), accumulate=True)

    prompt, output = count(*s["prompt"]), count(*s["output"])
    rep = s["repetition"][:, None]
    x = torch.where((prompt > 0) | (output > 0), torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * output - torch.where(output > 0, s["presence"][:, None], 0)
    if s["bias"][0].numel():
        # a token listed twice in a row has the later entry's bias
        ids, start = s["bias"]
        last = torch.full((B * V,), -1, dtype=torch.int64, device=DEVICE)
        last.scatter_reduce_(0, row_of(start) * V + ids, torch.arange(ids.numel(), device=DEVICE), "amax")
        last = last.view(B, V)
        x = x + torch.where(last >= 0, s["bias_value"][last.clamp(min=0)], 0)
    if c["grammar"]:
        t = torch.arange(V, device=DEVICE)
        bit = (s["mask"][s["mask_row"].long().clamp(min=0)][:, t // 32] >> (t % 32)) & 1
        x = torch.where((bit == 0) & (s["mask_row"][:, None] >= 0), -math.inf, x)
    return x.to(_dtype(c))


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------
def work(case):
    size = 4 if case.get("type") == "f32" else 2
    if case["op"] == "plan":
        # past is uniform: a token opens a page once in page times.
        R, T = case["requests"], sum(_fresh(case))
        return dict(bytes=8 * R + 2 * 4 * T / case["page"] + (T + case["spare"]) * 12 + 8 * R, flops=0)
    if case["op"] == "store":
        n = 2 * case["tokens"] * case["kv_heads"]
        return dict(bytes=n * (2 * case["dim"] * size + case["dim"] // 2 + 4) + 8 * case["tokens"],
                    flops=6 * n * case["dim"])
    if case["op"] == "logits":
        B, V = case["rows"], case["vocab"]
        sparse = 4 * ((case["prompt"] + case["output"]) / 2 + case["biases"])
        return dict(bytes=B * (2 * V * size + sparse + (V / 8 * 3 / 4 if case["grammar"] else 0)), flops=5 * B * V)
    H, D, w = (case[k] for k in ("kv_heads", "dim", "window"))
    rows = kv = seen = 0
    for p, f in zip(*_lengths(case)):  # paired as they fall; the seed pairs them otherwise
        rows += f
        kv += min(p + f, w - 1 + f) if w else p + f
        seen += f * (min(p + (f + 1) / 2, w) if w else p + (f + 1) / 2)
    return dict(bytes=2 * rows * case["heads"] * D * size + kv * H * (D + 8),
                flops=4 * seen * case["heads"] * D)


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return dict(store=_exact_store, attend=_exact_attend, logits=_exact_logits)[case["op"]](s)


def _exact_store(s):
    out = []
    for x in (s["k"].double(), s["v"].double()):
        top = torch.maximum(x.max(-1).values, x.new_zeros(()))[..., None]
        low = torch.minimum(x.min(-1).values, x.new_zeros(()))[..., None]
        d = torch.minimum((top - low) / 15, x.new_full((), 65504)).to(torch.float16).double()
        z = torch.round(-low / d)
        c = torch.minimum(torch.maximum(torch.round(x / d) + z, x.new_zeros(())), x.new_full((), 15))
        out.append(torch.where(d == 0, 0, d * (c - z)))
    return out


def _exact_attend(s):
    c, q = s["case"], s["q"].double()
    H, D, page = c["kv_heads"], c["dim"], c["page"]
    G = c["heads"] // H
    out = torch.zeros_like(q)
    raw = s["cache"].view(s["pages"], H, page // 16, 16 * (D + 8))
    for r in range(c["requests"]):
        a, b, n = int(s["q_start"][r]), int(s["q_start"][r + 1]), int(s["kv_len"][r])
        mine = raw[s["table"][r, :(n + page - 1) // page].long()]
        for h in range(H):
            part = mine[:, h].reshape(-1, 16 * (D + 8))
            both = part[:, :16 * D].reshape(-1, 2, 16, D // 2)
            code = torch.empty(part.shape[0], 2, 16, D, dtype=torch.float64, device=q.device)
            code[..., 0::2], code[..., 1::2] = both.remainder(16).double(), (both // 16).double()
            pair = part[:, 16 * D:].contiguous().view(torch.float16).reshape(-1, 2, 16, 2).double()
            value = pair[..., :1] * (code - pair[..., 1:])
            k, v = value[:, 0].reshape(-1, D)[:n], value[:, 1].reshape(-1, D)[:n]
            where = torch.arange(n, device=q.device)
            for at in range(a, b, 1024):
                rows = q[at:min(at + 1024, b), h * G:(h + 1) * G]
                at_pos = n - (b - a) + (torch.arange(at, at + rows.shape[0], device=q.device) - a)
                hidden = where > at_pos[:, None]
                if c["window"]:
                    hidden |= where <= at_pos[:, None] - c["window"]
                score = torch.einsum("tgd,nd->tgn", rows, k) * s["scale"]
                p = torch.softmax(score.masked_fill(hidden[:, None], -math.inf), -1)
                out[at:at + rows.shape[0], h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", p, v)
    return out


def _exact_logits(s):
    c, rows = s["case"], []
    for b in range(c["rows"]):
        x = s["x"][b].double()
        tokens = {}
        for k in ("prompt", "output", "bias"):
            ids, start = s[k]
            tokens[k] = ids[int(start[b]):int(start[b + 1])].long()
        seen = torch.unique(torch.cat([tokens["prompt"], tokens["output"]]))
        rep = s["repetition"][b].double()
        x[seen] = torch.where(x[seen] > 0, x[seen] / rep, x[seen] * rep)
        ids, times = torch.unique(tokens["output"], return_counts=True)
        x[ids] -= s["presence"][b].double() + s["frequency"][b].double() * times
        first = int(s["bias"][1][b])
        later = {int(t): first + i for i, t in enumerate(tokens["bias"].tolist())}
        if later:
            at = torch.tensor(list(later.items()), device=x.device)
            x[at[:, 0]] += s["bias_value"][at[:, 1]].double()
        row = int(s["mask_row"][b])
        if c["grammar"] and row >= 0:
            word = s["mask"][row].long()
            allowed = ((word[:, None] >> torch.arange(32, device=x.device)) & 1).flatten()[:c["vocab"]]
            x[allowed == 0] = -math.inf
        rows.append(x)
    return torch.stack(rows)
