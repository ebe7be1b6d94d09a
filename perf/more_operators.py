"""Measured cases of the operators for many continuations of one prompt: attention of a batch of sequences
that share a long prefix, and the draw of each one's next token from its logits.

Each case is one pass through one operator.  ``run`` computes it in plain torch operations; with ``own`` set
it makes the calls of the package instead.

Attention: query row i of sequence b sees the prefix [0, prefix_len), its sequence's own cached positions
[0, lens[b]), and of the rows drafted behind them the ones that its mask names.  Caches in 8 bits are int8
codes in groups of 32 with one fp16 scale.

Draw: tokens in order of falling logit x (ties by rising id), weights exp((x - max) / temperature); the first
top_k of them; of those the shortest head that holds at least top_p of their weight; of that the ones whose
weight is at least min_p of the greatest; then the first whose running weight exceeds u times what is left.
Temperature 0 takes the greatest logit.  Where a running weight meets its border decides a whole token, so the
plain form adds the weights in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases

def _prefix(name, n_seq, nodes, dtype, kv, prefix, ctx, ragged, heads=8, group=2, dim=128):
    return {"name": name, "op": "prefix", "n_seq": n_seq, "nodes": nodes, "dtype": dtype, "kv": kv, "prefix": prefix,
            "ctx": ctx, "ragged": ragged, "heads": heads, "group": group, "dim": dim}


def _sample(name, rows, vocab, dtype, mode):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "mode": mode}


def listed():
    return [
        # a batch of eight right after it was forked from a 512-token prompt: fp16 queries over f32 caches
        _prefix("prefix 8x1 f16 f32 512+64", 8, 1, "f16", "f32", 512, 63, True),
        # f32 throughout, 64-wide heads in groups of three, odd lengths
        _prefix("prefix 5x1 f32 f32 1001+33", 5, 1, "f32", "f32", 1001, 33, True, heads=5, group=3, dim=64),
        # sixteen requests over one system prompt, each checking a tree of five drafted tokens, 8-bit caches
        _prefix("prefix 16x5 f16 int8 2048+500", 16, 5, "f16", "int8", 2048, 500, True),
        # the batch of eight later on: a long prompt, a few hundred tokens of its own each
        _prefix("prefix 8x1 f16 f32 4096+300", 8, 1, "f16", "f32", 4096, 300, True),
        # 64 continuations of one prompt, bf16 throughout
        _prefix("prefix 64x1 bf16 4096+256", 64, 1, "bf16", "bf16", 4096, 256, True),
        # a document of 32K tokens in 8 bits, 32 questions about it
        _prefix("prefix 32x1 bf16 int8 32768+512", 32, 1, "bf16", "int8", 32768, 512, True),
        # the largest: 256 continuations of the 32K context
        _prefix("prefix 256x1 bf16 32768+128", 256, 1, "bf16", "bf16", 32768, 128, False),
        # one request of the small test model
        _sample("sample 1x8192", 1, 8192, "f32", "usual"),
        # a batch's step at the full vocabulary
        _sample("sample 8x151936", 8, 151936, "f32", "usual"),
        # the same drawn from nearly everything: high temperature, no top-k
        _sample("sample 8x151936 flat", 8, 151936, "f32", "flat"),
        # 64 requests, logits in bf16, whose values often tie
        _sample("sample 64x151936 bf16", 64, 151936, "bf16", "mixed"),
        # the largest: 256 requests, each with settings of its own
        _sample("sample 256x151936", 256, 151936, "f32", "mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.45:
        case = _sample("", _log(rng, 1, 256), _log(rng, 1000, 151936), rng.choice(["f32", "f32", "bf16", "f16"]),
                       rng.choice(["usual", "mixed", "mixed", "flat"]))
    else:
        heads, group, dim = rng.choice([(8, 2, 128), (8, 2, 128), (8, 1, 128), (4, 4, 128), (2, 7, 128), (8, 2, 64), (5, 3, 64)])
        dtype, kv = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "int8"), ("f16", "int8"), ("f16", "f32"),
                                ("f16", "bf16"), ("f32", "f32"), ("f32", "int8"), ("f32", "bf16"), ("bf16", "f32")])
        n_seq, nodes = _log(rng, 1, 256), _log(rng, 1, 8)
        if n_seq * nodes > 256 or rng.random() < 0.5:
            nodes = 1
        # f32 queries are for small models and checks: shorter contexts
        prefix = _log(rng, 1, 4096 if dtype == "f32" else 32768)
        ctx = _log(rng, 1, max(2, min(2048, 32768 // n_seq)))
        case = _prefix("", n_seq, nodes, dtype, kv, prefix, ctx, rng.random() < 0.6, heads, group, dim)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randint(g, lo, hi, shape):
    """Whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _uniform(g, lo, hi, shape):
    return lo + (hi - lo) * torch.rand(shape, generator=g, device="cuda")


def _cache(g, shape, kv):
    """K, V and their scales (None but for int8)."""
    if kv == "int8":
        k, v = (torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
        ks, vs = ((0.01 + 0.02 * torch.rand(shape[:-1] + (shape[-1] // 32,), generator=g, device="cuda")).half()
                  for _ in range(2))
        return k, v, ks, vs
    k, v = (torch.randn(shape, generator=g, device="cuda").to(DTYPES[kv]) for _ in range(2))
    return k, v, None, None


def prepare(case, seed):
    g = _generator(seed)
    return _prepare_sample(case, g) if case["op"] == "sample" else _prepare_prefix(case, g)


def _prepare_prefix(case, g):
    B, n, H, G, D = case["n_seq"], case["nodes"], case["heads"], case["group"], case["dim"]
    s = {"op": "prefix", "group": G, "max_len": case["ctx"], "max_prefix": case["prefix"], "scale": 1.0 / math.sqrt(D)}
    # both caches have room behind what they hold, as a program's have
    s["pk"], s["pv"], s["pks"], s["pvs"] = _cache(g, (1, H, case["prefix"] + 16, D), case["kv"])
    s["k"], s["v"], s["ks"], s["vs"] = _cache(g, (B, H, case["ctx"] + n, D), case["kv"])
    s["prefix_len"] = torch.full((1,), case["prefix"], dtype=torch.int32, device="cuda")
    if case["ragged"]:
        s["lens"] = _randint(g, 0, case["ctx"], (B,))
        s["counts"] = _randint(g, 1, n, (B,))
    else:
        s["lens"] = torch.full((B,), case["ctx"], dtype=torch.int32, device="cuda")
        s["counts"] = torch.full((B,), n, dtype=torch.int32, device="cuda")
    dt = DTYPES[case["dtype"]]
    s["q"] = (2.0 * torch.randn((B, n, H * G, D), generator=g, device="cuda")).to(dt)
    # each drafted token continues an earlier one (or the cache): bit j of mask[i] = row i sees drafted row j
    parent = (torch.rand((B, n), generator=g, device="cuda") * torch.arange(n, device="cuda")).long() \
        - (torch.rand((B, n), generator=g, device="cuda") < 0.2).long()
    mask = torch.zeros((B, n), dtype=torch.int64, device="cuda")
    for i in range(n):
        up = torch.gather(mask, 1, parent[:, i:i + 1].clamp(min=0)).squeeze(1) if i else mask[:, 0]
        mask[:, i] = torch.where(parent[:, i] >= 0, up, torch.zeros_like(up)) | (1 << i)
    s["mask"] = mask
    s["out"] = torch.zeros((B, n, H * G, D), device="cuda", dtype=dt)
    if own:  # what a program keeps: the caches' descriptions, and the attention's workspace
        from runtime_qwen3_decode_gb300 import qw
        s["prefix"] = qw.KvView(s["pk"], s["pv"], s["pks"], s["pvs"])
        s["view"] = qw.KvView(s["k"], s["v"], s["ks"], s["vs"])
        s["scratch"] = qw.prefix_attention_scratch(s["prefix"], s["view"], n, H * G, max_len=s["max_len"],
                                                   max_prefix=s["max_prefix"])
    return s


def _prepare_sample(case, g):
    R, V, mode = case["rows"], case["vocab"], case["mode"]
    # a bulk of unlikely tokens, and up to 64 that the model considers, some rows surer of them than others
    x = 2.0 * torch.randn((R, V), generator=g, device="cuda")
    n = min(64, V)
    ids = (_randint(g, 0, V - 1, (R, 1)) + _randint(g, 1, V // n, (R, 1)) * torch.arange(n, device="cuda")) % V
    sure = _uniform(g, 6.0, 16.0, (R, 1))
    x.scatter_(1, ids, sure - 2.0 * torch.log1p(torch.arange(n, device="cuda").float()) +
               0.5 * torch.randn((R, n), generator=g, device="cuda"))
    banned = torch.rand((R, V), generator=g, device="cuda") < 0.01   # as a grammar's mask leaves them
    x = torch.where(banned, torch.full((), -math.inf, device="cuda"), x)
    s = {"op": "sample", "logits": x.to(DTYPES[case["dtype"]]), "u": torch.rand((R,), generator=g, device="cuda")}
    if mode == "usual":
        s["temperature"] = _uniform(g, 0.6, 1.0, (R,))
        s["top_k"] = _randint(g, 20, 60, (R,))
        s["top_p"] = _uniform(g, 0.8, 0.95, (R,))
        s["min_p"] = torch.zeros((R,), device="cuda")
    elif mode == "flat":
        s["temperature"] = _uniform(g, 1.2, 2.0, (R,))
        s["top_k"] = torch.zeros((R,), dtype=torch.int32, device="cuda")
        s["top_p"] = torch.full((R,), 0.98, device="cuda")
        s["min_p"] = torch.zeros((R,), device="cuda")
    else:
        def pick(p, a, b):
            return torch.where(torch.rand((R,), generator=g, device="cuda") < p, a, b)
        s["temperature"] = pick(0.1, torch.zeros((R,), device="cuda"), _uniform(g, 0.3, 1.5, (R,)))
        s["top_k"] = torch.where(torch.rand((R,), generator=g, device="cuda") < 0.4, torch.zeros((), dtype=torch.int32, device="cuda"),
                                 _randint(g, 1, min(V, 2000), (R,)))
        s["top_p"] = pick(0.3, torch.ones((R,), device="cuda"), _uniform(g, 0.3, 0.99, (R,)))
        s["min_p"] = pick(0.5, torch.zeros((R,), device="cuda"), _uniform(g, 0.01, 0.3, (R,)))
    s["tokens"], s["kept"] = (torch.zeros((R,), dtype=torch.int32, device="cuda") for _ in range(2))
    s["probs"] = torch.zeros((R,), device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return _plain_sample(s) if s["op"] == "sample" else _plain_prefix(s)


def _run_own(s):
    from runtime_qwen3_decode_gb300 import qw
    if s["op"] == "sample":
        qw.sample_rows(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                       min_p=s["min_p"], tokens=s["tokens"], probs=s["probs"], kept=s["kept"])
        return {"tokens": s["tokens"], "probs": s["probs"], "kept": s["kept"]}
    return qw.prefix_attention(s["prefix"], s["view"], s["q"], s["lens"], s["prefix_len"], mask=s["mask"], out=s["out"],
                               counts=s["counts"], max_len=s["max_len"], max_prefix=s["max_prefix"], scale=s["scale"],
                               scratch=s["scratch"])


def _plain_rows(x, scale):
    x = x.float()
    return x if scale is None else (x.unflatten(-1, (-1, 32)) * scale.float().unsqueeze(-1)).flatten(-2)


def _plain_prefix(s):
    B, n, heads, D = s["q"].shape
    G, P = s["group"], s["max_prefix"]
    H = heads // G
    q = s["q"].float().view(B, n, H, G, D).permute(2, 0, 1, 3, 4)                 # [H, B, n, G, D]
    # the prefix once for all rows, each sequence's own positions beside it
    shared = torch.matmul(q.reshape(H, B * n * G, D), _plain_rows(s["pk"], s["pks"])[0, :, :P].transpose(-1, -2))
    each = torch.matmul(q.transpose(0, 1).reshape(B, H, n * G, D), _plain_rows(s["k"], s["ks"]).transpose(-1, -2))
    end = each.shape[-1]
    j = torch.arange(end, device="cuda")[None, :] - s["lens"][:, None]             # drafted index of a position
    bit = (s["mask"][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
    sees = (j < 0)[:, None, :] | ((j >= 0) & (j < s["counts"][:, None]))[:, None, :] & (bit != 0)  # [B, n, end]
    low = torch.full((), -math.inf, device="cuda")
    each = torch.where(sees[:, None, :, None, :], each.mul_(s["scale"]).view(B, H, n, G, end), low).view(B, H, n * G, end)
    inside = torch.arange(P, device="cuda") < s["prefix_len"]
    shared = torch.where(inside, shared.mul_(s["scale"]), low).view(H, B, n * G, P)
    top = torch.maximum(shared.amax(-1).transpose(0, 1), each.amax(-1))             # [B, H, n G]
    shared = torch.exp(shared.sub_(top.transpose(0, 1).unsqueeze(-1)))
    each = torch.exp(each.sub_(top.unsqueeze(-1)))
    o = torch.matmul(shared.view(H, B * n * G, P), _plain_rows(s["pv"], s["pvs"])[0, :, :P]).view(H, B, n * G, D).transpose(0, 1)
    o = o + torch.matmul(each, _plain_rows(s["v"], s["vs"]))
    o = o / (shared.sum(-1).transpose(0, 1) + each.sum(-1)).unsqueeze(-1)
    o = o.view(B, H, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, heads, D).to(s["out"].dtype)
    live = (torch.arange(n, device="cuda") < s["counts"][:, None])[:, :, None, None]
    s["out"].copy_(torch.where(live, o, s["out"]))
    return s["out"]


def _plain_sample(s):
    x = s["logits"].float()
    R, V = x.shape
    val, ids = torch.sort(x, dim=1, descending=True, stable=True)
    there = val > -math.inf
    t = s["temperature"].double()[:, None]
    z = (val.double() - val[:, :1].double()) / torch.where(t > 0, t, torch.ones_like(t))
    at = torch.arange(V, device="cuda")[None, :]
    k = torch.where(s["top_k"] > 0, s["top_k"], torch.full_like(s["top_k"], V))[:, None]
    w = torch.where(there & (at < k), torch.exp(z), torch.zeros((), dtype=torch.float64, device="cuda"))
    cum = torch.cumsum(w, 1)
    # kept: inside top-k, not behind the place where top_p is reached, not below min_p of the greatest
    keep = there & (at < k) & (w >= s["min_p"].double()[:, None])
    p = s["top_p"].double()[:, None]
    keep &= (p >= 1) | (at == 0) | (torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], 1) < p * cum[:, -1:])
    keep = torch.where(t > 0, keep, at == 0)
    n = keep.sum(1, keepdim=True)
    total = torch.gather(cum, 1, n - 1)
    hit = (cum > s["u"].double()[:, None] * total) & keep
    j = torch.where(hit.any(1, keepdim=True), hit.int().argmax(1, keepdim=True), n - 1)
    j = torch.where(t > 0, j, torch.zeros_like(j))
    s["tokens"].copy_(torch.gather(ids, 1, j).squeeze(1))
    s["kept"].copy_(n.squeeze(1))
    s["probs"].copy_(torch.where(t > 0, torch.gather(w, 1, j) / total, torch.ones_like(total)).squeeze(1))
    return {"tokens": s["tokens"], "probs": s["probs"], "kept": s["kept"]}


# ---------------------------------------------------------------- work

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "sample":
        R, V = case["rows"], case["vocab"]
        return {"bytes": R * V * e + 32 * R, "flops": 4 * R * V}
    B, H, D, G = case["n_seq"], case["heads"], case["dim"], case["group"]
    row = {"int8": D + D // 16, "bf16": 2 * D, "f32": 4 * D}[case["kv"]]
    half = 0.5 if case["ragged"] else 1.0      # of what a sequence may have that an average one has
    nodes = (case["nodes"] + 1) / 2 if case["ragged"] else case["nodes"]
    keys = case["ctx"] * half + nodes
    return {"bytes": 2 * H * row * (case["prefix"] + B * keys) + 2 * B * nodes * H * G * D * e,
            "flops": 4 * B * H * G * D * nodes * (case["prefix"] + keys)}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _exact_sample(s) if case["op"] == "sample" else _exact_prefix(s)


def _exact_prefix(s):
    B, n, heads, D = s["q"].shape
    P = int(s["prefix_len"])
    out = torch.zeros((B, n, heads, D), dtype=torch.float64, device="cuda")

    def wide(name, *at):
        x = s[name][at].double()
        return x if s[name + "s"] is None else x * s[name + "s"][at].double().repeat_interleave(32, -1)

    lens, counts = s["lens"].tolist(), s["counts"].tolist()
    masks = s["mask"].tolist()
    sees = [torch.tensor([[(m >> j) & 1 for j in range(c)] for m in row[:c]], device="cuda").bool()
            for row, c in zip(masks, counts)]
    for h in range(heads // s["group"]):
        pk, pv = wide("pk", 0, h, slice(0, P)), wide("pv", 0, h, slice(0, P))
        for b in range(B):
            end = lens[b] + counts[b]
            k = torch.cat([pk, wide("k", b, h, slice(0, end))])
            v = torch.cat([pv, wide("v", b, h, slice(0, end))])
            for g in range(s["group"]):
                z = (s["q"][b, :counts[b], h * s["group"] + g].double() @ k.T) * s["scale"]
                z[:, P + lens[b]:].masked_fill_(~sees[b], -math.inf)
                out[b, :counts[b], h * s["group"] + g] = torch.softmax(z, -1) @ v
    return out


def _exact_sample(s):
    R = s["logits"].shape[0]
    tokens, kept, probs = [], [], []
    for r in range(R):
        x = s["logits"][r].double()
        t, k, p, m, u = (float(s[name][r]) for name in ("temperature", "top_k", "top_p", "min_p", "u"))
        order = torch.argsort(x, descending=True, stable=True)
        order = order[x[order] > -math.inf]
        if t == 0:
            tokens.append(int(order[0]))
            kept.append(1)
            probs.append(1.0)
            continue
        if k > 0:
            order = order[:int(k)]
        w = torch.exp((x[order] - x[order[0]]) / t)
        if p < 1:
            n = int(torch.searchsorted(torch.cumsum(w, 0), p * w.sum().reshape(1))) + 1
            order, w = order[:n], w[:n]
        n = int((w >= m).sum())
        order, w = order[:n], w[:n]
        run_w = torch.cumsum(w, 0)
        j = min(int(torch.searchsorted(run_w, u * run_w[-1:], right=True)), n - 1)
        tokens.append(int(order[j]))
        kept.append(n)
        probs.append(float(w[j] / run_w[-1]))
    i32 = {"dtype": torch.int32, "device": "cuda"}
    return {"tokens": torch.tensor(tokens, **i32), "kept": torch.tensor(kept, **i32),
            "probs": torch.tensor(probs, dtype=torch.float64, device="cuda")}
