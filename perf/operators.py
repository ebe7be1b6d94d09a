"""Measured cases of the drafted-token operators: an 8-bit K/V cache that is written, read back and
attended to by a tree of drafted tokens, and the logits of the tree's nodes made ready for sampling.

Each case is one pass through one operator.  ``run`` computes it in plain torch operations in 32 bits;
with ``own`` set it makes the calls of the package instead.  Cache rows in 8 bits are int8 codes in
groups of 32 with one fp16 scale: d = amax / 127 in f32, code = round-half-away(a / d), scale = fp16(d),
value = code * scale.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of eight sequences of the 0.6B shape appends a row each, and reads it back
        {"name": "append 8x1 f32", "op": "append", "n_seq": 8, "heads": 8, "dim": 128, "ctx": 512, "rows": 1,
         "dtype": "f32", "layout": "head", "ragged": False},
        # drafted trees of up to 33 nodes of five sequences, bf16 rows as a projection leaves them (token-major)
        {"name": "append 5x33 bf16 ragged", "op": "append", "n_seq": 5, "heads": 8, "dim": 128, "ctx": 4000, "rows": 33,
         "dtype": "bf16", "layout": "token", "ragged": True},
        # a 2048-row prompt enters the cache
        {"name": "append 1x2048 f32", "op": "append", "n_seq": 1, "heads": 8, "dim": 128, "ctx": 2064, "rows": 2048,
         "dtype": "f32", "layout": "head", "ragged": False},
        # two sequences' rows leave the cache for another engine, 64-wide heads, odd count
        {"name": "read 2x1001 bf16", "op": "read", "n_seq": 2, "heads": 8, "dim": 64, "ctx": 1300, "rows": 1001,
         "dtype": "bf16", "layout": "token", "ragged": True},
        # the 32K context read back whole
        {"name": "read 1x32768 bf16", "op": "read", "n_seq": 1, "heads": 8, "dim": 128, "ctx": 32832, "rows": 32768,
         "dtype": "bf16", "layout": "head", "ragged": False},
        # plain batched decode: one token of eight sequences over f32 caches of up to 512 positions
        {"name": "tree 8x1 f32 ctx512", "op": "tree", "n_seq": 8, "heads": 8, "group": 2, "dim": 128, "ctx": 511,
         "nodes": 1, "dtype": "f32", "kv": "f32", "ragged": True},
        # one sequence verifies eight drafted tokens after a 2048-row prompt, 8-bit cache, fp16 queries
        {"name": "tree 1x8 f16 int8 ctx2048", "op": "tree", "n_seq": 1, "heads": 8, "group": 2, "dim": 128, "ctx": 2048,
         "nodes": 8, "dtype": "f16", "kv": "int8", "ragged": False},
        # sixteen requests with trees of up to 33 nodes and contexts of up to 4096, 8-bit caches
        {"name": "tree 16x33 bf16 int8 ctx4096", "op": "tree", "n_seq": 16, "heads": 8, "group": 2, "dim": 128, "ctx": 4096,
         "nodes": 33, "dtype": "bf16", "kv": "int8", "ragged": True},
        # the largest tree over the 32K context in bf16
        {"name": "tree 1x64 bf16 ctx32768", "op": "tree", "n_seq": 1, "heads": 8, "group": 2, "dim": 128, "ctx": 32768,
         "nodes": 64, "dtype": "bf16", "kv": "bf16", "ragged": False},
        # the small test model's vocabulary, one request
        {"name": "logits 1x8192", "op": "logits", "rows": 1, "vocab": 8192, "history": 24, "bias": 3, "masks": 1,
         "dtype": "f32"},
        # the nodes of one drafted tree at the full vocabulary
        {"name": "logits 8x151936", "op": "logits", "rows": 8, "vocab": 151936, "history": 700, "bias": 40, "masks": 8,
         "dtype": "f32"},
        # sixteen requests of sixteen nodes each
        {"name": "logits 256x151936", "op": "logits", "rows": 256, "vocab": 151936, "history": 2000, "bias": 300,
         "masks": 16, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "tree", "tree", "logits"])
    if op == "logits":
        vocab = _log(rng, 1000, 152000)
        rows = _log(rng, 1, 256)
        return {"op": op, "rows": rows, "vocab": vocab, "history": _log(rng, 1, 2000), "bias": rng.randint(0, 300),
                "masks": rng.randint(0, min(rows, 16)), "dtype": rng.choice(["f32", "f32", "bf16", "f16"])}
    heads, group, dim = rng.choice([(8, 2, 128), (8, 2, 128), (8, 1, 128), (4, 4, 128), (2, 7, 128), (8, 2, 64), (5, 3, 64)])
    if op == "tree":
        n_seq = _log(rng, 1, 16)
        ctx = _log(rng, 1, 32768 // n_seq)
        dtype, kv = rng.choice([("bf16", "bf16"), ("bf16", "int8"), ("f16", "int8"), ("f16", "f32"), ("f32", "f32"),
                                ("f32", "int8"), ("f16", "bf16"), ("f32", "bf16")])
        nodes = _log(rng, 1, 64)
        return {"op": op, "n_seq": n_seq, "heads": heads, "group": group, "dim": dim, "ctx": ctx, "nodes": nodes,
                "dtype": dtype, "kv": kv, "ragged": rng.random() < 0.6}
    n_seq = _log(rng, 1, 16)
    rows = _log(rng, 1, 16384 // n_seq)
    return {"op": op, "n_seq": n_seq, "heads": heads, "dim": dim, "ctx": rows + _log(rng, 1, 1000), "rows": rows,
            "dtype": rng.choice(["f32", "bf16", "f16"]), "layout": rng.choice(["head", "token"]),
            "ragged": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randint(g, lo, hi, shape, dtype=torch.int32):
    """Whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=dtype)


def _rows(g, case, dtype):
    """Keys or values [n_seq, heads, rows, dim]: a few dimensions stand out, as keys have them."""
    shape = (case["n_seq"], case["heads"], case["rows"], case["dim"])
    x = torch.randn(shape, generator=g, device="cuda")
    x = (x * (1 + 3 * (torch.arange(case["dim"], device="cuda") % 29 == 5))).to(dtype)
    if case["layout"] == "token":  # the same values, laid out [n_seq, rows, heads, dim]
        x = x.transpose(1, 2).contiguous().transpose(1, 2)
    return x


def _int8_cache(g, shape):
    codes = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
    scale = (0.01 + 0.02 * torch.rand(shape[:-1] + (shape[-1] // 32,), generator=g, device="cuda")).half()
    return codes, scale


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "logits":
        return _prepare_logits(case, g)
    B, H, D, ctx = case["n_seq"], case["heads"], case["dim"], case["ctx"]
    s = {"op": case["op"]}
    if case["op"] == "tree":
        n, ctx = case["nodes"], ctx + case["nodes"]
        s["n"], s["group"] = n, case["group"]
    else:
        n = case["rows"]
    shape = (B, H, ctx, D)
    kv = case.get("kv", "int8")
    if kv == "int8":
        (s["k"], s["ks"]), (s["v"], s["vs"]) = _int8_cache(g, shape), _int8_cache(g, shape)
    else:
        s["k"], s["v"] = (torch.randn(shape, generator=g, device="cuda").to(DTYPES[kv]) for _ in range(2))
        s["ks"] = s["vs"] = None
    room = ctx - n
    if case["ragged"]:
        s["count"] = _randint(g, 0 if B > 1 else 1, n, (B,))
        s["start"] = _randint(g, room // 3, room, (B,))
    else:
        s["count"] = torch.full((B,), n, dtype=torch.int32, device="cuda")
        s["start"] = torch.full((B,), room if case["op"] == "tree" else room // 2, dtype=torch.int32, device="cuda")
    dt = DTYPES[case["dtype"]]
    if case["op"] == "tree":
        heads = H * case["group"]
        s["q"] = (2.0 * torch.randn((B, n, heads, D), generator=g, device="cuda")).to(dt)
        # each node's parent is an earlier node (or the last cached token): bit j of mask[i] = node i sees node j
        parent = (torch.rand((B, n), generator=g, device="cuda") * torch.arange(n, device="cuda")).long() \
            - (torch.rand((B, n), generator=g, device="cuda") < 0.2).long()
        mask = torch.zeros((B, n), dtype=torch.int64, device="cuda")
        for i in range(n):
            up = torch.gather(mask, 1, parent[:, i:i + 1].clamp(min=0)).squeeze(1) if i else mask[:, 0]
            mask[:, i] = torch.where(parent[:, i] >= 0, up, torch.zeros_like(up)) | (1 << i if i < 63 else -(1 << 63))
        s["mask"] = mask
        s["out"] = torch.zeros((B, n, heads, D), device="cuda", dtype=dt)
        s["max_len"] = room
        s["scale"] = 1.0 / math.sqrt(D)
    else:
        if case["op"] == "append":
            s["k_new"], s["v_new"] = _rows(g, case, dt), _rows(g, case, dt)
            dt = torch.float32
        shape = (B, H, n, D) if case["layout"] == "head" else (B, n, H, D)
        s["k_out"], s["v_out"] = (torch.zeros(shape, device="cuda", dtype=dt) for _ in range(2))
        if case["layout"] == "token":
            s["k_out"], s["v_out"] = s["k_out"].transpose(1, 2), s["v_out"].transpose(1, 2)
    if own:  # what a program keeps: the cache's description, and the attention's workspace
        from runtime_qwen3_decode_gb300 import qw
        s["view"] = qw.KvView(s["k"], s["v"], s["ks"], s["vs"])
        if case["op"] == "tree":
            s["scratch"] = qw.tree_attention_scratch(s["view"], n, H * case["group"])
    return s


def _prepare_logits(case, g):
    R, V, h, nb, nm = case["rows"], case["vocab"], case["history"], case["bias"], case["masks"]
    s = {"op": "logits", "logits": (3.0 * torch.randn((R, V), generator=g, device="cuda")).to(DTYPES[case["dtype"]])}
    # requests of several rows (a tree's nodes) share their request's history and each has its own drafted path
    per = max(1, R // 16)
    nreq = -(-R // per)
    req = torch.arange(R, device="cuda") // per
    common = max(1, V // 50)  # text repeats itself: most tokens come from a small part of the vocabulary
    s["history"] = torch.where(torch.rand((nreq * h,), generator=g, device="cuda") < 0.7,
                               _randint(g, 0, common - 1, (nreq * h,)), _randint(g, 0, V - 1, (nreq * h,)))
    used = _randint(g, h // 2, h, (nreq,))
    s["range"] = torch.stack([req * h, req * h + used[req]], 1).int().contiguous()
    s["path"] = _randint(g, -1, V - 1, (R, 8))
    s["path"] = torch.where(torch.rand((R, 8), generator=g, device="cuda") < 0.4, torch.full_like(s["path"], -1), s["path"])
    s["penalties"] = torch.stack([1.0 + 0.3 * torch.rand((R,), generator=g, device="cuda"),
                                  torch.rand((R,), generator=g, device="cuda"),
                                  0.2 * torch.rand((R,), generator=g, device="cuda")], 1).contiguous()
    if nb:
        s["bias_ids"] = _randint(g, 0, V - 1, (nreq * nb,))
        s["bias"] = 4.0 * torch.randn((nreq * nb,), generator=g, device="cuda")
        s["bias_range"] = torch.stack([req * nb, req * nb + nb], 1).int().contiguous()
    else:
        s["bias_ids"] = s["bias"] = s["bias_range"] = None
    if nm:
        words = (V + 31) // 32
        m = torch.randint(-(1 << 31), 1 << 31, (nm, words), generator=g, device="cuda").int()
        s["mask"] = torch.where(_randint(g, 0, 3, (nm, 1)) == 0, m, m & m.roll(1, 1) & m.roll(2, 1))
        s["mask_index"] = torch.where(req % 5 == 4, torch.full_like(req, -1), req % nm).int()
    else:
        s["mask"] = s["mask_index"] = None
    s["out"] = torch.empty_like(s["logits"])
    s["longest"], s["longest_bias"] = h, nb
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "logits":
        return _plain_logits(s)
    if s["op"] == "tree":
        return _plain_tree(s)
    return _plain_append_read(s)


def _run_own(s):
    from runtime_qwen3_decode_gb300 import qw
    if s["op"] == "logits":
        qw.process_logits(s["logits"], s["out"], history=s["history"], history_range=s["range"], path=s["path"],
                          penalties=s["penalties"], bias_ids=s["bias_ids"], bias=s["bias"], bias_range=s["bias_range"],
                          mask=s["mask"], mask_index=s["mask_index"])
        return s["out"]
    if s["op"] == "tree":
        qw.tree_attention(s["view"], s["q"], s["mask"], s["start"], s["out"], counts=s["count"], max_len=s["max_len"],
                          scale=s["scale"], scratch=s["scratch"])
        return s["out"]
    if s["op"] == "append":
        qw.kv_append(s["view"], s["k_new"], s["v_new"], s["start"], s["count"])
    qw.kv_read(s["view"], s["k_out"], s["v_out"], s["start"], s["count"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_quantise(x):
    """f32 [..., dim] -> codes (as f32) and f32 group divisors."""
    b = x.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / b.new_full((1,), 127.0)  # a true division: torch multiplies by 1 / number
    r = torch.where(d > 0, b / d, torch.zeros_like(b))
    t = torch.trunc(r)
    codes = t + torch.sign(r) * ((r - t).abs() >= 0.5)
    return codes.clamp(-127, 127).flatten(-2), d.squeeze(-1)


def _plain_append_read(s):
    B, H, n, D = s["k_out"].shape
    at = s["start"].long()[:, None] + torch.arange(n, device="cuda")
    live = (torch.arange(n, device="cuda") < s["count"][:, None])[:, None, :, None]
    at = at[:, None, :, None].expand(B, H, n, 1)
    for new, codes, scales, out in (("k_new", "k", "ks", "k_out"), ("v_new", "v", "vs", "v_out")):
        cols, groups = at.expand(B, H, n, D), at.expand(B, H, n, D // 32)
        old_c, old_s = s[codes].gather(2, cols), s[scales].gather(2, groups)
        if s["op"] == "append":
            c, d = _plain_quantise(s[new].float())
            old_c, old_s = torch.where(live, c.to(torch.int8), old_c), torch.where(live, d.half(), old_s)
            s[codes].scatter_(2, cols, old_c)
            s[scales].scatter_(2, groups, old_s)
        val = (old_c.float().unflatten(-1, (-1, 32)) * old_s.float().unsqueeze(-1)).flatten(-2)
        s[out].copy_(torch.where(live, val.to(s[out].dtype), s[out]))
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_tree(s):
    B, n, heads, D = s["q"].shape
    G, end = s["group"], s["max_len"] + n
    k, v = s["k"][:, :, :end].float(), s["v"][:, :, :end].float()
    if s["ks"] is not None:
        k = (k.unflatten(-1, (-1, 32)) * s["ks"][:, :, :end].float().unsqueeze(-1)).flatten(-2)
        v = (v.unflatten(-1, (-1, 32)) * s["vs"][:, :, :end].float().unsqueeze(-1)).flatten(-2)
    H = heads // G
    q = s["q"].float().reshape(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    pos = torch.arange(end, device="cuda")
    j = pos[None, :] - s["start"][:, None]                                     # drafted index of a position
    bit = (s["mask"][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
    sees = (j < 0)[:, None, :] | ((j >= 0) & (j < s["count"][:, None]))[:, None, :] & (bit != 0)   # [B, n, end]
    sc = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    sc = torch.where(sees[:, None, :, None, :], sc.view(B, H, n, G, end), torch.full((), -math.inf, device="cuda"))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    o = torch.matmul(p.view(B, H, n * G, end), v) / p.sum(-1).view(B, H, n * G, 1)
    o = o.view(B, H, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, heads, D).to(s["out"].dtype)
    live = (torch.arange(n, device="cuda") < s["count"][:, None])[:, :, None, None]
    s["out"].copy_(torch.where(live, o, s["out"]))
    return s["out"]


def _plain_logits(s):
    x = s["logits"].float()
    R, V = x.shape
    # how often each row's history and drafted path name each token
    counts = torch.zeros((R, V + 1), dtype=torch.float32, device="cuda")
    h = torch.arange(s["longest"], device="cuda")
    at = s["range"][:, :1].long() + h
    ids = s["history"][at.clamp(max=s["history"].numel() - 1)].long()
    ids = torch.where(at < s["range"][:, 1:], ids, torch.full_like(ids, V))
    counts.scatter_add_(1, ids, torch.ones_like(ids, dtype=torch.float32))
    path = torch.where(s["path"] >= 0, s["path"], torch.full_like(s["path"], V)).long()
    counts.scatter_add_(1, path, torch.ones_like(path, dtype=torch.float32))
    counts = counts[:, :V]
    rep, pres, freq = (s["penalties"][:, i:i + 1] for i in range(3))
    named = counts > 0
    x = torch.where(named, torch.where(x > 0, x / rep, x * rep), x)
    x = x - torch.where(named, pres + freq * counts, torch.zeros_like(x))
    if s["bias_ids"] is not None:
        nb = torch.arange(s["longest_bias"], device="cuda")
        at = s["bias_range"][:, :1].long() + nb
        inside = at < s["bias_range"][:, 1:]
        at = at.clamp(max=s["bias_ids"].numel() - 1)
        add = torch.zeros((R, V + 1), device="cuda")
        add.scatter_add_(1, torch.where(inside, s["bias_ids"][at].long(), torch.full_like(at, V)), s["bias"][at])
        x = x + add[:, :V]
    if s["mask"] is not None:
        tok = torch.arange(V, device="cuda")
        word = s["mask"][s["mask_index"].clamp(min=0).long()][:, tok // 32]
        ok = ((word >> (tok % 32).int()) & 1).bool() | (s["mask_index"] < 0)[:, None]
        x = torch.where(ok, x, torch.full((), -math.inf, device="cuda"))
    s["out"].copy_(x)
    return s["out"]


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "logits":
        e = 4 if case["dtype"] == "f32" else 2
        R, V = case["rows"], case["vocab"]
        reqs = -(-R // max(1, R // 16))
        return {"bytes": 2 * R * V * e + case["masks"] * V / 8 + reqs * (3 * case["history"] + 8 * case["bias"]) + 44 * R,
                "flops": R * V}
    B, H, D = case["n_seq"], case["heads"], case["dim"]
    row = {"int8": D + D // 16, "bf16": 2 * D, "f32": 4 * D}[case.get("kv", "int8")]
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "tree":
        share = 2 / 3 if case["ragged"] else 1.0   # of the context that an average sequence holds
        nodes = case["nodes"] * (0.5 if case["ragged"] else 1.0)
        keys = case["ctx"] * share + nodes
        return {"bytes": B * H * (2 * keys * row + 2 * nodes * case["group"] * D * e),
                "flops": 4 * B * H * case["group"] * D * nodes * keys}
    n = B * H * case["rows"] * (0.5 if case["ragged"] else 1.0)
    if case["op"] == "append":  # source read, codes and scales written and read, f32 values written
        return {"bytes": 2 * n * (D * e + 2 * row + 4 * D), "flops": 8 * n * D}
    return {"bytes": 2 * n * (row + D * e), "flops": 2 * n * D}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "logits":
        return _exact_logits(s)
    if case["op"] == "tree":
        return _exact_tree(s)
    return {name: _exact_rows(s, name) for name in ("k", "v")}


def _exact_rows(s, name):
    out = torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda")
    for b in range(out.shape[0]):
        n, at = int(s["count"][b]), int(s["start"][b])
        if n == 0:
            continue
        if s["op"] == "append":
            x = s[name + "_new"][b, :, :n].double().reshape(out.shape[1], n, -1, 32)
            d = (x.abs().max(-1, keepdim=True).values / 127).float().double()  # the definition's divisor is an f32
            q = torch.where(d > 0, x / torch.where(d > 0, d, 1.0), 0.0).float().double()  # and so is its quotient
            q = torch.sign(q) * torch.floor(q.abs() + 0.5)
            val = q.clamp(-127, 127) * d.half().double()
        else:
            val = s[name][b, :, at:at + n].double().reshape(out.shape[1], n, -1, 32)
            val = val * s[name + "s"][b, :, at:at + n].double()[..., None]
        out[b, :, :n] = val.reshape(out.shape[1], n, -1)
    return out


def _exact_tree(s):
    B, n, heads, D = s["q"].shape
    out = torch.zeros((B, n, heads, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        c, ln = int(s["count"][b]), int(s["start"][b])
        if c == 0:
            continue
        bits = torch.tensor([[(int(m) >> j) & 1 for j in range(c)] for m in s["mask"][b, :c].tolist()], device="cuda").bool()
        sees = torch.cat([torch.ones((c, ln), dtype=torch.bool, device="cuda"), bits], 1)
        for h in range(heads):
            kvh = h // s["group"]
            k, v = s["k"][b, kvh, :ln + c].double(), s["v"][b, kvh, :ln + c].double()
            if s["ks"] is not None:
                k = k * s["ks"][b, kvh, :ln + c].double().repeat_interleave(32, -1)
                v = v * s["vs"][b, kvh, :ln + c].double().repeat_interleave(32, -1)
            z = (s["q"][b, :c, h].double() @ k.T) * s["scale"]
            out[b, :c, h] = torch.softmax(z.masked_fill(~sees, -math.inf), -1) @ v
    return out


def _exact_logits(s):
    R, V = s["logits"].shape
    out = torch.empty((R, V), dtype=torch.float64, device="cuda")
    words = None if s["mask"] is None else s["mask"].long() & 0xFFFFFFFF
    for r in range(R):
        a, b = s["range"][r].tolist()
        ids = torch.cat([s["history"][a:b].long(), s["path"][r][s["path"][r] >= 0].long()])
        c = torch.bincount(ids, minlength=V).double()
        rep, pres, freq = s["penalties"][r].double().tolist()
        x = s["logits"][r].double()
        seen = c > 0
        x = torch.where(seen & (x > 0), x / rep, torch.where(seen, x * rep, x)) - seen * pres - freq * c
        if s["bias_ids"] is not None:
            a, b = s["bias_range"][r].tolist()
            x = x.index_add(0, s["bias_ids"][a:b].long(), s["bias"][a:b].double())
        if words is not None and int(s["mask_index"][r]) >= 0:
            w = words[int(s["mask_index"][r])]
            allowed = ((w[:, None] >> torch.arange(32, device="cuda")) & 1).reshape(-1)[:V].bool()
            x = x.masked_fill(~allowed, -math.inf)
        out[r] = x
    return out
