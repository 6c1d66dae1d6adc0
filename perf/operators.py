"""The cache operators of a prefill and of a dense decode: quantised append, read back, chunk attention.

One KV row of the cache is 656 bytes: 512 e4m3 latent codes, four fp32 scales (one per 128
latent values), 64 bf16 rope values; pages hold 64 rows and a block table maps a request's
pages to pool pages. Index keys are 128 e4m3 codes with an fp32 scale, or 128 int8 values.

    append      x -> scale = amax / 448 per 128 values (1 where amax is 0), code = e4m3(x / scale)
    read        value = code * scale
    attention   z_t = sm_scale * q . k_t for t < limit, out = softmax(z) . v, lse = log sum exp z

Each is written below once in elementary torch operations (`own` false) and once as the calls
that a user makes of the framework (`own` true).
"""
import math

import torch

own = False

PAGE, ROW, LATENT, ROPE, KEY, GROUP = 64, 656, 512, 64, 128, 128
QK = LATENT + ROPE
FP8_PAGE = 8448            # a page of fp8 index keys: 64 x 128 codes, then 64 fp32 scales
E4M3 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
INT8_STEP = 0.03125        # step of the int8 index keys
DEV = "cuda"


def listed():
    return [
        # a decode step writes one token of one layer and its index key: launch latency
        {"name": "append 1", "op": "append", "dtype": "bf16", "keys": "fp8", "ctx": "4097", "new": "1"},
        # the input of a later turn (753 tokens), its projections still in fp32, int8 index keys
        {"name": "append 753 fp32", "op": "append", "dtype": "fp32", "keys": "int8", "ctx": "74913", "new": "753"},
        # the first turn of a history, written at once; latent and rope are columns of one projection
        {"name": "append 74160", "op": "append", "dtype": "bf16", "keys": "fp8", "ctx": "74160", "new": "74160"},
        # a few positions of several requests, as a recomputation or a check reads them
        {"name": "read 5x13 fp32", "op": "read", "dtype": "fp32", "keys": "fp8", "ctx": "100,1000,4096,257,8191",
         "new": "13,13,13,13,13"},
        # a whole history read back for an attention in its up-projected form
        {"name": "read 74160", "op": "read", "dtype": "bf16", "keys": "fp8", "ctx": "74160", "new": "74160"},
        # one token over a short context with few heads: latency
        {"name": "attend 1 of 201", "op": "attend", "dtype": "bf16", "heads": 16, "ctx": "201", "new": "1",
         "empty": 0, "pad": 0},
        # one token over a long context
        {"name": "attend 1 of 131072", "op": "attend", "dtype": "bf16", "heads": 64, "ctx": "131072", "new": "1",
         "empty": 0, "pad": 0},
        # 32 requests of 8K to 256K tokens decode one token each
        {"name": "attend 32 ragged", "op": "attend", "dtype": "bf16", "heads": 64,
         "ctx": ",".join(str(int(8192 * 32 ** (i / 31))) for i in range(32)), "new": ",".join(["1"] * 32),
         "empty": 0, "pad": 0},
        # a prompt from its first token, odd length, few heads, fp16
        {"name": "attend 1777 of 1777", "op": "attend", "dtype": "fp16", "heads": 16, "ctx": "1777", "new": "1777",
         "empty": 0, "pad": 0},
        # decodes, verifications of four tokens and prompt chunks in one padded batch: the last segment ends in
        # tokens that see nothing, and rows lie behind the last segment
        {"name": "attend mixed", "op": "attend", "dtype": "bf16", "heads": 32, "ctx": "20001,8192,333,4,12345,130,19,64",
         "new": "1,4,1,4,129,130,19,40", "empty": 3, "pad": 5},
        # the input of a later turn over its history
        {"name": "attend 753 of 74913", "op": "attend", "dtype": "bf16", "heads": 64, "ctx": "74913", "new": "753",
         "empty": 0, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend"])
    if op != "attend":
        n = rng.randint(1, 8)
        new = [_log(rng, 1, 9000) for _ in range(n)]
        ctx = [max(m, _log(rng, 64, 70000)) for m in new]
        return {"op": op, "dtype": rng.choice(sorted(DTYPES)), "keys": rng.choice(["fp8", "int8"]),
                "ctx": ",".join(map(str, ctx)), "new": ",".join(map(str, new))}
    n, heads = rng.randint(1, 12), rng.choice([16, 32, 64])
    new, ctx, budget = [], [], 7.0e12 / (2 * heads * (QK + LATENT))
    for _ in range(n):
        c = _log(rng, 64, 130000)
        m = min(c, rng.choice([1, 1, 4, _log(rng, 2, 1500)]))
        m = max(1, min(m, int(budget / n / c)))
        new.append(m)
        ctx.append(c)
    # the plain form pads: keep its score matrix within memory
    while len(new) * max(new) * heads * max(ctx) > 6.0e9:
        i = max(range(len(new)), key=lambda j: new[j])
        new[i] = max(1, new[i] // 2)
    return {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16"]), "heads": heads, "ctx": ",".join(map(str, ctx)),
            "new": ",".join(map(str, new)), "empty": min(rng.choice([0, 0, 2]), new[-1] - 1), "pad": rng.choice([0, 3])}


def _ints(text):
    return [int(x) for x in text.split(",")]


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _quantise(x, groups):
    """x [n, d] -> e4m3 codes [n, d] and fp32 scales [n, groups]."""
    x = x.float().unflatten(1, (groups, -1))
    amax = x.abs().amax(2, keepdim=True)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x / scale).to(E4M3).flatten(1), scale[:, :, 0]


def _row_views(kv):
    """The parts of the KV rows [pages * 64, 656] as the types they hold."""
    return kv[:, :LATENT].view(E4M3), kv[:, LATENT:LATENT + 16].view(torch.float32), kv[:, LATENT + 16:].view(torch.bfloat16)


def _key_views(idx, kind):
    """Index keys [pages, bytes of a page] as codes [pages, 64, 128] and scales [pages, 64] (None for int8)."""
    if kind == "int8":
        return idx.view(torch.int8).unflatten(1, (PAGE, KEY)), None
    return idx[:, :PAGE * KEY].view(E4M3).unflatten(1, (PAGE, KEY)), idx[:, PAGE * KEY:].view(torch.float32)


def _inputs(case, seed):
    """The cache, its block table and the call's inputs, from the seed alone."""
    gen = torch.Generator(DEV).manual_seed(seed)
    ctx, new = _ints(case["ctx"]), _ints(case["new"])
    dtype = DTYPES[case["dtype"]]
    max_pages = -(-max(ctx) // 128) * 2
    n_pages = sum(-(-c // PAGE) for c in ctx)
    s = {"case": case, "ctx": ctx, "new": new, "n_pages": n_pages, "max_pages": max_pages}
    perm = torch.randperm(n_pages, generator=gen, device=DEV, dtype=torch.int64)
    table = torch.full((len(ctx), max_pages), -1, dtype=torch.int64, device=DEV)
    at = 0
    for r, c in enumerate(ctx):
        k = -(-c // PAGE)
        table[r, :k] = perm[at:at + k]
        at += k
    s["table"] = table
    # cached rows: unit normal values, with a magnitude of each row's own
    kv = torch.empty(n_pages * PAGE, ROW, dtype=torch.uint8, device=DEV)
    codes, scales, rope = _row_views(kv)
    for lo in range(0, n_pages * PAGE, 1 << 18):
        hi = min(n_pages * PAGE, lo + (1 << 18))
        mag = torch.exp(0.25 * _randn(gen, hi - lo, 1))
        c, sc = _quantise(_randn(gen, hi - lo, LATENT) * mag, LATENT // GROUP)
        codes[lo:hi], scales[lo:hi] = c, sc
        rope[lo:hi] = (_randn(gen, hi - lo, ROPE) * mag).bfloat16()
    s["kv"] = kv
    kind = case.get("keys", "int8")
    s["idx"] = torch.zeros(n_pages if case["op"] != "attend" else 1, FP8_PAGE if kind == "fp8" else PAGE * KEY,
                           dtype=torch.uint8, device=DEV)
    n = sum(new)
    if case["op"] == "attend":
        heads, pad = case["heads"], case["pad"]
        start = [0]
        for m in new:
            start.append(start[-1] + m)
        limit = torch.cat([torch.arange(c - m + 1, c + 1) for c, m in zip(ctx, new)] + [torch.zeros(pad, dtype=torch.int64)])
        if case["empty"]:
            limit[n - case["empty"]:n] = 0
        s["seg_req"] = torch.arange(len(ctx), dtype=torch.int32, device=DEV)
        s["seg_start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        s["limit"] = limit.to(torch.int32).to(DEV)
        s["q"] = (1.5 * _randn(gen, n + pad, heads, QK)).to(dtype)
        s["out"] = torch.full((n + pad, heads, LATENT), 0.5, dtype=dtype, device=DEV)
        s["lse"] = torch.full((n + pad, heads), 0.5, dtype=torch.float32, device=DEV)
        s["scale"] = 1.0 / math.sqrt(QK)
        return s
    key_codes, key_scales = _key_views(s["idx"], kind)
    for lo in range(0, n_pages, 4096):
        hi = min(n_pages, lo + 4096)
        k = _randn(gen, (hi - lo) * PAGE, KEY)
        if kind == "fp8":
            c, sc = _quantise(k, 1)
            key_codes[lo:hi], key_scales[lo:hi] = c.unflatten(0, (-1, PAGE)), sc.unflatten(0, (-1, PAGE))[:, :, 0]
        else:
            key_codes[lo:hi] = (k / INT8_STEP).round().clamp(-127, 127).to(torch.int8).unflatten(0, (-1, PAGE))
    s["req"] = torch.cat([torch.full((m,), r, dtype=torch.int32) for r, m in enumerate(new)]).to(DEV)
    s["pos"] = torch.cat([torch.arange(c - m, c, dtype=torch.int32) for c, m in zip(ctx, new)]).to(DEV)
    if case["op"] == "append":
        proj = (_randn(gen, n, QK) * torch.exp(0.25 * _randn(gen, n, 1))).to(dtype)
        s["latent"], s["rope"] = proj[:, :LATENT], proj[:, LATENT:]
        s["keys"] = _randn(gen, n, KEY).to(dtype)
    else:
        s["latent"] = torch.empty(n, LATENT, dtype=dtype, device=DEV)
        s["rope"] = torch.empty(n, ROPE, dtype=dtype, device=DEV)
        s["keys"] = torch.empty(n, KEY, dtype=dtype, device=DEV)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the pool that a user's program keeps over its cache, and the attention's workspace
        from sparse_mla_kv_indexer_gb300 import hisparse as H
        idx_pages = s["idx"].shape[0]
        cfg = H.PoolConfig(page_size=PAGE, row_bytes=ROW, idx_dim=KEY, n_idx_heads=64, n_heads=case.get("heads", 64),
                           topk=2048, n_layers=1, layers_per_indexer=1, num_pages=s["n_pages"], num_idx_pages=idx_pages,
                           max_requests=len(s["ctx"]), max_ctx=s["max_pages"] * PAGE, max_q_per_req=1, hot_rows=64,
                           max_tokens=1, idx_format=H.IDX_FP8 if case.get("keys") == "fp8" else H.IDX_INT8, host_pages=1)
        host = torch.zeros(PAGE * ROW, dtype=torch.uint8, pin_memory=True)
        s["pool"] = H.Pool(cfg, [s["kv"]], [s["idx"]], host)
        table = s["table"].cpu().tolist()
        for r, c in enumerate(s["ctx"]):
            pages = table[r][:-(-c // PAGE)]
            s["pool"].set_pages(r, 0, block_table=pages, idx_pages=None if case["op"] == "attend" else pages)
        if case["op"] == "attend":
            s["work"] = torch.empty(s["pool"].chunk_workspace_bytes(), dtype=torch.uint8, device=DEV)
    return s


def run(s):
    return {"append": _append, "read": _read, "attend": _attend}[s["case"]["op"]](s)


def _append(s):
    kind = s["case"]["keys"]
    if own:
        s["pool"].append_quantized(0, s["req"], s["pos"], s["latent"], s["rope"], s["keys"], key_scale=INT8_STEP)
    else:
        pos = s["pos"].long()
        page, off = s["table"][s["req"].long(), pos // PAGE], pos % PAGE
        row = page * PAGE + off
        codes, scale = _quantise(s["latent"], LATENT // GROUP)
        packed = torch.cat([codes.view(torch.uint8), scale.contiguous().view(torch.uint8),
                            s["rope"].to(torch.bfloat16).contiguous().view(torch.uint8)], 1)
        s["kv"][row] = packed
        key_codes, key_scales = _key_views(s["idx"], kind)
        if kind == "fp8":
            c, sc = _quantise(s["keys"], 1)
            key_codes.view(torch.uint8)[page, off] = c.view(torch.uint8)
            key_scales[page, off] = sc[:, 0]
        else:
            key_codes[page, off] = (s["keys"].float() / INT8_STEP).round().clamp(-127, 127).to(torch.int8)
    key_codes, key_scales = _key_views(s["idx"], kind)
    return {"rows": list(_row_views(s["kv"])), "keys": [key_codes] + ([] if key_scales is None else [key_scales])}


def _read(s):
    kind = s["case"]["keys"]
    if own:
        s["pool"].read_rows(0, s["req"], s["pos"], s["latent"], s["rope"], s["keys"], key_scale=INT8_STEP)
        return [s["latent"], s["rope"], s["keys"]]
    dtype = DTYPES[s["case"]["dtype"]]
    pos = s["pos"].long()
    page, off = s["table"][s["req"].long(), pos // PAGE], pos % PAGE
    rows = s["kv"][page * PAGE + off]
    codes, scale, rope = _row_views(rows)
    latent = (codes.float().unflatten(1, (-1, GROUP)) * scale[:, :, None]).flatten(1).to(dtype)
    key_codes, key_scales = _key_views(s["idx"], kind)
    if kind == "fp8":
        keys = key_codes.view(torch.uint8)[page, off].view(E4M3).float() * key_scales[page, off][:, None]
    else:
        keys = key_codes[page, off].float() * INT8_STEP
    return [latent, rope.to(dtype), keys.to(dtype)]


def _attend(s):
    if own:
        s["pool"].chunk_attention(0, s["seg_req"], s["seg_start"], s["limit"], s["q"], s["scale"], s["out"], s["work"],
                                  lse=s["lse"])
        return [s["out"], s["lse"]]
    start = s["seg_start"].long()
    n_seg, t_max, l_max = len(s["new"]), max(s["new"]), max(s["ctx"])
    # the segments' tokens and keys, padded to the longest
    tok = start[:-1, None] + torch.arange(t_max, device=DEV)
    real = tok < start[1:, None]
    tok = torch.where(real, tok, torch.zeros_like(tok))
    t = torch.arange(l_max, device=DEV)
    page = s["table"][s["seg_req"].long()][:, t // PAGE].clamp(min=0)
    codes, scale, rope = _row_views(s["kv"][page * PAGE + t % PAGE].flatten(0, 1))
    k = torch.cat([(codes.float().unflatten(1, (-1, GROUP)) * scale[:, :, None]).flatten(1), rope.float()], 1).unflatten(0, (n_seg, l_max))
    q = s["q"][tok].float().flatten(1, 2)                                   # [segment, token x head, 576]
    heads = s["q"].shape[1]
    z = (torch.matmul(q, k.transpose(1, 2)) * s["scale"]).unflatten(1, (t_max, heads))
    seen = t[None, None, :] < torch.where(real, s["limit"].long()[tok], torch.zeros_like(tok))[:, :, None]
    z = z.masked_fill_(~seen[:, :, None, :], -math.inf)
    m = z.amax(3, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = z.sub_(m).exp_()
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p.flatten(1, 2), k[:, :, :LATENT]).unflatten(1, (t_max, heads))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    s["out"][tok[real]] = o[real].to(s["out"].dtype)
    s["lse"][tok[real]] = (m + total.log())[real][:, :, 0]
    return [s["out"], s["lse"]]


def work(case):
    ctx, new = _ints(case["ctx"]), _ints(case["new"])
    n, size = sum(new), {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if case["op"] == "attend":
        h, e = case["heads"], case["empty"]
        limits = [range(c - m + 1, c + 1) for c, m in zip(ctx, new)]
        seen = sum((r[0] + r[-1]) * len(r) // 2 for r in limits) - sum(limits[-1][len(limits[-1]) - e:])
        rows = sum(ctx) - e
        return {"bytes": rows * ROW + n * h * (QK + LATENT) * size + n * h * 4 + n * 4, "flops": 2 * seen * h * (QK + LATENT)}
    key = KEY + (4 if case["keys"] == "fp8" else 0)
    return {"bytes": n * ((QK + KEY) * size + ROW + key + 8), "flops": n * (QK + KEY) * 2}


def exact(case, seed):
    """What run() returns for these inputs, from the definitions, in 64 bits."""
    s = _inputs(case, seed)
    pos = [(r, p) for r, (c, m) in enumerate(zip(s["ctx"], s["new"])) for p in range(c - m, c)] if case["op"] != "attend" else []
    e4m3_values = torch.arange(256, dtype=torch.uint8, device=DEV).view(E4M3).double()
    as_bytes = lambda x: x.contiguous().view(torch.uint8).long()  # noqa: E731
    if case["op"] == "attend":
        out, lse = s["out"].double(), s["lse"].double()
        first = 0
        for r, (c, m) in enumerate(zip(s["ctx"], s["new"])):
            ids = s["table"][r][:-(-c // PAGE)]
            rows = s["kv"].unflatten(0, (-1, PAGE))[ids].flatten(0, 1)[:c]
            scale = rows[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double().repeat_interleave(GROUP, 1)
            v = e4m3_values[as_bytes(rows[:, :LATENT])] * scale
            k = torch.cat([v, rows[:, LATENT + 16:].contiguous().view(torch.bfloat16).double()], 1)
            step = max(1, int(2.0e9 / (case["heads"] * c)))
            for lo in range(first, first + m, step):
                hi = min(first + m, lo + step)
                z = torch.einsum("jhd,td->jht", s["q"][lo:hi].double(), k).mul_(s["scale"])
                dark = torch.arange(c, device=DEV)[None, :] >= s["limit"][lo:hi, None]
                z.masked_fill_(dark[:, None, :], -math.inf)
                lse[lo:hi] = torch.logsumexp(z, 2)
                w = z.sub_(torch.nan_to_num(lse[lo:hi], neginf=0.0)[:, :, None]).exp_()
                out[lo:hi] = torch.einsum("jht,td->jhd", w, v)
            first += m
        return [out, lse]
    table = s["table"].cpu().tolist()
    where = torch.tensor([table[r][p // PAGE] * PAGE + p % PAGE for r, p in pos], device=DEV)
    flat_codes, flat_scales = _flat_keys(s["idx"], case["keys"])
    if case["op"] == "read":
        rows = s["kv"][where]
        scale = rows[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double()
        latent = e4m3_values[as_bytes(rows[:, :LATENT])] * scale.repeat_interleave(GROUP, 1)
        rope = rows[:, LATENT + 16:].contiguous().view(torch.bfloat16).double()
        if case["keys"] == "fp8":
            keys = e4m3_values[flat_codes[where].long()] * flat_scales[where].double()[:, None]
        else:
            keys = flat_codes[where].view(torch.int8).double() * INT8_STEP
        return [latent, rope, keys]

    def nearest(y):
        """The e4m3 value nearest to y, ties to the even code."""
        grid = e4m3_values[:127]
        a = y.abs()
        up = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
        down = (up - 1).clamp(min=0)
        near_up, near_down = grid[up] - a, a - grid[down]
        pick = torch.where((near_up < near_down) | ((near_up == near_down) & (up % 2 == 0)), up, down)
        return grid[pick].copysign(y)

    def quantised(x):
        a = x.abs().amax(2, keepdim=True)
        sc = torch.where(a > 0, a / 448.0, torch.ones_like(a))
        return nearest(x / sc).flatten(1), sc[:, :, 0]

    codes = e4m3_values[s["kv"][:, :LATENT].long()]
    scales = s["kv"][:, LATENT:LATENT + 16].contiguous().view(torch.float32).double()
    rope = s["kv"][:, LATENT + 16:].contiguous().view(torch.bfloat16).double()
    codes[where], scales[where] = quantised(s["latent"].double().unflatten(1, (-1, GROUP)))
    rope[where] = s["rope"].double()
    n_pages = s["n_pages"]
    if case["keys"] == "fp8":
        key_codes, key_scales = e4m3_values[flat_codes.long()], flat_scales.double()
        c, sc = quantised(s["keys"].double()[:, None, :])
        key_codes[where], key_scales[where] = c, sc[:, 0]
        keys = [key_codes.unflatten(0, (n_pages, PAGE)), key_scales.unflatten(0, (n_pages, PAGE))]
    else:  # whole numbers: the plain form's are the definition
        keys = [None]
    return {"rows": [codes, scales, rope], "keys": keys}


def _flat_keys(idx, kind):
    """Index keys as byte codes [pages * 64, 128] and fp32 scales [pages * 64] (None for int8)."""
    if kind == "int8":
        return idx.reshape(-1, KEY), None
    return idx[:, :PAGE * KEY].reshape(-1, KEY), idx[:, PAGE * KEY:].contiguous().view(torch.float32).reshape(-1)
