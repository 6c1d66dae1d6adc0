"""Operators around a cache that several requests share: rotary positions, forks, page moves, shared-prefix attention.

One KV row of the cache is 656 bytes: 512 e4m3 latent codes, four fp32 scales (one per 128
latent values), 64 bf16 rope values; pages hold 64 rows and a block table maps a request's
pages to pool pages. An index key is 128 e4m3 codes with an fp32 scale.

    rotary   (x_a, x_b) -> magnitude (x_a cos - x_b sin, x_a sin + x_b cos), the angle position x frequency;
             the pairs are neighbours (2 i, 2 i + 1) or lie in two halves (i, i + dims / 2)
    fork     a request that starts with the first positions of another one: their whole pages shared, the
             rows of the last, partly filled page copied
    move     pages copied to other places in every layer, and every table that names them brought in line
    prefix   z_t = sm_scale * q . k_t for t < limit, out = softmax(z) . v, lse = log sum exp z, for requests
             whose first positions hold the same rows

Each is written below once in elementary torch operations (`own` false) and once as the calls
that a user makes of the framework (`own` true).
"""
import math

import torch

own = False

PAGE, ROW, LATENT, ROPE, KEY, GROUP = 64, 656, 512, 64, 128, 128
QK = LATENT + ROPE
FP8_PAGE = 8448            # a page of index keys: 64 x 128 codes, then 64 fp32 scales
NOPE = 128                 # dims of a query head that carry no position
E4M3 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
THETA = 10000.0
DEV = "cuda"


def listed():
    return [
        # a decode step rotates one token: its query heads, its rope, its index queries and key. Launch latency
        {"name": "rotary 1", "op": "rotary", "dtype": "bf16", "tokens": 1, "heads": 64, "idx_heads": 64, "dims": 64,
         "ctx": 131072, "scaling": "ramp"},
        # the input of a later turn, projections still in fp32, an odd count, no indexer in this layer
        {"name": "rotary 753 fp32", "op": "rotary", "dtype": "fp32", "tokens": 753, "heads": 32, "idx_heads": 0,
         "dims": 64, "ctx": 74913, "scaling": "none"},
        # a prefill chunk at the end of a long context
        {"name": "rotary 16411", "op": "rotary", "dtype": "bf16", "tokens": 16411, "heads": 64, "idx_heads": 64,
         "dims": 64, "ctx": 1000000, "scaling": "ramp"},
        # one more answer is begun from a short prompt
        {"name": "fork 1", "op": "fork", "layers": 4, "idx_layers": 1, "forks": 1, "len": "201", "host": 0},
        # 48 samples of three long prompts, some of whose pages are on the host alone
        {"name": "fork 48", "op": "fork", "layers": 8, "idx_layers": 2, "forks": 48, "len": "74913,8191,131009", "host": 3},
        # a few pages leave the end of the pool
        {"name": "move 7", "op": "move", "layers": 4, "idx_layers": 1, "moves": 7, "ctx": "4097,333,64"},
        # a pool whose free pages are scattered is compacted
        {"name": "move 2500", "op": "move", "layers": 4, "idx_layers": 2, "moves": 2500,
         "ctx": "74160,74913,8192,20001,131072,33333,65,12345"},
        # two answers to one short prompt, few heads: latency
        {"name": "prefix 2 of 201", "op": "prefix", "dtype": "bf16", "heads": 16, "groups": "2", "shared": "193",
         "ctx": "200,201", "new": "1,1", "empty": 0, "pad": 0},
        # 64 requests behind one prompt decode a token each
        {"name": "prefix 64 of 32768", "op": "prefix", "dtype": "bf16", "heads": 64, "groups": "64", "shared": "32768",
         "ctx": ",".join(str(32768 + int(16 * 128 ** (i / 63))) for i in range(64)), "new": ",".join(["1"] * 64),
         "empty": 0, "pad": 0},
        # 96 requests behind a long document, a shard of 16 heads
        {"name": "prefix 96 of 131009", "op": "prefix", "dtype": "bf16", "heads": 16, "groups": "96", "shared": "131009",
         "ctx": ",".join(str(131009 + 1 + (i * 397) % 900) for i in range(96)), "new": ",".join(["1"] * 96),
         "empty": 0, "pad": 0},
        # verifications of four tokens behind prompts of several lengths, a request that shares nothing, a padded batch
        {"name": "prefix ragged fp16", "op": "prefix", "dtype": "fp16", "heads": 32, "groups": "5,1,9,2", "shared": "8192,0,20001,130",
         "ctx": "8200,8300,9001,8196,12000,5000,20005,20100,20010,23001,20064,20065,20066,21000,20500,134,700",
         "new": "4,4,4,4,4,1,4,4,4,4,4,4,4,4,4,4,4", "empty": 2, "pad": 3},
        # eight questions about one document are prefilled together
        {"name": "prefix 8x129 of 20001", "op": "prefix", "dtype": "bf16", "heads": 64, "groups": "8", "shared": "20001",
         "ctx": ",".join(["20130"] * 8), "new": ",".join(["129"] * 8), "empty": 0, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(numbers):
    return ",".join(map(str, numbers))


def draw(rng):
    op = rng.choice(["rotary", "fork", "move", "prefix", "prefix", "prefix"])
    if op == "rotary":
        idx_heads = rng.choice([0, 16, 64])
        return {"op": op, "dtype": rng.choice(sorted(DTYPES)), "tokens": _log(rng, 1, 8000), "heads": rng.choice([1, 16, 32, 64]),
                "idx_heads": idx_heads, "dims": rng.choice([32, 64, 64, 96, 128]), "ctx": _log(rng, 8000, 1300000),
                "scaling": rng.choice(["none", "linear", "theta", "ramp"])}
    if op == "fork":
        layers = rng.randint(1, 8)
        return {"op": op, "layers": layers, "idx_layers": rng.randint(1, min(2, layers)), "forks": _log(rng, 1, 60),
                "len": _text(_log(rng, 1, 60000) for _ in range(rng.randint(1, 4))), "host": rng.choice([0, 2])}
    if op == "move":
        ctx = [_log(rng, 1, 60000) for _ in range(rng.randint(1, 8))]
        pages, layers = sum(-(-c // PAGE) for c in ctx), rng.randint(1, 6)
        return {"op": op, "layers": layers, "idx_layers": rng.randint(1, min(2, layers)),
                "moves": max(1, min(pages - 1, _log(rng, 1, 2000))), "ctx": _text(ctx)}
    heads, groups, shared, ctx, new = rng.choice([16, 32, 64]), [], [], [], []
    for _ in range(rng.randint(1, 5)):
        m = rng.choice([1, 2, _log(rng, 2, 24), _log(rng, 2, 24)])
        p = _log(rng, 30, 60000) if m > 1 else 0
        groups.append(m)
        shared.append(p)
        for _ in range(m):
            t = rng.choice([1, 1, 1, 4, _log(rng, 1, 120)])
            new.append(t)
            ctx.append(p + t + _log(rng, 1, 900) - 1)
    # no more than the largest listed, and the plain form's scores within memory
    cost = lambda: sum(n * c for n, c in zip(new, ctx)) * heads  # noqa: E731
    room = lambda: (len(groups) * max(shared + [1]) * max(sum(new[sum(groups[:i]):sum(groups[:i + 1])]) for i in range(len(groups))) +  # noqa: E731
                    len(new) * max(new) * max(c for c in ctx)) * heads
    while cost() > 1.2e9 or room() > 3.0e9:
        i = max(range(len(new)), key=lambda j: new[j])
        if new[i] == 1:
            g = max(range(len(groups)), key=lambda j: shared[j])
            lo, cut = sum(groups[:g]), shared[g] // 2
            shared[g] -= cut
            for j in range(lo, lo + groups[g]):
                ctx[j] -= cut
        else:
            ctx[i] -= new[i] // 2
            new[i] -= new[i] // 2
    return {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16"]), "heads": heads, "groups": _text(groups), "shared": _text(shared),
            "ctx": _text(ctx), "new": _text(new), "empty": min(rng.choice([0, 0, 2]), new[-1] - 1), "pad": rng.choice([0, 3])}


def _ints(text):
    return [int(x) for x in text.split(",")]


def _pages(n):
    return -(-n // PAGE)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _row_views(kv):
    """The parts of KV rows [..., 656] as the types they hold."""
    return kv[..., :LATENT].view(E4M3), kv[..., LATENT:LATENT + 16].view(torch.float32), kv[..., LATENT + 16:].view(torch.bfloat16)


SCALING = {"none": {}, "linear": {"factor": 8.0}, "theta": {"factor": 8.0},
           "ramp": {"factor": 40.0, "original_ctx": 4096.0, "beta_fast": 32.0, "beta_slow": 1.0, "magnitude": 0.1}}


def _frequencies(dims, scaling):
    """Radians per position of each pair, and what the rotated values are multiplied by."""
    s, half = SCALING[scaling], dims // 2
    i = torch.arange(half, dtype=torch.float64)
    theta = THETA * s["factor"] ** (dims / (dims - 2)) if scaling == "theta" else THETA
    f = theta ** (-2.0 * i / dims)
    if scaling == "linear":
        f = f / s["factor"]
    if scaling != "ramp":
        return f, 1.0
    # pairs that turn more than beta_fast times over the original context keep their frequency, those that turn
    # less than beta_slow times take a factor-th of it, in between a line over the pairs
    at = lambda turns: dims * math.log(s["original_ctx"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(THETA))  # noqa: E731
    low, high = max(math.floor(at(s["beta_fast"])), 0), min(math.ceil(at(s["beta_slow"])), dims - 1)
    part = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
    return f * (1.0 - part) + f / s["factor"] * part, 1.0 + s["magnitude"] * math.log(s["factor"])


def _rotary_inputs(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    n, h, hi, d, dtype = case["tokens"], case["heads"], case["idx_heads"], case["dims"], DTYPES[case["dtype"]]
    s = {"case": case}
    first = torch.randint(0, max(1, case["ctx"] - n), (1,), generator=gen, device=DEV, dtype=torch.int32)
    s["pos"] = first + torch.arange(n, dtype=torch.int32, device=DEV)
    # the query projection's last dims go behind the 512 latent dims of the attention's queries; the rope of the
    # new rows is the last part of the latent projection; an indexer's heads are rotated in their first dims
    up = _randn(gen, n, h, NOPE + d).to(dtype)
    down = _randn(gen, n, LATENT + d).to(dtype)
    q = torch.zeros(n, h, LATENT + d, dtype=dtype, device=DEV)
    rope = torch.zeros(n, d, dtype=dtype, device=DEV)
    s["parts"] = [(up[:, :, NOPE:], q[:, :, LATENT:], "pairs"), (down[:, LATENT:], rope, "pairs")]
    if hi:
        iq, ik = _randn(gen, n, hi, KEY).to(dtype), _randn(gen, n, KEY).to(dtype)
        to_q, to_k = torch.zeros(n, hi, KEY, dtype=dtype, device=DEV), torch.zeros(n, KEY, dtype=dtype, device=DEV)
        s["parts"] += [(iq[:, :, :d], to_q[:, :, :d], "halves"), (ik[:, :d], to_k[:, :d], "halves")]
    return s


def _scatter(gen, live, moves, room):
    """`live` page ids below live + room with `moves` of them at or above `live`; those, and the free ids below."""
    holes = torch.randperm(live, generator=gen, device=DEV)[:moves]
    high = live + torch.randperm(room, generator=gen, device=DEV)[:moves]
    keep = torch.ones(live, dtype=torch.bool, device=DEV)
    keep[holes] = False
    ids = torch.cat([torch.arange(live, device=DEV)[keep], high])
    return ids[torch.randperm(live, generator=gen, device=DEV)], high.to(torch.int32), holes.to(torch.int32)


def _page_inputs(case, seed):
    """The tensors of a pool of several layers and its tables, from the seed alone."""
    gen = torch.Generator(DEV).manual_seed(seed)
    s = {"case": case}
    fork = case["op"] == "fork"
    lens = _ints(case["len"] if fork else case["ctx"])
    live = sum(_pages(c) for c in lens)
    n_req = len(lens) + (case["forks"] if fork else 0)
    room = case["forks"] if fork else 2 * case["moves"]
    s["max_pages"] = -(-max(lens) // 128) * 2
    s["n_pages"], s["n_req"], s["lens"] = live + room, n_req, lens
    s["kv"] = torch.randint(0, 256, (case["layers"], live + room, PAGE, ROW), generator=gen, device=DEV, dtype=torch.uint8)
    s["idx"] = torch.randint(0, 256, (case["idx_layers"], live + room, FP8_PAGE), generator=gen, device=DEV, dtype=torch.uint8)
    for name in ("table", "idx_table", "host_table"):
        s[name] = torch.full((n_req, s["max_pages"]), -1, dtype=torch.int64 if name == "host_table" else torch.int32, device=DEV)
    if fork:
        ids, idx_ids = (torch.randperm(live + room, generator=gen, device=DEV) for _ in range(2))
    else:
        ids, s["src"], s["dst"] = _scatter(gen, live, case["moves"], room)
        idx_ids, s["idx_src"], s["idx_dst"] = _scatter(gen, live, case["moves"], room)
    at = 0
    for r, c in enumerate(lens):
        k = _pages(c)
        s["table"][r, :k], s["idx_table"][r, :k] = ids[at:at + k].int(), idx_ids[at:at + k].int()
        if fork and case["host"]:  # the first pages left to the host
            m = min(case["host"], k - 1)
            s["table"][r, :m] = -1
            s["host_table"][r, :m] = torch.arange(m, device=DEV)
        at += k
    if fork:
        of = torch.arange(case["forks"], device=DEV) % len(lens)
        s["fork_src"] = of.int()
        s["fork_dst"] = (len(lens) + torch.arange(case["forks"], device=DEV)).int()
        s["fork_len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)[of]
        s["tail"], s["idx_tail"] = ids[live:].int(), idx_ids[live:].int()
    s["all"] = torch.arange(n_req, dtype=torch.int32, device=DEV)
    return s


def _prefix_inputs(case, seed):
    """One layer's cache in which the requests of a group share the pages of their first positions."""
    gen = torch.Generator(DEV).manual_seed(seed)
    ctx, new, groups, shared = (_ints(case[k]) for k in ("ctx", "new", "groups", "shared"))
    dtype, heads, pad = DTYPES[case["dtype"]], case["heads"], case["pad"]
    s = {"case": case, "ctx": ctx, "new": new, "groups": groups, "shared": shared}
    group_of = [g for g, m in enumerate(groups) for _ in range(m)]
    s["max_pages"] = -(-max(ctx) // 128) * 2
    s["n_pages"] = sum(p // PAGE for p in shared) + sum(_pages(c) - shared[g] // PAGE for c, g in zip(ctx, group_of))
    perm = torch.randperm(s["n_pages"], generator=gen, device=DEV)
    table = torch.full((len(ctx), s["max_pages"]), -1, dtype=torch.int64, device=DEV)
    at, first = 0, []
    for g, (m, p) in enumerate(zip(groups, shared)):
        first.append(sum(groups[:g]))
        table[first[g]:first[g] + m, :p // PAGE] = perm[at:at + p // PAGE]
        at += p // PAGE
        for r in range(first[g], first[g] + m):
            k = _pages(ctx[r]) - p // PAGE
            table[r, p // PAGE:p // PAGE + k] = perm[at:at + k]
            at += k
    s["table"] = table
    kv = torch.empty(s["n_pages"] * PAGE, ROW, dtype=torch.uint8, device=DEV)
    codes, scales, rope = _row_views(kv)
    for lo in range(0, s["n_pages"] * PAGE, 1 << 18):
        hi = min(s["n_pages"] * PAGE, lo + (1 << 18))
        mag = torch.exp(0.25 * _randn(gen, hi - lo, 1))
        x = (_randn(gen, hi - lo, LATENT) * mag).unflatten(1, (-1, GROUP))
        sc = x.abs().amax(2, keepdim=True) / 448.0
        codes[lo:hi], scales[lo:hi] = (x / sc).to(E4M3).flatten(1), sc[:, :, 0]
        rope[lo:hi] = (_randn(gen, hi - lo, ROPE) * mag).bfloat16()
    for g, (m, p) in enumerate(zip(groups, shared)):  # the shared rows of a page that is not shared whole
        if m > 1 and p % PAGE:
            rows = table[first[g]:first[g] + m, p // PAGE][:, None] * PAGE + torch.arange(p % PAGE, device=DEV)
            kv[rows[1:]] = kv[rows[0]]
    s["kv"], s["idx"] = kv, torch.zeros(1, FP8_PAGE, dtype=torch.uint8, device=DEV)
    start = [0]
    for m in new:
        start.append(start[-1] + m)
    n = start[-1]
    limit = torch.cat([torch.arange(c - m + 1, c + 1) for c, m in zip(ctx, new)] + [torch.zeros(pad, dtype=torch.int64)])
    if case["empty"]:
        limit[n - case["empty"]:n] = 0
    int32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(DEV)  # noqa: E731
    s["group_start"], s["group_len"] = int32(first + [len(ctx)]), int32(shared)
    s["seg_req"], s["seg_start"], s["limit"] = int32(range(len(ctx))), int32(start), int32(limit)
    s["group_of"], s["ends"] = torch.tensor(group_of, device=DEV), torch.tensor(ctx, device=DEV)
    s["group_tokens"] = max(sum(new[f:f + m]) for f, m in zip(first, groups))
    s["longest"] = max(c - shared[g] for c, g in zip(ctx, group_of))
    s["q"] = (1.5 * _randn(gen, n + pad, heads, QK)).to(dtype)
    s["out"] = torch.full((n + pad, heads, LATENT), 0.5, dtype=dtype, device=DEV)
    s["lse"] = torch.full((n + pad, heads), 0.5, dtype=torch.float32, device=DEV)
    s["scale"] = 1.0 / math.sqrt(QK)
    return s


def _inputs(case, seed):
    return {"rotary": _rotary_inputs, "fork": _page_inputs, "move": _page_inputs, "prefix": _prefix_inputs}[case["op"]](case, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        if case["op"] == "rotary":
            s["freq"], s["magnitude"] = _frequencies(case["dims"], case["scaling"])
            s["freq"] = s["freq"].to(DEV)
        return s
    # What a serving program keeps between its calls, and no pass makes again: the pool (0.1 to 0.4 ms) and the tables in
    # it. A request's pages are entered one by one, when the program's allocator hands them out; to enter all of them at
    # once, as here, takes 0.04 to 4 ms (198,000 entries as Python numbers, 96 requests of 131,000 positions; 6.7 us for
    # one entry). From here on the tables are the pool's: the passes read those, and not the tensors that they were
    # entered from, which forks and moves read them back into. The pages that a pass's own tokens begin are entered in it.
    from sparse_mla_kv_indexer_gb300 import hisparse as H
    if case["op"] == "rotary":  # the pool whose queries and rows are rotated: its sizes do not matter here
        s["kv"] = torch.zeros(1, 1, PAGE, ROW, dtype=torch.uint8, device=DEV)
        s["idx"] = torch.zeros(1, 1, FP8_PAGE, dtype=torch.uint8, device=DEV)
        steps, s["magnitude"] = H.rotary_steps(case["dims"], THETA, case["scaling"], **SCALING[case["scaling"]])
        s["steps"] = steps.to(DEV)
    kv = s["kv"] if s["kv"].dim() == 4 else s["kv"][None]
    idx = s["idx"] if s["idx"].dim() == 3 else s["idx"][None]
    layers, max_pages = kv.shape[0], s.get("max_pages", 2)
    host_pages = max(1, case.get("host", 0))
    cfg = H.PoolConfig(page_size=PAGE, row_bytes=ROW, idx_dim=KEY, n_idx_heads=64, n_heads=64 if case["op"] != "prefix" else case["heads"],
                       topk=2048, n_layers=layers, layers_per_indexer=-(-layers // idx.shape[0]), num_pages=s.get("n_pages", 1),
                       num_idx_pages=idx.shape[1], max_requests=s.get("n_req", len(s.get("ctx", [0]))), max_ctx=max_pages * PAGE,
                       max_q_per_req=1, hot_rows=64, max_tokens=1, idx_format=H.IDX_FP8, host_pages=host_pages)
    host = torch.zeros(host_pages * layers * PAGE * ROW, dtype=torch.uint8, pin_memory=True)
    groups = -(-layers // cfg.layers_per_indexer)
    s["pool"] = H.Pool(cfg, list(kv), list(idx[:groups]), host)
    if case["op"] == "prefix":
        table = s["table"].cpu().tolist()
        for r, c in enumerate(s["ctx"]):
            s["pool"].set_pages(r, 0, block_table=table[r][:_pages(c)])
        s["work"] = torch.empty(s["pool"].prefix_workspace_bytes(len(s["limit"]), len(s["ctx"]), len(s["groups"])),
                                dtype=torch.uint8, device=DEV)
    elif case["op"] != "rotary":
        tables = [s[k].cpu().tolist() for k in ("table", "idx_table", "host_table")]
        for r, c in enumerate(s["lens"]):
            s["pool"].set_pages(r, 0, *[t[r][:_pages(c)] for t in tables])
    return s


def run(s):
    return {"rotary": _rotary, "fork": _fork, "move": _move, "prefix": _prefix}[s["case"]["op"]](s)


def _rotary(s):
    if own:
        s["pool"].rotary(s["pos"], s["steps"], s["parts"], magnitude=s["magnitude"])
        return [out for _, out, _ in s["parts"]]
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["magnitude"]).float() for f in (torch.cos, torch.sin))
    return [_turned(x, out, layout, cos, sin) for x, out, layout in s["parts"]]


def _turned(x, out, layout, cos, sin):
    if x.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    half = x.shape[-1] // 2
    v = x.float()
    a, b = (v[..., 0::2], v[..., 1::2]) if layout == "pairs" else (v[..., :half], v[..., half:])
    r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1 if layout == "pairs" else -2).flatten(-2)
    out.copy_(r.to(out.dtype))
    return out


def _state(s):
    """The whole pool: its layers, its index keys and every request's tables."""
    return {"kv": s["kv"], "idx": s["idx"], "tables": [s["table"], s["idx_table"], s["host_table"]]}


def _fork(s):
    if own:
        s["pool"].fork_requests(s["fork_src"], s["fork_dst"], s["fork_len"], s["tail"], s["idx_tail"])
        s["pool"].get_pages(s["all"], 0, s["table"], s["idx_table"], s["host_table"])
        return _state(s)
    src, dst, n = s["fork_src"].long(), s["fork_dst"].long(), s["fork_len"].long()
    page = torch.arange(s["max_pages"], device=DEV)
    whole, part = page < (n // PAGE)[:, None], page == (n // PAGE)[:, None]
    part &= (n % PAGE > 0)[:, None]
    for name, tail in (("table", s["tail"]), ("idx_table", s["idx_tail"]), ("host_table", None)):
        t = s[name]
        last = torch.full_like(n, -1).to(t.dtype) if tail is None else tail
        t[dst] = torch.where(whole, t[src], torch.where(part, last[:, None].expand_as(whole), t[dst]))
    # the rows of the last page: the destination keeps what lies behind them
    at = (n // PAGE).clamp(max=s["max_pages"] - 1)
    row = torch.arange(PAGE, device=DEV) < (n % PAGE)[:, None]
    old, fresh = s["table"][src, at].long().clamp(min=0), s["tail"].long()
    s["kv"][:, fresh] = torch.where(row[None, :, :, None], s["kv"][:, old], s["kv"][:, fresh])
    old, fresh = s["idx_table"][src, at].long().clamp(min=0), s["idx_tail"].long()
    key = torch.cat([row.repeat_interleave(KEY, 1), row.repeat_interleave(4, 1)], 1)
    s["idx"][:, fresh] = torch.where(key, s["idx"][:, old], s["idx"][:, fresh])
    return _state(s)


def _move(s):
    if own:
        # From the second pass on no entry names a source any more. With all of them to rename, as in a program's one
        # move, 2,500 pages take 168 us on the GPU and not 166 to 167; 7 pages 10.2 us either way.
        s["pool"].copy_pages(s["src"], s["dst"], s["idx_src"], s["idx_dst"], remap=True)
        s["pool"].get_pages(s["all"], 0, s["table"], s["idx_table"], s["host_table"])
        return _state(s)
    _moved(s["kv"], s["table"], s["src"], s["dst"])
    _moved(s["idx"], s["idx_table"], s["idx_src"], s["idx_dst"])
    return _state(s)


def _moved(pages, table, src, dst):
    pages[:, dst.long()] = pages[:, src.long()]
    now = torch.arange(pages.shape[1], dtype=torch.int32, device=DEV)
    now[src.long()] = dst
    table.copy_(torch.where(table >= 0, now[table.clamp(min=0).long()], table))


def _values(rows):
    codes, scale, rope = _row_views(rows)
    return torch.cat([(codes.float().unflatten(-1, (-1, GROUP)) * scale[..., None]).flatten(-2), rope.float()], -1)


def _padded(start, end, longest):
    """Token ids [ranges, longest] of ranges of tokens, and which of them are real."""
    tok = start[:, None] + torch.arange(longest, device=DEV)
    real = tok < end[:, None]
    return torch.where(real, tok, torch.zeros_like(tok)), real


def _part(s, req, tok, real, lo, hi, longest):
    """(maximum, sum, weighted values) of tokens [ranges, longest] over the positions lo <= t < min(hi, limit) of req."""
    heads = s["q"].shape[1]
    t = lo[:, None] + torch.arange(max(1, longest), device=DEV)
    page = s["table"][req[:, None], (t // PAGE).clamp(max=s["max_pages"] - 1)].clamp(min=0)
    k = _values(s["kv"][page * PAGE + t % PAGE])
    z = (torch.matmul(s["q"][tok].float().flatten(1, 2), k.transpose(1, 2)) * s["scale"]).unflatten(1, (-1, heads))
    upto = torch.minimum(torch.where(real, s["limit"].long()[tok], torch.zeros_like(tok)), hi[:, None])
    z.masked_fill_(~(t[:, None, :] < upto[:, :, None])[:, :, None, :], -math.inf)
    m = z.amax(3, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.full_like(m, -3.0e38))
    p = z.sub_(m).exp_()
    return m[real], p.sum(3, keepdim=True)[real], torch.matmul(p.flatten(1, 2), k[..., :LATENT]).unflatten(1, (-1, heads))[real]


def _entered(s):
    """Enters the pages that the pass's new tokens begin, as the step of a program does before it appends to them. Their ids
    are numbers on the host, the allocator's; here they are looked up in the first pass."""
    if "begun" not in s:
        spans = [(r, _pages(c - m), _pages(c)) for r, (c, m) in enumerate(zip(s["ctx"], s["new"]))]
        s["begun"] = [(r, lo, s["table"][r, lo:hi].tolist()) for r, lo, hi in spans if lo < hi]
    for r, first, ids in s["begun"]:
        s["pool"].set_pages(r, first, block_table=ids)


def _prefix(s):
    if own:
        _entered(s)
        s["pool"].prefix_attention(0, s["group_start"], s["group_len"], s["seg_req"], s["seg_start"], s["limit"], s["q"],
                                   s["scale"], s["out"], s["work"], lse=s["lse"])
        return [s["out"], s["lse"]]
    start, bounds, shared = s["seg_start"].long(), s["group_start"].long(), s["group_len"].long()
    # the shared positions once for all tokens of a group, the others for each request
    tok, real = _padded(start[bounds[:-1]], start[bounds[1:]], s["group_tokens"])
    m1, l1, o1 = _part(s, s["seg_req"].long()[bounds[:-1]], tok, real, torch.zeros_like(shared), shared, max(s["shared"]))
    tok, real = _padded(start[:-1], start[1:], max(s["new"]))
    m2, l2, o2 = _part(s, s["seg_req"].long(), tok, real, shared[s["group_of"]], s["ends"], s["longest"])
    m = torch.maximum(m1, m2)
    f1, f2 = (m1 - m).exp(), (m2 - m).exp()
    total = l1 * f1 + l2 * f2
    o = torch.where(total > 0, (o1 * f1 + o2 * f2) / total, torch.zeros_like(o1))
    n = total.shape[0]
    s["out"][:n] = o.to(s["out"].dtype)
    s["lse"][:n] = torch.where(total > 0, m + total.log(), torch.full_like(m, -math.inf))[:, :, 0]
    return [s["out"], s["lse"]]


def work(case):
    if case["op"] == "rotary":
        n, size = case["tokens"], {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        heads = case["heads"] + 1 + (case["idx_heads"] + 1 if case["idx_heads"] else 0)
        return {"bytes": n * (heads * case["dims"] * size * 2 + 4), "flops": n * heads * case["dims"] * 3}
    if case["op"] == "fork":
        lens = _ints(case["len"])
        of = [lens[i % len(lens)] for i in range(case["forks"])]
        entries = sum(n // PAGE for n in of) * 2 * 16 + len(of) * 20
        return {"bytes": entries + sum(n % PAGE for n in of) * 2 * (case["layers"] * ROW + case["idx_layers"] * (KEY + 4)), "flops": 0}
    if case["op"] == "move":
        entries = sum(_pages(c) for c in _ints(case["ctx"])) * 8
        return {"bytes": case["moves"] * (2 * (case["layers"] * PAGE * ROW + case["idx_layers"] * FP8_PAGE) + 32) + entries, "flops": 0}
    ctx, new, groups, shared = (_ints(case[k]) for k in ("ctx", "new", "groups", "shared"))
    h, e, n = case["heads"], case["empty"], sum(_ints(case["new"]))
    limits = [range(c - m + 1, c + 1) for c, m in zip(ctx, new)]
    seen = sum((r[0] + r[-1]) * len(r) // 2 for r in limits) - sum(limits[-1][len(limits[-1]) - e:])
    rows = sum(shared) + sum(c - p for c, p in zip(ctx, [p for p, m in zip(shared, groups) for _ in range(m)]))
    return {"bytes": rows * ROW + n * h * ((QK + LATENT) * 2 + 4) + n * 4, "flops": 2 * seen * h * (QK + LATENT)}


def exact(case, seed):
    """What run() returns for these inputs, from the definitions, in 64 bits."""
    if case["op"] in ("fork", "move"):
        return None  # bytes and whole numbers: the plain form's are the definition
    s = _inputs(case, seed)
    if case["op"] == "rotary":
        freq, magnitude = _frequencies(case["dims"], case["scaling"])
        turn = torch.polar(torch.full((1, 1), magnitude, dtype=torch.float64, device=DEV).expand(case["tokens"], case["dims"] // 2).contiguous(),
                           torch.outer(s["pos"].double(), freq.to(DEV)))
        found = []
        for x, _, layout in s["parts"]:
            v = x.double().unflatten(-1, (-1, 2) if layout == "pairs" else (2, -1))
            if layout == "halves":
                v = v.transpose(-1, -2)
            r = torch.view_as_real(torch.view_as_complex(v.contiguous()) * (turn if x.dim() == 2 else turn[:, None]))
            found.append((r if layout == "pairs" else r.transpose(-1, -2)).flatten(-2))
        return found
    values = torch.arange(256, dtype=torch.uint8, device=DEV).view(E4M3).double()
    out, lse = s["out"].double(), s["lse"].double()
    first = 0
    for r, (c, m) in enumerate(zip(s["ctx"], s["new"])):
        rows = s["kv"].unflatten(0, (-1, PAGE))[s["table"][r][:_pages(c)]].flatten(0, 1)[:c]
        v = values[rows[:, :LATENT].long()] * rows[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double().repeat_interleave(GROUP, 1)
        k = torch.cat([v, rows[:, LATENT + 16:].contiguous().view(torch.bfloat16).double()], 1)
        step = max(1, int(2.0e9 / (case["heads"] * c)))
        for lo in range(first, first + m, step):
            hi = min(first + m, lo + step)
            z = torch.einsum("jhd,td->jht", s["q"][lo:hi].double(), k).mul_(s["scale"])
            z.masked_fill_((torch.arange(c, device=DEV)[None, :] >= s["limit"][lo:hi, None])[:, None, :], -math.inf)
            lse[lo:hi] = torch.logsumexp(z, 2)
            w = z.sub_(torch.nan_to_num(lse[lo:hi], neginf=0.0)[:, :, None]).exp_()
            out[lo:hi] = torch.einsum("jht,td->jhd", w, v)
        first += m
    return [out, lse]
