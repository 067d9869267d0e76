"""What is measured of the speculative-decoding operators: cases, inputs, the
operators' plain form, their exact values and the work they cannot do without.

The operators are the four calls of a serving step that drafts a tree of tokens
for each of B sequences and checks them against the model at once, on the
framework's shapes (32 query heads, 8 key/value heads, head dimension 64,
16-token pages):

  norm     per-head RMS norm of queries and keys and the position rotation
           (``attn_qk_norm_rope``)
  append   the same on the way into a paged cache, with the values
           (``attn_append_paged``, ``attn_append_paged_bf16kv``)
  tree     attention of the drafted rows over their sequence's cache and their
           own ancestors (``attn_tree_paged``, ``attn_tree_paged_bf16kv``)
  compact  the accepted rows' keys and values moved to the front of the drafted
           ones (``attn_compact_paged``, ``attn_compact_paged_bf16kv``)

A batch is described as the calls take it: sequence b has ``contextLens[b]``
tokens in its cache and the rows ``rowStart[b] .. rowStart[b + 1] - 1`` of the
packed tensors; row i of the sequence belongs to its slot contextLens[b] + i.
"""
import math

import torch

own = False

HQ, HKV, D, PAGE = 32, 8, 64, 16
GROUP = HQ // HKV
EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def norm_case(name, n, act, cache, pairing):
    return {"name": name, "op": "norm", "n": n, "act": act, "cache": cache, "pairing": pairing}


def append_case(name, batch, rows, context, ragged, act, cache, pairing, normed):
    return {"name": name, "op": "append", "batch": batch, "rows": rows, "context": context, "ragged": ragged,
            "act": act, "cache": cache, "pairing": pairing, "normed": normed}


def tree_case(name, batch, rows, context, ragged, cache):
    return {"name": name, "op": "tree", "batch": batch, "rows": rows, "context": context, "ragged": ragged,
            "cache": cache}


def compact_case(name, batch, rows, context, ragged, cache):
    return {"name": name, "op": "compact", "batch": batch, "rows": rows, "context": context, "ragged": ragged,
            "cache": cache}


def listed():
    return [
        # A drafted chain of one sequence, seven tokens: latency.
        norm_case("norm 7 tokens", 7, "f32", "f32", 1),
        # The serving chunk (2048 rows) of a model whose projections leave bf16.
        norm_case("norm chunk 2048", 2048, "bf16", "bf16", 0),
        # One decode step of 16 sequences: the rotation, no norms, no queries.
        append_case("append decode 16", 16, 1, 16384, False, "f32", "f32", 0, False),
        # The serving chunk, 2048 rows behind 2048 cached tokens, with queries and norms.
        append_case("append chunk 2048", 1, 2048, 2048, False, "bf16", "bf16", 0, True),
        # Drafted trees of up to 61 rows for 48 sequences.
        append_case("append trees 48x61", 48, 61, 1000, True, "f32", "f32", 1, True),
        # Eight drafted tokens of one sequence with a short cache: latency.
        tree_case("tree 1x8 at 1000", 1, 8, 1000, False, "f32"),
        # The decode benchmark's batch (16 sequences of 16384 tokens), 16 drafted rows each.
        tree_case("tree 16x16 at 16384", 16, 16, 16384, False, "f32"),
        # A busy server's short sequences with a few drafted tokens each, ragged.
        tree_case("tree 48x5 to 4096", 48, 5, 4096, True, "bf16"),
        # The same batch as above with wide trees and a bf16 cache.
        tree_case("tree 16x32 at 16384", 16, 32, 16384, False, "bf16"),
        # One long document, the widest tree: the key axis is all there is to split.
        tree_case("tree 1x64 at 131071", 1, 64, 131071, False, "bf16"),
        # After the check: a few rows of a few sequences, latency.
        compact_case("compact 16x32", 16, 32, 1000, False, "f32"),
        # After the check of a large ragged batch.
        compact_case("compact 251x64", 251, 64, 500, True, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("norm", "append", "append", "tree", "tree", "tree", "compact"))
    cache = rng.choice(("f32", "bf16"))
    act = rng.choice(("f32", "bf16"))
    pairing = rng.randrange(2)
    ragged = rng.random() < 0.6
    if op == "norm":
        c = norm_case("", _log_int(rng, 1, 8192), act, cache, pairing)
    elif op == "append":
        batch = _log_int(rng, 1, 256)
        rows = _log_int(rng, 1, min(4096, 8192 // batch))
        c = append_case("", batch, rows, _log_int(rng, 1, min(16384, 262144 // batch)), ragged, act, cache, pairing,
                        rng.random() < 0.6)
    elif op == "tree":
        batch = _log_int(rng, 1, 64)
        rows = _log_int(rng, 1, min(64, 512 // batch))
        # At most 2^23 visible (row, key) pairs, as the largest listed case has.
        most = min(131072, 262144 // batch, (1 << 23) // (batch * rows) - rows)
        c = tree_case("", batch, rows, _log_int(rng, 1, most), ragged, cache)
    else:
        batch = _log_int(rng, 1, 256)
        c = compact_case("", batch, _log_int(rng, 1, 64), _log_int(rng, 1, 2048), ragged, cache)
    del c["name"]
    return c


def lengths(case):
    """(context, rows) of every sequence: from the case alone, the same for every seed."""
    got = []
    for b in range(case["batch"]):
        c, t = case["context"], case["rows"]
        if case["ragged"] and b:
            f, g = (b * 0.6180339887498949) % 1.0, (b * 0.7548776662466927) % 1.0
            c, t = max(1, int(c * (0.1 + 0.9 * f))), max(1, math.ceil(t * g))
        got.append((c, t))
    return got


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def rotation_table(positions):
    """[positions][64] fp32: cos of the 32 angles, then sin, base 10000, made in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _randn(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def _paged_batch(case, gen, filled):
    """The cache of a batch: shuffled pages, the block table, lengths and row starts."""
    lens = lengths(case)
    pages = [(c + t + PAGE - 1) // PAGE for c, t in lens]
    total = sum(pages) + 3
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    # The last entries of a short sequence's row of the table hold no page.
    first = torch.tensor([sum(pages[:b]) for b in range(len(pages))], device="cuda")
    count = torch.tensor(pages, device="cuda")
    j = torch.arange(max(pages), device="cuda")
    at = (first[:, None] + j[None, :]).clamp(max=total - 1)
    table = torch.where(j[None, :] < count[:, None], perm[at], torch.full_like(perm[at], -1)).contiguous()
    dtype = DTYPES[case["cache"]]
    make = (lambda: _randn(gen, total, PAGE, HKV, D, dtype=dtype)) if filled else \
        (lambda: torch.zeros(total, PAGE, HKV, D, device="cuda", dtype=dtype))
    starts = [0]
    for _, t in lens:
        starts.append(starts[-1] + t)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"kPages": make(), "vPages": make(), "table": table, "ctx": ints([c for c, _ in lens]),
            "rowStart": ints(starts), "n": starts[-1], "max_rows": case["rows"], "max_context": case["context"]}


def _trees(case, seed):
    """Parents are drawn as a drafter grows a tree: mostly a recent row, sometimes
    the last cached token. Returns each row's 64-bit mask (itself and its
    ancestors) and depth."""
    state = (seed * 2654435761 + 12345) & 0xFFFFFFFF
    masks, depths = [], []
    for _, t in lengths(case):
        m, d = [], []
        for i in range(t):
            state = (state * 1664525 + 1013904223) & 0xFFFFFFFF
            back = 1 + (state >> 24) % 5
            p = i - back
            m.append((m[p] if p >= 0 else 0) | (1 << i))
            d.append(d[p] + 1 if p >= 0 else 0)
        masks += [x - (1 << 64) if x >> 63 else x for x in m]
        depths += d
    return masks, depths


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op in ("norm", "append"):
        s["pairing"] = case["pairing"]
        act = DTYPES[case["act"]]
        if op == "norm":
            n, far = case["n"], 32768
            s["positions"] = torch.randint(0, far, (n,), generator=gen, device="cuda").to(torch.int32)
            s["kOut"] = torch.empty(n, HKV, D, device="cuda", dtype=DTYPES[case["cache"]])
            normed = True
        else:
            s.update(_paged_batch(case, gen, filled=False))
            n, far, normed = s["n"], case["context"] + case["rows"], case["normed"]
            if case["rows"] <= 64:  # drafted trees: the position goes by the depth, the slot by the row
                _, depths = _trees(case, seed)
                ctx = [c for c, t in lengths(case) for _ in range(t)]
                s["positions"] = torch.tensor([c + d for c, d in zip(ctx, depths)], dtype=torch.int32, device="cuda")
            else:
                s["positions"] = None  # consecutive: contextLens[b] + i
        s["cosSin"] = rotation_table(far)
        # Queries and keys leave one projection, keys and values another, so
        # each has its own stride between rows.
        s["q"] = _randn(gen, n, HQ + 1, D, dtype=act)[:, :HQ] if normed else None
        kv = _randn(gen, n, 2 * HKV, D, dtype=act)
        s["k"], s["v"] = kv[:, :HKV], kv[:, HKV:]
        s["qOut"] = torch.empty(n, HQ, D, device="cuda") if normed else None
        s["qWeight"] = 1.0 + _randn(gen, D, scale=0.1) if normed else None
        s["kWeight"] = 1.0 + _randn(gen, D, scale=0.1) if normed else None
        return s
    s.update(_paged_batch(case, gen, filled=True))
    if op == "tree":
        masks, _ = _trees(case, seed)
        s["masks"] = torch.tensor(masks, dtype=torch.int64, device="cuda")
        s["q"] = _randn(gen, s["n"], HQ, D, scale=2.0)  # scores of spread 2: some keys stand out
        s["out"] = torch.empty_like(s["q"])
        return s
    # compact: a path of the tree, its rows in rising order
    lens = lengths(case)
    width = min(case["rows"], 16)
    keep = torch.zeros(len(lens), width, dtype=torch.int32)
    counts = []
    state = (seed * 2654435761 + 777) & 0xFFFFFFFF
    for b, (_, t) in enumerate(lens):
        at, k = -1, 0
        while k < width:
            state = (state * 1664525 + 1013904223) & 0xFFFFFFFF
            at += 1 + (state >> 24) % 5
            if at >= t:
                break
            keep[b, k] = at
            k += 1
        counts.append(k)
    s["keep"] = keep.cuda()
    s["keepCounts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# The plain form
# ---------------------------------------------------------------------------
def _rows(s):
    """The sequence of every packed row, and its index there."""
    r = torch.arange(s["n"], device="cuda")
    b = torch.searchsorted(s["rowStart"][1:].contiguous(), r, right=True)
    return b, r - s["rowStart"].long()[b]


def _slots(s, b, token):
    """Row of the flattened page pool that holds the sequence's token."""
    return s["table"].long()[b, token // PAGE] * PAGE + token % PAGE


def _norm_rotate(x, weight, positions, table, pairing):
    x = x.float()
    if weight is not None:
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight
    row = table[positions]
    cos, sin = row[:, None, :D // 2], row[:, None, D // 2:]
    if pairing == 0:  # halves: (d, d + 32)
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]  # neighbours: (2 d, 2 d + 1)
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _plain_norm(s):
    pos = s["positions"].long()
    s["qOut"].copy_(_norm_rotate(s["q"], s["qWeight"], pos, s["cosSin"], s["pairing"]))
    s["kOut"].copy_(_norm_rotate(s["k"], s["kWeight"], pos, s["cosSin"], s["pairing"]))
    return {"q": s["qOut"], "k": s["kOut"]}


def _plain_append(s):
    b, i = _rows(s)
    token = s["ctx"].long()[b] + i
    pos = token if s["positions"] is None else s["positions"].long()
    at = _slots(s, b, token)
    k = _norm_rotate(s["k"], s["kWeight"], pos, s["cosSin"], s["pairing"])
    s["kPages"].view(-1, HKV, D)[at] = k.to(s["kPages"].dtype)
    s["vPages"].view(-1, HKV, D)[at] = s["v"].float().to(s["vPages"].dtype)
    if s["q"] is not None:
        s["qOut"].copy_(_norm_rotate(s["q"], s["qWeight"], pos, s["cosSin"], s["pairing"]))
    return {"k": s["kPages"], "v": s["vPages"], "q": s["qOut"]}


def _plain_tree(s):
    b, i = _rows(s)
    batch, most = s["table"].shape[0], s["max_rows"]
    page = s["table"].long().clamp(min=0)
    k = s["kPages"][page].flatten(1, 2).float()  # [batch][keys][8][64]
    v = s["vPages"][page].flatten(1, 2).float()
    keys = k.shape[1]
    q = torch.zeros(batch, most, HQ, D, device="cuda")
    q[b, i] = s["q"]
    mask = torch.zeros(batch, most, dtype=torch.int64, device="cuda")
    mask[b, i] = s["masks"]
    q = q.view(batch, most, HKV, GROUP, D).permute(0, 2, 1, 3, 4).reshape(batch, HKV, most * GROUP, D)
    score = q @ k.permute(0, 2, 3, 1) * 0.125
    ctx = s["ctx"].long()
    rows = (s["rowStart"][1:] - s["rowStart"][:-1]).long()
    j = torch.arange(keys, device="cuda")[None, :] - ctx[:, None]  # < 0: cached, else the drafted row
    drafted = (mask[:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1 == 1
    seen = (j < 0)[:, None, :] | (drafted & ((j >= 0) & (j < rows[:, None]))[:, None, :])
    seen = seen[:, None, :, None, :].expand(batch, HKV, most, GROUP, keys).reshape(score.shape)
    score = score.masked_fill_(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (score - top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(batch, HKV, most, GROUP, D).permute(0, 2, 1, 3, 4).reshape(batch, most, HQ, D)
    s["out"].copy_(o[b, i])
    return s["out"]


def _plain_compact(s):
    batch, width = s["keep"].shape
    b = torch.arange(batch, device="cuda")[:, None].expand(batch, width)
    i = torch.arange(width, device="cuda")[None, :].expand(batch, width)
    used = i < s["keepCounts"].long()[:, None]
    ctx = s["ctx"].long()[:, None]
    rows = (s["rowStart"][1:] - s["rowStart"][:-1]).long()[:, None]
    i = torch.minimum(i, rows - 1)  # places past a short sequence's rows stay with its last
    source = torch.where(used, s["keep"].long(), i)
    to, source = _slots(s, b, ctx + i), _slots(s, b, ctx + source)
    for pool in (s["kPages"], s["vPages"]):
        flat = pool.view(-1, HKV, D)
        moved = flat[source]
        flat[to] = torch.where(used[..., None, None], moved, flat[to])
    return {"k": s["kPages"], "v": s["vPages"]}


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _own_run(s):
    import chunked_prefill_gqa_gb300 as cp
    if s["op"] == "norm":
        cp.attn_qk_norm_rope(s["q"], s["k"], s["positions"], s["cosSin"], s["qOut"], s["kOut"],
                             qWeight=s["qWeight"], kWeight=s["kWeight"], eps=EPS, pairing=s["pairing"])
        return {"q": s["qOut"], "k": s["kOut"]}
    bf16 = s["kPages"].dtype == torch.bfloat16
    if s["op"] == "append":
        call = cp.attn_append_paged_bf16kv if bf16 else cp.attn_append_paged
        call(s["k"], s["v"], s["kPages"], s["vPages"], s["table"], s["ctx"], s["rowStart"], s["cosSin"],
             positions=s["positions"], kWeight=s["kWeight"], q=s["q"], qOut=s["qOut"], qWeight=s["qWeight"],
             eps=EPS, pairing=s["pairing"])
        return {"k": s["kPages"], "v": s["vPages"], "q": s["qOut"]}
    if s["op"] == "tree":
        if "workspace" not in s:  # a program keeps one for all of its batches, as large as any of them asks for
            need = cp.attn_tree_workspace_bytes(s["table"].shape[0], s["n"], s["max_rows"], s["max_context"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        call = cp.attn_tree_paged_bf16kv if bf16 else cp.attn_tree_paged
        return call(s["q"], s["kPages"], s["vPages"], s["table"], s["ctx"], s["rowStart"], s["masks"], s["out"],
                    s["max_rows"], s["max_context"], workspace=s["workspace"])
    call = cp.attn_compact_paged_bf16kv if bf16 else cp.attn_compact_paged
    call(s["kPages"], s["vPages"], s["table"], s["ctx"], s["keep"], s["keepCounts"], s["max_rows"])
    return {"k": s["kPages"], "v": s["vPages"]}


def run(s):
    if own:
        return _own_run(s)
    if s["op"] == "norm":
        return _plain_norm(s)
    if s["op"] == "append":
        return _plain_append(s)
    if s["op"] == "tree":
        return _plain_tree(s)
    return _plain_compact(s)


# ---------------------------------------------------------------------------
# Work and exact values
# ---------------------------------------------------------------------------
def work(case):
    size = {"f32": 4, "bf16": 2}
    op = case["op"]
    if op == "norm":
        n, head = case["n"], D
        read = n * (HQ + HKV) * head * size[case["act"]] + n * 4 + n * head * 4 + 2 * head * 4
        write = n * (HQ * head * 4 + HKV * head * size[case["cache"]])
        return {"bytes": read + write, "flops": 9 * n * (HQ + HKV) * head}
    lens = lengths(case)
    n, elem = sum(t for _, t in lens), size[case["cache"]]
    tables = 4 * sum((c + t + PAGE - 1) // PAGE for c, t in lens) + 8 * len(lens)
    if op == "append":
        heads = 2 * HKV + (HQ if case["normed"] else 0)
        rotated = HKV + (HQ if case["normed"] else 0)
        read = n * heads * D * size[case["act"]] + n * D * 4
        write = n * 2 * HKV * D * elem + (n * HQ * D * 4 if case["normed"] else 0)
        return {"bytes": read + write + 8 * len(lens) + 4 * n, "flops": (9 if case["normed"] else 3) * n * rotated * D}
    if op == "tree":
        keys = sum(c + t for c, t in lens)
        # Every row sees its sequence's cache and, of the drafted rows, a few ancestors.
        pairs = sum(t * c for c, t in lens)
        return {"bytes": keys * 2 * HKV * D * elem + 2 * n * HQ * D * 4 + 8 * n + tables,
                "flops": 4 * D * HQ * pairs}
    kept = sum(min(16, max(1, t // 3)) for _, t in lens)  # a path's rows, about
    return {"bytes": 4 * kept * HKV * D * elem + 12 * len(lens) + 4 * kept, "flops": 0}


def _exact_rotated(x, weight, positions, table, pairing):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * weight.double()
    half = D // 2
    first = torch.arange(half, device=x.device) if pairing == 0 else 2 * torch.arange(half, device=x.device)
    second = first + (half if pairing == 0 else 1)
    y = torch.empty_like(x)
    c, s = table.double()[positions, :half].unsqueeze(1), table.double()[positions, half:].unsqueeze(1)
    y[:, :, first] = c * x[:, :, first] - s * x[:, :, second]
    y[:, :, second] = s * x[:, :, first] + c * x[:, :, second]
    return y


def _exact_tree(s, case):
    out = torch.zeros(s["n"], HQ, D, dtype=torch.float64, device="cuda")
    masks, r = s["masks"].tolist(), 0
    for b, (c, t) in enumerate(lengths(case)):
        token = torch.arange(c + t, device="cuda")
        place = s["table"][b].long()[token // PAGE]
        k, v = (s[p][place, token % PAGE].double() for p in ("kPages", "vPages"))
        seen = torch.ones(t, c + t, dtype=torch.bool)
        for i in range(t):
            for j in range(t):
                seen[i, c + j] = bool(masks[r + i] >> j & 1)
        hidden = ~seen.cuda()
        for h in range(HQ):
            e = (s["q"][r:r + t, h].double() @ k[:, h // GROUP].T) / 8.0
            p = torch.softmax(e.masked_fill(hidden, -math.inf), -1)
            out[r:r + t, h] = p @ v[:, h // GROUP]
        r += t
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        pos = s["positions"].long()
        return {n: _exact_rotated(s[n], s[n + "Weight"], pos, s["cosSin"], s["pairing"]) for n in ("q", "k")}
    if op == "tree":
        return _exact_tree(s, case)
    pool = {n: s[n + "Pages"].double().clone() for n in ("k", "v")}
    if op == "append":
        token, page = [], []
        table = s["table"].tolist()
        for b, (c, t) in enumerate(lengths(case)):
            token += range(c, c + t)
            page += [table[b][j // PAGE] for j in range(c, c + t)]
        token, page = torch.tensor(token, device="cuda"), torch.tensor(page, device="cuda")
        pos = token if s["positions"] is None else s["positions"].long()
        pool["k"][page, token % PAGE] = _exact_rotated(s["k"], s["kWeight"], pos, s["cosSin"], s["pairing"])
        pool["v"][page, token % PAGE] = s["v"].double()
        pool["q"] = None if s["q"] is None else _exact_rotated(s["q"], s["qWeight"], pos, s["cosSin"], s["pairing"])
        return pool
    table, keep, counts = s["table"].tolist(), s["keep"].tolist(), s["keepCounts"].tolist()
    for b, (c, _) in enumerate(lengths(case)):
        for i in range(counts[b]):  # rising rows: none is overwritten before it is read
            a, z = c + keep[b][i], c + i
            for p in pool.values():
                p[table[b][z // PAGE], z % PAGE] = p[table[b][a // PAGE], a % PAGE]
    return pool
