"""What is measured of the operators that keep a long cache within bounds, and of
rows whose positions have several axes: cases, inputs, the operators' plain form,
their exact values and the work they cannot do without.

On the framework's shapes (32 query heads, 8 key/value heads, head dimension 64,
16-token pages):

  axes    per-head RMS norm and the rotation of rows with several positions each
          (time, height, width), into contiguous keys (``attn_qk_norm_rope_axes``)
          or into a paged cache (``attn_append_paged_axes[_bf16kv]``)
  decode  attention of one new token a sequence over its paged cache, which also
          adds what each cached token was given to that token's weight
          (``attn_decode_weigh_paged[_bf16kv]``)
  weigh   the same weights from the last rows of a prompt, a window of up to 64,
          without their attention (``attn_weigh_paged[_bf16kv]``)
  evict   the tokens of least weight leave the cache, per key/value head, and the
          others close up (``attn_evict_paged[_bf16kv]``)

Weights are fp32 [pages][8][16] beside the pages: of every cached token and
key/value head the sum, over rows and the head's four query heads, of the
probabilities that the token was given.
"""
import math

import numpy as np
import torch

own = False

HQ, HKV, D, PAGE = 32, 8, 64, 16
GROUP = HQ // HKV
EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
# Which of the axes (time, height, width) turns each of the 32 pairs of dims.
AXES = {"sections": [0] * 8 + [1] * 12 + [2] * 12, "interleaved": [i % 3 for i in range(32)]}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def axes_case(name, batch, rows, context, ragged, act, cache, pairing, layout, paged):
    return {"name": name, "op": "axes", "batch": batch, "rows": rows, "context": context, "ragged": ragged, "act": act,
            "cache": cache, "pairing": pairing, "layout": layout, "paged": paged}


def decode_case(name, batch, context, ragged, cache, decay):
    return {"name": name, "op": "decode", "batch": batch, "rows": 1, "context": context, "ragged": ragged,
            "cache": cache, "decay": decay}


def weigh_case(name, batch, rows, context, ragged, cache, decay):
    return {"name": name, "op": "weigh", "batch": batch, "rows": rows, "context": context, "ragged": ragged,
            "cache": cache, "decay": decay}


def evict_case(name, batch, context, ragged, cache, keep, first, last):
    return {"name": name, "op": "evict", "batch": batch, "rows": 0, "context": context, "ragged": ragged,
            "cache": cache, "keep": keep, "first": first, "last": last}


def listed():
    return [
        # A few rows of text behind an image, contiguous keys: latency.
        axes_case("axes norm 7 rows", 1, 7, 0, False, "f32", "f32", 0, "sections", False),
        # The serving chunk, 2048 rows of a video, behind 2048 cached tokens.
        axes_case("axes append chunk 2048", 1, 2048, 2048, False, "bf16", "bf16", 0, "interleaved", True),
        # Images of up to 500 patches for 16 sequences at once.
        axes_case("axes append 16x500", 16, 500, 1000, True, "f32", "f32", 1, "sections", True),
        # A decode step of one short sequence: latency.
        decode_case("decode 1 at 1000", 1, 1000, False, "f32", 1.0),
        # The decode benchmark's batch.
        decode_case("decode 16 at 16384", 16, 16384, False, "bf16", 1.0),
        # A busy server's ragged sequences, old weights fading.
        decode_case("decode 48 to 4096", 48, 4096, True, "f32", 0.97),
        # One long document.
        decode_case("decode 1 at 131071", 1, 131071, False, "bf16", 1.0),
        # The last rows of a short prompt: latency.
        weigh_case("weigh 1x8 at 1000", 1, 8, 1000, False, "f32", 1.0),
        # The last 32 rows of the prompts of a batch.
        weigh_case("weigh 16x32 at 16384", 16, 32, 16384, False, "f32", 1.0),
        # The widest window over one long document.
        weigh_case("weigh 1x64 at 131071", 1, 64, 131071, False, "bf16", 0.0),
        # One short sequence back to half its length: latency.
        evict_case("evict 1 at 1000", 1, 1000, False, "f32", 0.5, 4, 64),
        # Half of the decode benchmark's batch leaves.
        evict_case("evict 16 at 16384", 16, 16384, False, "bf16", 0.5, 4, 128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("axes", "axes", "decode", "decode", "weigh", "weigh", "evict", "evict"))
    cache, ragged = rng.choice(("f32", "bf16")), rng.random() < 0.6
    batch = _log_int(rng, 1, 64)
    if op == "axes":
        paged = rng.random() < 0.7
        batch = batch if paged else 1
        rows = _log_int(rng, 1, 8192 // batch)
        context = _log_int(rng, 1, min(16384, 262144 // batch)) if paged else 0
        c = axes_case("", batch, rows, context, ragged and paged, rng.choice(("f32", "bf16")), cache, rng.randrange(2),
                      rng.choice(sorted(AXES)), paged)
    elif op == "decode":
        c = decode_case("", batch, _log_int(rng, 1, min(131071, 262144 // batch)), ragged, cache, rng.choice((0.0, 0.9, 1.0)))
    elif op == "weigh":
        rows = _log_int(rng, 1, min(64, 512 // batch))
        most = min(131071, 262144 // batch, (1 << 23) // (batch * rows) - rows)
        c = weigh_case("", batch, rows, _log_int(rng, 1, most), ragged, cache, rng.choice((0.0, 0.9, 1.0)))
    else:
        c = evict_case("", batch, _log_int(rng, 16, min(131071, 262144 // batch)), ragged, cache, rng.uniform(0.1, 0.95),
                       rng.randrange(9), rng.randrange(257))
    del c["name"]
    return c


def lengths(case):
    """(context, rows) of every sequence: from the case alone, the same for every seed."""
    got = []
    for b in range(case["batch"]):
        c, t = case["context"], case["rows"]
        if case["ragged"] and b:
            f, g = (b * 0.6180339887498949) % 1.0, (b * 0.7548776662466927) % 1.0
            c, t = max(1, int(c * (0.1 + 0.9 * f))), math.ceil(t * max(g, 0.01))
        got.append((c, t))
    return got


def kept(case):
    """(tokens to keep, first ones that stay, last ones that stay) of every sequence of an eviction."""
    got = []
    for c, _ in lengths(case):
        keep = max(1, int(c * case["keep"]))
        got.append(keep)
    least = min(got)
    first = min(case["first"], least)
    return got, first, min(case["last"], least - first)


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


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _paged_batch(case, gen):
    """The cache of a batch: shuffled pages, the block table, lengths and row starts."""
    lens = lengths(case)
    own_token = case["op"] == "decode"  # whose context counts the new token, already in the cache
    pages = [(c + (0 if own_token else t) + PAGE - 1) // PAGE for c, t in lens]
    total = sum(pages) + 3
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor([sum(pages[:b]) for b in range(len(pages))], device="cuda")
    count = torch.tensor(pages, device="cuda")
    j = torch.arange(max(pages), device="cuda")
    at = (first[:, None] + j[None, :]).clamp(max=total - 1)
    # The last entries of a short sequence's row of the table hold no page.
    table = torch.where(j[None, :] < count[:, None], perm[at], torch.full_like(perm[at], -1)).contiguous()
    dtype = DTYPES[case["cache"]]
    starts = [0]
    for _, t in lens:
        starts.append(starts[-1] + t)
    s = {"kPages": _randn(gen, total, PAGE, HKV, D, dtype=dtype), "table": table, "ctx": _ints([c for c, _ in lens]),
         "rowStart": _ints(starts), "n": starts[-1], "max_rows": case["rows"], "max_context": case["context"]}
    if case["op"] != "weigh":
        s["vPages"] = _randn(gen, total, PAGE, HKV, D, dtype=dtype)
    if case["op"] != "axes":
        # What earlier steps left, of the size of what a pass adds: heavy-tailed, a few tokens
        # far above the others, and some that no row has given anything to.
        w = _randn(gen, total, HKV, PAGE, scale=2.0).exp_() * (max(1, case["rows"]) / case["context"])
        s["weights"] = w * (torch.rand(w.shape, generator=gen, device="cuda") > 0.1)
    return s


def _grid_positions(n, gen):
    """[3][n]: frames of 16 x 24 patches with a few rows of text (the same on every axis) between them."""
    i = torch.arange(n, device="cuda")
    frame, patch = i // 392, i % 392
    text = patch >= 384
    start = frame * 32 + int(torch.randint(0, 1000, (1,), generator=gen, device="cuda"))
    t, h, w = start, start + patch // 24, start + patch % 24
    flat = start + 24 + patch - 384
    return torch.stack([torch.where(text, flat, x) for x in (t, h, w)]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op == "axes":
        act = DTYPES[case["act"]]
        s = _paged_batch(case, gen) if case["paged"] else {"n": case["rows"]}
        n = s["n"]
        s.update(op=op, pairing=case["pairing"], axes=AXES[case["layout"]], paged=case["paged"])
        s["axisOf"] = torch.tensor(s["axes"], device="cuda")
        s["positions"] = _grid_positions(n, gen)
        s["cosSin"] = rotation_table(n // 392 * 32 + 1100)
        s["q"] = _randn(gen, n, HQ + 1, D, dtype=act)[:, :HQ]
        kv = _randn(gen, n, 2 * HKV, D, dtype=act)
        s["k"], s["v"] = kv[:, :HKV], kv[:, HKV:]
        s["qOut"] = torch.empty(n, HQ, D, device="cuda")
        if not case["paged"]:
            s["kOut"] = torch.empty(n, HKV, D, device="cuda", dtype=DTYPES[case["cache"]])
        s["qWeight"] = 1.0 + _randn(gen, D, scale=0.1)
        s["kWeight"] = 1.0 + _randn(gen, D, scale=0.1)
        return s
    s = _paged_batch(case, gen)
    s["op"] = op
    # Every entry of the table that holds a page, as (sequence, entry).
    s["used"] = (s["table"] >= 0).nonzero().T.contiguous()
    if op == "evict":
        keep, s["first"], s["last"] = kept(case)
        s["keep"] = _ints(keep)
        s["before"] = s["weights"].clone()  # the weights as the steps before this one left them
        return s
    s["decay"] = case["decay"]
    s["q"] = _randn(gen, s["n"], HQ, D, scale=2.0)  # scores of spread 2: some keys stand out
    if op == "decode":
        s["out"] = torch.empty_like(s["q"])
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


def _norm_rotate(x, weight, pos, table, pairing):
    """pos [N][32]: the position that turns each pair of dims."""
    x = x.float()
    x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight
    i = torch.arange(D // 2, device="cuda")
    cos, sin = table[pos, i][:, None], table[pos, i + D // 2][:, None]
    if pairing == 0:  # halves: (d, d + 32)
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]  # neighbours: (2 d, 2 d + 1)
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _plain_axes(s):
    pos = s["positions"].long()[s["axisOf"]].T
    q = _norm_rotate(s["q"], s["qWeight"], pos, s["cosSin"], s["pairing"])
    k = _norm_rotate(s["k"], s["kWeight"], pos, s["cosSin"], s["pairing"])
    s["qOut"].copy_(q)
    if not s["paged"]:
        s["kOut"].copy_(k)
        return {"q": s["qOut"], "k": s["kOut"]}
    b, i = _rows(s)
    at = _slots(s, b, s["ctx"].long()[b] + i)
    s["kPages"].view(-1, HKV, D)[at] = k.to(s["kPages"].dtype)
    s["vPages"].view(-1, HKV, D)[at] = s["v"].float().to(s["vPages"].dtype)
    return {"q": s["qOut"], "k": s["kPages"], "v": s["vPages"]}


def _probabilities(s, q, visible):
    """[batch][8][rows * 4][keys]: q [batch][rows][32][64], visible [batch][rows][keys]."""
    batch, rows = q.shape[:2]
    page = s["table"].long().clamp(min=0)
    k = s["kPages"][page].flatten(1, 2).float()
    q = q.view(batch, rows, HKV, GROUP, D).permute(0, 2, 1, 3, 4).reshape(batch, HKV, rows * GROUP, D)
    score = q @ k.permute(0, 2, 3, 1) * 0.125
    visible = visible[:, None, :, None, :].expand(batch, HKV, rows, GROUP, k.shape[1]).reshape(score.shape)
    score = score.masked_fill_(~visible, float("-inf"))
    p = (score - score.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _add_weights(s, given, weighed, last):
    """given [batch][8][keys] joins the weights of tokens below last; those from weighed on had none."""
    batch, keys = given.shape[0], given.shape[2]
    page = s["table"].long().clamp(min=0)
    old = s["weights"][page].permute(0, 2, 1, 3).reshape(batch, HKV, keys)
    j = torch.arange(keys, device="cuda")[None, None, :]
    had = torch.where(j < weighed[:, None, None], old * s["decay"], torch.zeros_like(old)) if s["decay"] else 0.0
    new = torch.where(j < last[:, None, None], had + given, old)
    new = new.view(batch, HKV, keys // PAGE, PAGE).permute(0, 2, 1, 3)
    b, e = s["used"]
    s["weights"][page[b, e]] = new[b, e]
    return s["weights"]


def _plain_decode(s):
    ctx = s["ctx"].long()
    batch, keys = s["table"].shape[0], s["table"].shape[1] * PAGE
    visible = (torch.arange(keys, device="cuda")[None, :] < ctx[:, None])[:, None, :]
    p = _probabilities(s, s["q"].view(batch, 1, HQ, D), visible)
    v = s["vPages"][s["table"].long().clamp(min=0)].flatten(1, 2).float()
    s["out"].copy_((p @ v.permute(0, 2, 1, 3)).reshape(batch, HQ, D))
    return {"out": s["out"], "weights": _add_weights(s, p.sum(2), ctx - 1, ctx)}


def _plain_weigh(s):
    b, i = _rows(s)
    ctx, rows = s["ctx"].long(), (s["rowStart"][1:] - s["rowStart"][:-1]).long()
    batch, keys, most = s["table"].shape[0], s["table"].shape[1] * PAGE, s["max_rows"]
    q = torch.zeros(batch, most, HQ, D, device="cuda")
    q[b, i] = s["q"]
    r, j = torch.arange(most, device="cuda")[None, :, None], torch.arange(keys, device="cuda")[None, None, :]
    visible = (j <= ctx[:, None, None] + r) & (r < rows[:, None, None])
    p = _probabilities(s, q, visible)
    return _add_weights(s, p.sum(2), ctx, ctx + rows)


def _sources(s):
    """[batch][8][tokens]: the token that each token's place takes its key, value and weight from."""
    ctx, keep = s["ctx"].long()[:, None, None], s["keep"].long()[:, None, None]
    page = s["table"].long().clamp(min=0)
    w = s["weights"][page].permute(0, 2, 1, 3).flatten(2)
    batch, _, n = w.shape
    t = torch.arange(n, device="cuda").expand(batch, HKV, n)
    new = torch.minimum(ctx, keep)
    middle = (t >= s["first"]) & (t < ctx - s["last"])
    order = torch.sort(torch.where(middle, w, torch.full_like(w, -1.0)), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, t)
    stays = middle & (rank < new - s["first"] - s["last"])
    edge = new - s["last"]
    hole, mover = middle & ~stays & (t < edge), stays & (t >= edge)
    # The i-th hole takes the i-th mover.
    place = torch.where(mover, mover.cumsum(-1) - 1, torch.full_like(t, n))
    listed_ = torch.zeros(batch, HKV, n + 1, dtype=torch.long, device="cuda").scatter_(-1, place, t)
    source = torch.where(hole, listed_.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), t)
    return torch.where((t >= edge) & (t < new), t + ctx - new, source)


def _plain_evict(s):
    s["weights"].copy_(s["before"])
    source = _sources(s)
    b, e = s["used"]
    token = e[:, None] * PAGE + torch.arange(PAGE, device="cuda")  # [pages][16]
    source = source[b[:, None], :, token]                         # [pages][16][8]
    head = torch.arange(HKV, device="cuda")
    slot = _slots(s, b[:, None, None], source)
    page = s["table"].long()[b, e]
    for pool in (s["kPages"], s["vPages"]):
        pool[page] = pool.view(-1, HKV, D)[slot, head]
    s["weights"][page] = s["weights"][slot // PAGE, head, slot % PAGE].permute(0, 2, 1)
    return {"k": s["kPages"], "v": s["vPages"], "weights": s["weights"]}


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _workspace(s, bytes_of, *sizes):
    if "workspace" not in s:  # a program asks once and keeps one for all of its steps
        need = bytes_of(*sizes)
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    return s["workspace"]


def _own_run(s):
    import chunked_prefill_gqa_gb300 as cp
    op = s["op"]
    if op == "axes" and not s["paged"]:
        cp.attn_qk_norm_rope_axes(s["q"], s["k"], s["positions"], s["axes"], s["cosSin"], s["qOut"], s["kOut"],
                                  qWeight=s["qWeight"], kWeight=s["kWeight"], eps=EPS, pairing=s["pairing"])
        return {"q": s["qOut"], "k": s["kOut"]}
    bf16 = s["kPages"].dtype == torch.bfloat16
    if op == "axes":
        call = cp.attn_append_paged_axes_bf16kv if bf16 else cp.attn_append_paged_axes
        call(s["k"], s["v"], s["kPages"], s["vPages"], s["table"], s["ctx"], s["rowStart"], s["cosSin"], s["positions"],
             s["axes"], kWeight=s["kWeight"], q=s["q"], qOut=s["qOut"], qWeight=s["qWeight"], eps=EPS,
             pairing=s["pairing"])
        return {"q": s["qOut"], "k": s["kPages"], "v": s["vPages"]}
    batch = s["table"].shape[0]
    if op == "decode":
        ws = _workspace(s, cp.attn_decode_weigh_workspace_bytes, batch, s["max_context"])
        call = cp.attn_decode_weigh_paged_bf16kv if bf16 else cp.attn_decode_weigh_paged
        call(s["q"], s["kPages"], s["vPages"], s["weights"], s["table"], s["ctx"], s["out"], s["max_context"],
             decay=s["decay"], workspace=ws)
        return {"out": s["out"], "weights": s["weights"]}
    if op == "weigh":
        ws = _workspace(s, cp.attn_weigh_workspace_bytes, batch, s["n"], s["max_rows"], s["max_context"])
        call = cp.attn_weigh_paged_bf16kv if bf16 else cp.attn_weigh_paged
        return call(s["q"], s["kPages"], s["weights"], s["table"], s["ctx"], s["rowStart"], s["max_rows"],
                    s["max_context"], decay=s["decay"], workspace=ws)
    s["weights"].copy_(s["before"])
    ws = _workspace(s, cp.attn_evict_workspace_bytes, batch, s["max_context"])
    call = cp.attn_evict_paged_bf16kv if bf16 else cp.attn_evict_paged
    call(s["kPages"], s["vPages"], s["weights"], s["table"], s["ctx"], s["keep"], s["max_context"],
         keep_first=s["first"], keep_last=s["last"], workspace=ws)
    return {"k": s["kPages"], "v": s["vPages"], "weights": s["weights"]}


def run(s):
    if own:
        return _own_run(s)
    return {"axes": _plain_axes, "decode": _plain_decode, "weigh": _plain_weigh, "evict": _plain_evict}[s["op"]](s)


# ---------------------------------------------------------------------------
# Work and exact values
# ---------------------------------------------------------------------------
def work(case):
    op, lens, elem = case["op"], lengths(case), SIZE[case["cache"]]
    n = sum(t for _, t in lens)
    if op == "axes":
        heads = HQ + (2 * HKV if case["paged"] else HKV)
        read = n * heads * D * SIZE[case["act"]] + 3 * 4 * n + 4 * 64 * (n // 392 * 32 + 1100) + 2 * 4 * D
        write = n * (heads - HQ) * D * elem + n * HQ * D * 4
        return {"bytes": read + write, "flops": 9 * n * (HQ + HKV) * D}
    token_kv = 2 * HKV * D * elem
    if op == "decode":
        keys = sum(c for c, _ in lens)
        tables = 4 * sum((c + PAGE - 1) // PAGE for c, _ in lens) + 4 * len(lens)
        weights = keys * HKV * 4 * (2 if case["decay"] else 1)
        return {"bytes": keys * token_kv + weights + 2 * n * HQ * D * 4 + tables, "flops": 4 * D * HQ * keys}
    if op == "weigh":
        keys = sum(c + t for c, t in lens)
        pairs = sum(t * c + t * (t + 1) // 2 for c, t in lens)
        tables = 4 * sum((c + t + PAGE - 1) // PAGE for c, t in lens) + 8 * len(lens)
        weights = keys * HKV * 4 * (2 if case["decay"] else 1)
        return {"bytes": keys * token_kv // 2 + weights + n * HQ * D * 4 + tables, "flops": 2 * D * HQ * pairs}
    keep, first, last = kept(case)
    read = moved = 0
    for (c, _), k in zip(lens, keep):
        new = min(c, k)
        middle = c - first - last
        if new < c and middle > 0:
            read += c
            # Of the kept middle tokens, as many lie behind the new end as its share of the middle;
            # the last ones follow.
            stay = new - first - last
            moved += stay * (middle - stay) // middle + last
    return {"bytes": read * HKV * 4 + moved * 2 * (token_kv + HKV * 4), "flops": 0}


def _exact_rotated(x, weight, pos, table, pairing):
    x = x.double()
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * weight.double()
    y = torch.empty_like(x)
    for i in range(D // 2):
        a, b = (i, i + D // 2) if pairing == 0 else (2 * i, 2 * i + 1)
        c, s = table[pos[i], i].double()[:, None], table[pos[i], D // 2 + i].double()[:, None]
        y[:, :, a] = c * x[:, :, a] - s * x[:, :, b]
        y[:, :, b] = s * x[:, :, a] + c * x[:, :, b]
    return y


def _exact_given(s, case):
    """Yields (sequence, head, probabilities in 64 bits [rows][keys], page, slot of its keys)."""
    r = 0
    for b, (c, t) in enumerate(lengths(case)):
        n = c if case["op"] == "decode" else c + t
        token = torch.arange(n, device="cuda")
        page, slot = s["table"][b].long()[token // PAGE], token % PAGE
        k = s["kPages"][page, slot].double()
        limit = torch.arange(t, device="cuda")[:, None] + (c if case["op"] == "weigh" else c - 1)
        for h in range(HQ):
            e = (s["q"][r:r + t, h].double() @ k[:, h // GROUP].T) / 8.0
            yield b, r, h, torch.softmax(e.masked_fill(token[None, :] > limit, -math.inf), -1), page, slot
        r += t


def exact(case, seed):
    s = prepare(case, seed)
    op, lens = case["op"], lengths(case)
    if op == "axes":
        pos = [s["positions"][a].long() for a in s["axes"]]
        q, k = (_exact_rotated(s[n], s[n + "Weight"], pos, s["cosSin"], s["pairing"]) for n in ("q", "k"))
        if not case["paged"]:
            return {"q": q, "k": k}
        pool = {n: s[n + "Pages"].double() for n in ("k", "v")}
        table = s["table"].tolist()
        token = [j for c, t in lens for j in range(c, c + t)]
        page = torch.tensor([table[b][j // PAGE] for b, (c, t) in enumerate(lens) for j in range(c, c + t)], device="cuda")
        slot = torch.tensor(token, device="cuda") % PAGE
        pool["k"][page, slot], pool["v"][page, slot] = k, s["v"].double()
        return {"q": q, **pool}
    weights = s["weights"].double()
    if op in ("decode", "weigh"):
        out = torch.zeros(s["n"], HQ, D, dtype=torch.float64, device="cuda")
        for b, r, h, p, page, slot in _exact_given(s, case):
            g = h // GROUP
            if h % GROUP == 0:
                old = lens[b][0] - (1 if op == "decode" else 0)
                weights[page[:old], g, slot[:old]] *= case["decay"]
                weights[page[old:], g, slot[old:]] = 0.0
            weights[page, g, slot] += p.sum(0)
            if op == "decode":
                out[r:r + p.shape[0], h] = p @ s["vPages"][page, slot, g].double()
        return {"out": out, "weights": weights} if op == "decode" else weights
    pools = [s["kPages"].double(), s["vPages"].double()]
    keep, first, last = kept(case)
    for b, (c, _) in enumerate(lens):
        new = min(c, keep[b])
        token = torch.arange(c, device="cuda")
        page, slot = s["table"][b].long()[token // PAGE], token % PAGE
        for g in range(HKV):
            w = s["weights"][page, g, slot].cpu().numpy()
            middle = np.arange(first, c - last)
            best = middle[np.lexsort((middle, -w[middle]))][:new - first - last]
            stays = np.zeros(c, bool)
            stays[best] = True
            holes = [j for j in range(first, new - last) if not stays[j]]
            movers = np.flatnonzero(stays[new - last:]) + new - last
            source = np.arange(c)
            source[holes] = movers
            source[new - last:new] = np.arange(c - last, c)
            at = torch.from_numpy(source).cuda()
            for pool in pools:
                pool[page, slot, g] = pool[page[at], slot[at], g]
            weights[page, g, slot] = weights[page[at], g, slot[at]]
    return {"k": pools[0], "v": pools[1], "weights": weights}
