"""Batches for the serving-step calls (norm, rotation, append, drafted-tree
attention, compaction) and their plain forms in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

HQ, HKV, D, PAGE = 32, 8, 64, 16


def make_batch(lens, bf16=False, seed=0, spare=3, num_pages=None, extra_blocks=0):
    """A paged batch: lens = [(context, rows)]. The pools are NaN everywhere but
    in the sequences' tokens; table entries past a sequence's pages are -1."""
    rng = np.random.default_rng(seed)
    pages = [(c + t + PAGE - 1) // PAGE for c, t in lens]
    total = num_pages or sum(pages) + spare
    perm = (total - 1 - np.arange(sum(pages)) if num_pages else rng.permutation(total)[:sum(pages)]).astype(np.int32)
    width = max([1] + pages) + extra_blocks
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    dtype = torch.bfloat16 if bf16 else torch.float32
    kp = torch.full((total, PAGE, HKV, D), float("nan"), dtype=dtype, device="cuda")
    vp = torch.full((total, PAGE, HKV, D), float("nan"), dtype=dtype, device="cuda")
    for b, (c, t) in enumerate(lens):
        if c + t == 0:
            continue
        tok = np.arange(c + t)
        pg, sl = torch.from_numpy(table[b, tok // PAGE].astype(np.int64)).cuda(), torch.from_numpy(tok % PAGE).cuda()
        kp[pg, sl] = torch.from_numpy(rng.standard_normal((c + t, HKV, D), dtype=np.float32)).cuda().to(dtype)
        vp[pg, sl] = torch.from_numpy(rng.standard_normal((c + t, HKV, D), dtype=np.float32)).cuda().to(dtype)
    starts = np.concatenate([[0], np.cumsum([t for _, t in lens])]).astype(np.int32)
    return {"lens": list(lens), "kp": kp, "vp": vp, "table": torch.from_numpy(table).cuda(),
            "ctx": torch.tensor([c for c, _ in lens], dtype=torch.int32, device="cuda"),
            "starts": torch.from_numpy(starts).cuda(), "n": int(starts[-1]),
            "max_rows": max([1] + [t for _, t in lens]), "max_context": max([0] + [c for c, _ in lens])}


def tree_masks(lens, kind="tree", seed=0):
    """int64 masks, one a row: "tree" (itself and its ancestors), "chain", "self",
    "empty" (no drafted row), "mixed" (any bits, also of later rows and past the last)."""
    rng = np.random.default_rng(seed + 99)
    out = []
    for _, t in lens:
        m = []
        for i in range(t):
            if kind == "chain":
                x = (2 << i) - 1
            elif kind == "self":
                x = 1 << i
            elif kind == "empty":
                x = 0
            elif kind == "mixed":
                x = int(rng.integers(0, 1 << 63)) * 2 + int(rng.integers(0, 2))
            else:
                p = i - int(rng.integers(1, 5))
                x = (m[p] if p >= 0 else 0) | 1 << i
            m.append(x & (1 << 64) - 1)
        out += m
    return np.array(out, dtype=np.uint64).view(np.int64)


def gather(pool, table_row, n):
    tok = torch.arange(n, device="cuda")
    return pool[table_row.long()[tok // PAGE], tok % PAGE].double()


def tree_reference(q, batch, masks):
    """(out, tolerance) in fp64. The tolerance counts the roundings of a kernel
    that keeps fp32 precision on split operands:
      - a product keeps all but 2^-19 of |x y| (two tf32 terms each: the dropped
        lo lo below 2^-20, two truncated lo parts of 2^-21; three bf16 terms drop
        less), a score's chain of 24 accumulations at most 2^-23 each of A =
        sum |q_d k_d| / 8: d_j = (2^-19 + 24 2^-23) A_j;
      - the exponent's argument, (|s| + |m|) log2 e, rounds three times at 2^-24,
        e^x itself and the weights of merged partials within 2^-21:
        eps_j = d_j + 3 2^-24 (|s_j| + |m|) + 2^-21, twice in the quotient;
      - p v: 2^-19 and a chain of 6 accumulations, then one rounded addition a
        page of a warp (four warps at least share the pages), 80 for the merges.
    """
    out = torch.zeros(batch["n"], HQ, D, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    masks = np.asarray(masks).view(np.uint64)
    r = 0
    for b, (c, t) in enumerate(batch["lens"]):
        if t == 0:
            continue
        k, v = gather(batch["kp"], batch["table"][b], c + t), gather(batch["vp"], batch["table"][b], c + t)
        seen = np.ones((t, c + t), dtype=bool)
        for i in range(t):
            seen[i, c:] = (masks[r + i] >> np.arange(t, dtype=np.uint64)) & np.uint64(1)
        seen = torch.from_numpy(seen).cuda()
        qb = q[r:r + t].double()
        for h in range(HQ):
            kh, vh = k[:, h // 4], v[:, h // 4]
            s = (qb[:, h] @ kh.T / 8).masked_fill(~seen, float("-inf"))
            m = s.amax(-1, keepdim=True)
            m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
            p = torch.exp(s - m0)
            l = p.sum(-1, keepdim=True)
            l1 = torch.where(l > 0, l, torch.ones_like(l))
            out[r:r + t, h] = (p @ vh) / l1
            A = (qb[:, h].abs() @ kh.abs().T / 8).masked_fill(~seen, 0.0)
            eps = (2.0 ** -19 + 24 * 2.0 ** -23) * A + 3 * 2.0 ** -24 * (s.masked_fill(~seen, 0.0).abs() + m0.abs()) \
                + 2.0 ** -21
            pages = (c + t) / PAGE / 4 + 80
            tol[r:r + t, h] = (2 * eps.amax(-1, keepdim=True) + 2.0 ** -19 + 6 * 2.0 ** -23 + pages * 2.0 ** -24) \
                * (p @ vh.abs()) / l1
        r += t
    return out, tol


def norm_rotate_reference(x, weight, positions, table, pairing, eps):
    """(y, tolerance without the store's rounding) in fp64. The norm's factor: the
    sum of squares rounds at most 10 times (half of that under the root), the
    root's reciprocal is within 2 ulp = 4 half steps, two products; the rotation
    rounds a product and a sum: 12 half steps of 2^-24 in |a| + |b|, with a table
    of |cos|, |sin| <= 1. Without a norm only the rotation's two are left."""
    x = x.double()
    steps = 2.0
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
        steps = 12.0
    if table is None:
        return x, steps * 2.0 ** -24 * x.abs()
    cos, sin = table.double()[positions, None, :32], table.double()[positions, None, 32:]
    y, tol = torch.empty_like(x), torch.empty_like(x)
    a, b = (slice(0, 32), slice(32, 64)) if pairing == 0 else (slice(0, 64, 2), slice(1, 64, 2))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    tol[..., a] = tol[..., b] = steps * 2.0 ** -24 * (x[..., a].abs() + x[..., b].abs())
    return y, tol


def stored(y, tol, dtype):
    """The tolerance of y once it is stored in dtype: half a step more for bf16."""
    return tol + (2.0 ** -8 * y.abs() if dtype == torch.bfloat16 else 0.0) + 1e-37
