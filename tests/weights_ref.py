"""Plain forms in 64 bits of the cache weights (decode step and window) and of the
eviction by them."""
from __future__ import annotations

import numpy as np
import torch

from spec_ref import D, HKV, HQ, PAGE, gather

GROUP = HQ // HKV


def weight_pool(batch, seed=0, known=None):
    """fp32 [pages][8][16]: NaN but for each sequence's first known[b] tokens (None: its context)."""
    rng = np.random.default_rng(seed + 7)
    w = torch.full((batch["kp"].shape[0], HKV, PAGE), float("nan"), device="cuda")
    for b, (c, _) in enumerate(batch["lens"]):
        n = c if known is None else known[b]
        put_weights(w, batch, b, np.exp(rng.standard_normal((n, HKV))).astype(np.float32) / 8)
    return w


def put_weights(pool, batch, b, values):
    """Weights [tokens][8] of sequence b's first tokens."""
    n = len(values)
    if n == 0:
        return
    tok = np.arange(n)
    page = batch["table"][b].long().cpu().numpy()[tok // PAGE]
    pool[torch.from_numpy(page).cuda()[:, None], torch.arange(HKV, device="cuda")[None], torch.from_numpy(tok % PAGE).cuda()[:, None]] = \
        torch.as_tensor(values, device="cuda", dtype=torch.float32)


def get_weights(pool, batch, b, n):
    """[n][8] of sequence b's first n tokens, as they are."""
    tok = torch.arange(n, device="cuda")
    page = batch["table"][b].long()[tok // PAGE]
    return pool[page[:, None], torch.arange(HKV, device="cuda")[None], (tok % PAGE)[:, None]]


def softmax_reference(q, k, seen):
    """(p, relative error of a row's p's) of one head in fp64: q [t][64], k [n][64], seen [t][n].

    As for attention of drafted rows: a product keeps all but 2^-19 of |x y|, a score's
    chain of at most 24 accumulations 2^-23 each of A = sum |q_d k_d| / 8; the exponent's
    argument rounds three times at 2^-24 of (|s| + |m|) log2 e, e^x and the factor that
    joins partial sums lie within 2^-21 each: eps_j, in the numerator and in the sum.
    The sum's own chains are at most n / 4 + 100 rounded additions of positive terms, and
    where it is kept as a logarithm, m log2 e + log2 sum <= 1.45 |m| + 20, that rounds
    twice at 2^-24 of it, in the exponent again."""
    s = (q @ k.T / 8).masked_fill(~seen, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.softmax(s, -1)
    A = (q.abs() @ k.abs().T / 8).masked_fill(~seen, 0.0)
    eps = (2.0 ** -19 + 24 * 2.0 ** -23) * A + 3 * 2.0 ** -24 * 1.45 * (s.masked_fill(~seen, 0.0).abs() + m.abs()) + 2.0 ** -21
    n = k.shape[0]
    rel = 2 * eps.amax(-1, keepdim=True) + (n / 4 + 100) * 2.0 ** -24 + 2.0 ** -23 * (1.45 * m.abs() + 20)
    return p, rel


def weigh_reference(q, batch, weights, weighed, decay, decode=False):
    """([b]: (weights [n][8], tolerance)), and with decode (out, tolerance): sequence b's
    rows q[first:first + t], the row i at token c + i (decode: the one row at c - 1)."""
    got, r = [], 0
    out = torch.zeros(q.shape[0], HQ, D, dtype=torch.float64, device="cuda")
    out_tol = torch.zeros_like(out)
    for b, (c, t) in enumerate(batch["lens"]):
        rows, n = (1, c) if decode else (t, c + t)
        if rows == 0 or n == 0:
            got.append(None)
            r += rows
            continue
        k = gather(batch["kp"], batch["table"][b], n)
        tok = torch.arange(n, device="cuda")
        seen = tok[None] <= (c - 1 if decode else c + torch.arange(rows, device="cuda")[:, None])
        old = get_weights(weights, batch, b, n).double()
        had = torch.where((tok < weighed[b])[:, None], old * decay if decay else torch.zeros_like(old), torch.zeros_like(old))
        w, tol = had.clone(), torch.zeros_like(had)
        for h in range(HQ):
            p, rel = softmax_reference(q[r:r + rows, h].double(), k[:, h // GROUP], seen.expand(rows, n))
            w[:, h // GROUP] += p.sum(0)
            tol[:, h // GROUP] += (p * rel).sum(0)
            if decode:
                v = gather(batch["vp"], batch["table"][b], n)[:, h // GROUP]
                out[r, h] = (p @ v)[0]
                # p v as 2^-19 and a chain of 6 accumulations; one addition a page of a warp, 80 for the merges
                out_tol[r, h] = ((rel + 2.0 ** -19 + 6 * 2.0 ** -23 + (n / PAGE / 4 + 80) * 2.0 ** -24) * (p @ v.abs()))[0]
        # The weight's own sum: 64 additions in a chain, one for each 32 rows, the old weight's product.
        tol += (70 + rows / 32) * 2.0 ** -24 * w
        got.append((w, tol))
        r += rows
    return (got, out, out_tol) if decode else got


def evict_reference(w, context, keep, first, last):
    """[min(keep, context)] the token that each kept place's key, value and weight come from,
    of one head: w [context] its weights. Equal weights by the lower token, NaN behind all."""
    if keep >= context:
        return np.arange(context)
    middle = np.arange(first, context - last)
    nan = np.isnan(w)
    value = np.where(nan, 0.0, w).astype(np.float64)
    order = np.lexsort((middle, -value[middle], nan[middle]))  # the last key counts first
    stays = np.zeros(context, dtype=bool)
    stays[middle[order][:keep - first - last]] = True
    edge = keep - last
    source = np.arange(keep)
    holes = [t for t in range(first, edge) if not stays[t]]
    movers = [t for t in range(edge, context - last) if stays[t]]
    assert len(holes) == len(movers)
    source[holes] = movers
    source[edge:] = np.arange(context - last, context)
    return source
