"""The smoke run's checks of a cache kept within bounds, on the CPU against plain forms of
the calls: right ones pass, and a mistake in any call's output is found."""
import numpy as np
import pytest

import __graft_entry__ as entry
import oracle

torch = pytest.importorskip("torch")


class Plain:
    """The calls in elementary operations on CPU tensors. `wrong` names one that is spoiled."""

    def __init__(self, wrong=None):
        self.wrong = wrong

    def _turned(self, x, weight, positions, axes, table):
        x = x.double()
        x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
        row = positions.long()[[0] * 32 if self.wrong == "one axis" else axes].T
        i = torch.arange(32)
        c, s = table.double()[row, i][:, None], table.double()[row, i + 32][:, None]
        a, b = x[..., :32], x[..., 32:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    def attn_qk_norm_rope_axes(self, q, k, positions, axes, table, q_out, k_out, qWeight, kWeight):
        q_out.copy_(self._turned(q, qWeight, positions, axes, table) + 0.1 * (self.wrong == "norm queries"))
        k_out.copy_(self._turned(k, kWeight, positions, axes, table))

    def attn_append_paged_axes(self, k, v, k_pages, v_pages, blocks, ctx, starts, table, positions, axes, kWeight, q, qOut, qWeight):
        rows = [(b, int(ctx[b]) + i) for b in range(len(ctx)) for i in range(int(starts[b + 1] - starts[b]))]
        at = torch.tensor([t for _, t in rows])
        page, slot = blocks.long()[torch.tensor([b for b, _ in rows]), at // 16], at % 16
        k_pages[page, slot] = self._turned(k, kWeight, positions, axes, table).to(k_pages.dtype)
        v_pages[page, slot] = (v * (1.02 if self.wrong == "append values" else 1.0)).to(v_pages.dtype)
        qOut.copy_(self._turned(q, qWeight, positions, axes, table))

    def attn_weigh_workspace_bytes(self, *sizes):
        return 0

    attn_decode_weigh_workspace_bytes = attn_evict_workspace_bytes = attn_weigh_workspace_bytes

    def _add(self, weights, blocks, b, known, n, decay, p):
        tok = torch.arange(n)
        page, slot = blocks[b].long()[tok // 16], tok % 16
        old = torch.where((tok < known)[:, None], weights[page, :, slot].double() * decay, 0.0)
        weights[page, :, slot] = (old + p.view(8, 4, n).sum(1).T).float()

    def _given(self, q, k):
        return torch.einsum("hd,thd->ht", q.double(), k.double().repeat_interleave(4, 1)).div(8).softmax(-1)

    def attn_weigh_paged(self, q, k_pages, weights, blocks, ctx, starts, rows, bound, decay, workspace):
        for b in range(len(ctx)):
            c, first, t = int(ctx[b]), int(starts[b]), int(starts[b + 1] - starts[b])
            assert c <= bound and t <= rows
            tok = torch.arange(c + t)
            k, p = k_pages[blocks[b].long()[tok // 16], tok % 16], torch.zeros(32, c + t, dtype=torch.float64)
            for i in range(t):
                n = c + t if self.wrong == "window mask" else c + i + 1
                p[:, :n] += self._given(q[first + i], k[:n])
            self._add(weights, blocks, b, c, c + t, 1.0 if self.wrong == "window decay" else decay, p)

    def attn_evict_paged(self, k_pages, v_pages, weights, blocks, ctx, keep, bound, keep_first, keep_last, workspace):
        for b in range(len(ctx)):
            n, m = int(ctx[b]), int(keep[b])
            assert n <= bound and keep_first + keep_last <= m
            tok = torch.arange(n)
            page, slot = blocks[b].long()[tok // 16], tok % 16
            for g in range(8):
                w = weights[page, g, slot].clone()
                middle = torch.argsort(-w[keep_first:n - keep_last], stable=True) + keep_first
                if self.wrong == "evict largest":
                    middle = middle.flip(0)
                stays = torch.cat([tok[:keep_first], middle[:m - keep_first - keep_last].sort()[0], tok[n - keep_last:]])
                for pages in (k_pages, v_pages)[:1 if self.wrong == "evict values" else 2]:
                    pages[page[:m], slot[:m], g] = pages[page[stays], slot[stays], g].clone()
                weights[page[:m], g, slot[:m]] = w[stays]

    def attn_decode_weigh_paged(self, q, k_pages, v_pages, weights, blocks, ctx, out, bound, decay, workspace):
        for b in range(len(ctx)):
            n = int(ctx[b])
            assert n <= bound
            tok = torch.arange(n)
            k, v = (x[blocks[b].long()[tok // 16], tok % 16].double() for x in (k_pages, v_pages))
            p = self._given(q[b], k)
            out[b] = torch.einsum("ht,thd->hd", p, v.repeat_interleave(4, 1)).float()
            self._add(weights, blocks, b, n if self.wrong == "decode known" else n - 1, n, decay, p)

    attn_append_paged_axes_bf16kv, attn_weigh_paged_bf16kv = attn_append_paged_axes, attn_weigh_paged
    attn_evict_paged_bf16kv, attn_decode_weigh_paged_bf16kv = attn_evict_paged, attn_decode_weigh_paged


def check(wrong):
    entry._compare(entry._bounded_cache(Plain(wrong), torch, np, device="cpu"), oracle, np)


def test_right_calls_pass():
    check(None)


@pytest.mark.parametrize("wrong", ["one axis", "norm queries", "append values", "window mask", "window decay",
                                   "evict largest", "evict values", "decode known"])
def test_a_mistake_is_found(wrong):
    with pytest.raises(RuntimeError, match="disagrees"):
        check(wrong)
