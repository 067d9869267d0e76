"""The smoke run's checks of the serving step, on the CPU against plain forms of the
calls: right ones pass, and a mistake in any call's output is found."""
import numpy as np
import pytest

import __graft_entry__ as entry
import oracle

torch = pytest.importorskip("torch")


class Plain:
    """The calls of the serving step in elementary operations on CPU tensors. `wrong`
    names one output that is spoiled."""

    def __init__(self, wrong=None):
        self.wrong = wrong

    def attn_rope_table(self, table):
        ang = torch.arange(table.shape[0], dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32) / 32.0).double()
        return table.copy_(torch.cat([ang.cos(), ang.sin()], 1) + 0.1 * (self.wrong == "table"))

    def _turned(self, x, weight, positions, table):
        x = x.double()
        x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
        c, s = table.double()[positions.long(), None, :32], table.double()[positions.long(), None, 32:]
        a, b = x[..., :32], x[..., 32:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    def attn_qk_norm_rope(self, q, k, positions, table, q_out, k_out, qWeight, kWeight):
        q_out.copy_(self._turned(q, qWeight, positions, table) + 0.1 * (self.wrong == "norm queries"))
        k_out.copy_(self._turned(k, kWeight, positions, table) + 0.1 * (self.wrong == "norm keys"))

    def attn_append_paged(self, k, v, k_pages, v_pages, blocks, ctx, starts, table, kWeight, q, qOut, qWeight):
        rows = [(b, int(ctx[b]) + i) for b in range(len(ctx)) for i in range(int(starts[b + 1] - starts[b]))]
        pos = torch.tensor([t for _, t in rows])
        at = pos + (self.wrong == "append slot")
        page, slot = blocks.long()[torch.tensor([b for b, _ in rows]), at // 16], at % 16
        key = k.double() if self.wrong == "append unnormed" else self._turned(k, kWeight, pos, table)
        k_pages[page, slot] = key.to(k_pages.dtype)
        v_pages[page, slot] = (v * (1.02 if self.wrong == "append values" else 1.0)).to(v_pages.dtype)
        if self.wrong == "append nothing else":
            k_pages[int(blocks[0, 0]), 0, 0, 0] += 1.0
        qOut.copy_(self._turned(q, qWeight, pos, table) + 0.1 * (self.wrong == "append queries"))

    def attn_tree_workspace_bytes(self, *sizes):
        return 0

    def attn_tree_paged(self, q, k_pages, v_pages, blocks, ctx, starts, masks, out, max_rows, bound, splits, workspace):
        for b in range(len(ctx)):
            c, t, first = int(ctx[b]), int(starts[b + 1] - starts[b]), int(starts[b])
            tok = torch.arange(c + t)
            k, v = (p[blocks[b].long()[tok // 16], tok % 16].double() for p in (k_pages, v_pages))
            seen = torch.ones(t, c + t, dtype=torch.bool)
            for i in range(t):
                seen[i, c:] = (masks[first + i] >> torch.arange(t)) & 1 == 1
            if self.wrong == "tree mask":
                seen[:, c:] = True
            for h in range(32):
                s = (q[first:first + t, h].double() @ k[:, h // 4].T / 8).masked_fill(~seen, float("-inf"))
                out[first:first + t, h] = (s.softmax(-1) @ v[:, h // 4]).float()

    def attn_compact_paged(self, k_pages, v_pages, blocks, ctx, keep, counts, max_rows):
        for pages in (k_pages, v_pages)[:1 if self.wrong == "compact values" else 2]:
            for b in range(len(ctx)):
                a, z = int(ctx[b]) + int(keep[b, 0]), int(ctx[b])
                pages[int(blocks[b, z // 16]), z % 16] = pages[int(blocks[b, a // 16]), a % 16].clone()

    attn_append_paged_bf16kv, attn_tree_paged_bf16kv = attn_append_paged, attn_tree_paged
    attn_compact_paged_bf16kv = attn_compact_paged


def check(wrong):
    entry._compare(entry._serving_step(Plain(wrong), torch, np, device="cpu"), oracle, np)


def test_right_calls_pass():
    check(None)


@pytest.mark.parametrize("wrong", ["table", "norm queries", "norm keys", "append unnormed", "append slot",
                                   "append values", "append nothing else", "append queries", "tree mask",
                                   "compact values"])
def test_a_mistake_is_found(wrong):
    with pytest.raises(RuntimeError, match="disagrees"):
        check(wrong)
