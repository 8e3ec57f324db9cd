"""Batches over the 4-bit cache in which one warp holds whole long rows, for the
tests of its sums and weights.  More rows than the GPU has warps (2432 at
most are used) are not cut finer than about a row; all sequences share one
sequence's pages, so the pool stays small.

q is a multiple of ones per head and K is constant over each token's head row
(step 0), so a score is the token's K value times the head's multiple: chosen
freely, and exact."""
import numpy as np
import torch

import q4_ref

SEQS = 2500
CHECKED = (0, 1, 1249, 2499)     # sequence 0 lies in the first warp's stretch whole


class Shared:
    """One KV head, n tokens.  scores [n]: bf16 numbers; codes [n, hd], step and
    low [n, hd / group]: V's codes and parameters (bf16 numbers)."""

    def __init__(self, scores, codes, step, low, group, bs=32, heads=(1.0,)):
        n, hd = codes.shape
        self.group, self.bs, self.hd, self.n = group, bs, hd, n
        blocks = -(-n // bs)
        page, cut = q4_ref.page_bytes(hd, bs, group), bs * hd // 2
        rng = np.random.default_rng(n)
        order = rng.permutation(blocks)
        byte, shift = q4_ref.spot(hd)

        def cache(codes, step, low):
            out = np.zeros((blocks * bs, hd // 2), np.uint8)
            for d in range(hd):
                out[:n, byte[d]] |= (codes[:, d] << shift[d]).astype(np.uint8)
            par = np.zeros((blocks * bs, hd // group, 2), np.uint16)
            par[:n, :, 0], par[:n, :, 1] = q4_ref.bf16_bits(step), q4_ref.bf16_bits(low)
            pages = np.empty((blocks, page), np.uint8)
            pages[:, :cut] = out.reshape(blocks, cut)
            pages[:, cut:] = par.view(np.uint8).reshape(blocks, -1)
            shuffled = np.empty_like(pages)
            shuffled[order] = pages
            return torch.from_numpy(shuffled[:, None])

        groups = hd // group
        scores = np.asarray(scores, np.float64)
        self.k = cache(rng.integers(0, 16, (n, hd)), np.zeros((n, groups)), np.repeat(scores[:, None], groups, 1))
        self.v = cache(codes, step, low)
        self.table = torch.from_numpy(order.astype(np.int32))
        self.heads = torch.tensor(heads, dtype=torch.float64)
        rounded = lambda x: torch.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()
        self.scores = rounded(scores)
        self.step, self.low = rounded(step), rounded(low)
        self.values = codes * np.repeat(self.step, group, 1) + np.repeat(self.low, group, 1)

    def reference(self, window=0, sinks=0):
        """fp64 [heads, hd]."""
        t = np.arange(self.n)
        seen = (t >= self.n - window) | (t < sinks) if window else t >= 0
        out = []
        for a in self.heads.tolist():
            x = self.scores[seen] * a
            p = np.exp(x - x.max())
            out.append((p / p.sum()) @ self.values[seen])
        return np.array(out)

    def run(self, pa, dtype, seqs=SEQS, **kw):
        """[checked sequences, heads, hd] in fp64; every sequence's rows must be alike."""
        q = self.heads.to(dtype)[None, :, None].expand(seqs, -1, self.hd).contiguous().cuda()
        out = torch.full_like(q, float("nan"))
        status = pa.DeviceStatus()
        pa.pa_decode_q4(out, q, self.k.cuda(), self.v.cuda(),
                        self.table.cuda()[None].expand(seqs, -1).contiguous(),
                        torch.full((seqs,), self.n, dtype=torch.int32, device="cuda"), 1.0 / self.hd,
                        max_context_len=self.n, group_size=self.group, status=status, **kw)
        assert status.read() == 0 and torch.isfinite(out).all()
        return out[[s for s in CHECKED if s < seqs]].double().cpu().numpy()
