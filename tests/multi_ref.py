"""Plain fp64 forms of the operators with several queries per sequence, and the
batches their tests use.  Shares no code with the kernels."""
import numpy as np
import torch

KINDS = ("mask", "chain", "cross")


def random_tree(rng, c):
    """Parents of c nodes: node 0 the root, the others below any earlier node."""
    p = np.array([int(rng.integers(max(0, r - 6), r)) if r else -1 for r in range(c)], np.int64)
    return p


def ancestors(parents):
    """[c, c] bool: row r is set at r and its ancestors."""
    c = len(parents)
    see = np.zeros((c, c), bool)
    for r in range(c):
        if parents[r] >= 0:
            see[r] = see[parents[r]]
        see[r, r] = True
    return see


def mask_words(rows, words):
    """Bit rows [c, <= 64 words] as int64 [c, words]."""
    c = len(rows)
    out = np.zeros((c, words), np.uint64)
    for r in range(c):
        for j in np.flatnonzero(rows[r]):
            out[r, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out.view(np.int64)


class Batch:
    """Sequences of lens[i] tokens with news[i] queries each over a shuffled pool;
    every slot that belongs to no token holds NaN, every table entry without a
    token junk.  kind: "mask" (see[i] [c, c] over the last c tokens), "chain",
    "cross"."""

    def __init__(self, kind, lens, news, Hq, Hkv, hd, bs, dtype, seed, see=None, padding=0, spare=3):
        rng = np.random.default_rng(seed)
        self.kind, self.lens, self.news, self.bs, self.dtype = kind, list(lens), list(news), bs, dtype
        per = [-(-n // bs) for n in lens]
        nb, width = sum(per) + spare, max(1, max(per))
        perm = rng.permutation(nb)
        self.tables = rng.choice([-1, 2**31 - 1, nb, -2**31], size=(len(lens), width)).astype(np.int32)
        live, at = np.zeros((nb, bs), bool), 0
        for i, n in enumerate(lens):
            self.tables[i, :per[i]] = perm[at:at + per[i]]
            at += per[i]
            t = np.arange(n)
            live[self.tables[i, t // bs], t % bs] = True
        self.start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        T = int(self.start[-1]) + padding
        g = torch.Generator().manual_seed(seed)
        self.k, self.v = (torch.randn(nb, Hkv, bs, hd, generator=g).to(dtype).masked_fill_(
            ~torch.from_numpy(live)[:, None, :, None], float("nan")) for _ in range(2))
        self.q = torch.randn(T, Hq, hd, generator=g).to(dtype)
        self.q[int(self.start[-1]):] = float("nan")
        self.see = see
        if kind == "mask" and see is None:
            self.see = [ancestors(random_tree(rng, c)) for c in news]
        self.words = max(1, -(-max([1, *news]) // 64))
        self.mask = None
        if kind == "mask":
            rows = [mask_words(s, self.words) for s in self.see]
            self.mask = torch.from_numpy(np.concatenate([*rows, np.full((padding, self.words), -1, np.int64)]))

    def visible(self, i):
        """[c, n] bool: what sequence i's queries see."""
        n, c = self.lens[i], self.news[i]
        if self.kind == "cross":
            return np.ones((c, n), bool)
        if c > n:
            return np.zeros((c, n), bool)
        see = np.ones((c, n), bool)
        see[:, n - c:] = np.tri(c, dtype=bool) if self.kind == "chain" else self.see[i]
        return see

    def reference(self, scale):
        """fp64 [tokens, Hq, hd]; rows that see nothing are zero."""
        q, k, v = (x.double().numpy() for x in (self.q, self.k, self.v))
        Hq, Hkv = q.shape[1], k.shape[1]
        out = np.zeros((int(self.start[-1]), Hq, q.shape[2]))
        nb = k.shape[0]
        for i, n in enumerate(self.lens):
            t, see = np.arange(n), self.visible(i)
            blk = self.tables[i][t // self.bs]
            ok = ((blk >= 0) & (blk < nb))[:, None, None]          # a bad block id reads as zeros
            ki = np.where(ok, k[np.where(ok[:, 0, 0], blk, 0), :, t % self.bs], 0.0)
            vi = np.where(ok, v[np.where(ok[:, 0, 0], blk, 0), :, t % self.bs], 0.0)
            for r in range(self.news[i]):
                w = see[r]
                if not w.any():
                    continue
                row = int(self.start[i]) + r
                for h in range(Hq):
                    kh = h // (Hq // Hkv)
                    x = scale * (ki[w, kh] @ q[row, h])
                    e = np.exp(x - x.max())
                    with np.errstate(invalid="ignore"):
                        out[row, h] = (e @ vi[w, kh]) / e.sum()
        return torch.from_numpy(out)

    def on_gpu(self, pa, scale, out=None, **kw):
        """(out, flags) of the kernel; rows behind the last sequence start as 7."""
        status = pa.DeviceStatus()
        if out is None:
            out = torch.full_like(self.q, 7.0).cuda()
        args = [out, self.q.cuda(), self.k.cuda(), self.v.cuda(), torch.from_numpy(self.tables).cuda(),
                torch.tensor(self.lens, dtype=torch.int32).cuda(), torch.from_numpy(self.start).cuda(), scale]
        kw.setdefault("max_context_len", max(1, max(self.lens)))
        if self.kind == "cross":
            pa.pa_decode_cross(*args, status=status, **kw)
        else:
            pa.pa_decode_tree(*args, tree_mask=None if self.mask is None else self.mask.cuda(), status=status, **kw)
        torch.cuda.synchronize()
        return out, status.read()


def accept(n, c, draft, target, parents, most, slot):
    """(length, nodes, next token, new length, pairs) of one tree, in plain Python."""
    path = [0] if c else []
    while path and len(path) < most:
        kids = [r for r in range(c) if parents[r] == path[-1] and draft[r] == target[path[-1]]]
        if not kids:
            break
        path.append(kids[0])
    pad = [-1] * (most - len(path))
    pairs = [(slot(n - c + r), slot(n - c + j)) if r != j else (-1, -1) for j, r in enumerate(path)]
    return (len(path), path + pad, target[path[-1]] if path else -1, n - c + len(path),
            pairs + [(-1, -1)] * len(pad))
