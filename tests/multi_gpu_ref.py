"""fp64 attention of several queries per sequence in torch operations on the GPU, with the sizes that a bound on a
result's error needs.  Shares no code with the kernels."""
import numpy as np
import torch


def attend(q, k, v, scale, see=None):
    """Of one sequence: q [c, Hq, hd], k and v [n, Hkv, hd], see [c, n] bool or None.

    (out, spread, size, total): out [c, Hq, hd]; spread [c, Hq, hd] = sum w |v| / sum w; size [c, Hq] = the largest
    scale * sum |q_d k_d| of a seen position; total [c, Hq] = sum w over the largest w.  Rows that see nothing are zero."""
    c, Hq, hd = q.shape
    n, Hkv, _ = k.shape
    group = Hq // Hkv
    out, spread = (torch.zeros(c, Hq, hd, dtype=torch.float64, device=q.device) for _ in range(2))
    size, weights = (torch.zeros(c, Hq, dtype=torch.float64, device=q.device) for _ in range(2))
    if n == 0 or c == 0:
        return out, spread, size, weights
    for h in range(Hkv):
        rows = q[:, h * group:(h + 1) * group].double()
        kh, vh = k[:, h].double(), v[:, h].double()
        x, y = (torch.einsum("cgd,nd->cgn", a, b) * s for a, b, s in ((rows, kh, scale), (rows.abs(), kh.abs(), abs(scale))))
        if see is not None:
            x = x.masked_fill(~see[:, None], -float("inf"))
            y = y.masked_fill(~see[:, None], 0.0)
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(top == -float("inf"), 0.0, top))
        total = e.sum(-1, keepdim=True).clamp_min(1e-300)
        at = slice(h * group, (h + 1) * group)
        out[:, at] = torch.einsum("cgn,nd->cgd", e, vh) / total
        spread[:, at] = torch.einsum("cgn,nd->cgd", e, vh.abs()) / total
        size[:, at] = y.amax(-1)
        weights[:, at] = e.sum(-1)
    return out, spread, size, weights


def batch(b, scale):
    """The same of a multi_ref.Batch, all sequences' rows end to end."""
    parts = []
    for i, n in enumerate(b.lens):
        rows = b.q[int(b.start[i]):int(b.start[i + 1])].cuda()
        t = np.arange(n)
        at = torch.from_numpy(b.tables[i][t // b.bs]).long(), slice(None), torch.from_numpy(t % b.bs)
        see = None if b.kind == "cross" else torch.from_numpy(b.visible(i)).cuda()
        parts.append(attend(rows, b.k[at].cuda(), b.v[at].cuda(), scale, see))
    return tuple(torch.cat(x) for x in zip(*parts))


def repeated(b, times):
    """The batch with all of its sequences `times` times, over the same blocks: enough tiles that each CTA walks many."""
    T = int(b.start[-1])
    b.q = torch.cat([b.q[:T]] * times + [b.q[T:]])
    b.start = np.concatenate([[0], np.cumsum(np.tile(b.news, times))]).astype(np.int32)
    b.lens, b.news, b.tables = b.lens * times, b.news * times, np.tile(b.tables, (times, 1))
    if b.see is not None:
        b.see = list(b.see) * times
    if b.mask is not None:
        b.mask = torch.cat([b.mask[:T]] * times + [b.mask[T:]])
    return b


def bf16_bound(out, spread, size, n, hd):
    """How far a bf16 result may be off, elementwise: its own rounding (2^-8); weights in two bf16 parts (2^-16 of
    themselves) and their exponential (2^-21); scores, whose products are exact and whose sums of hd take hd / 8 fp32
    steps of 2^-22 of the sum of sizes (a tensor core cuts off where additions round), and e to them, in numerator and
    denominator; sums over n tokens, in n / 16 such steps."""
    weight = 2.0 ** -16 + 2.0 ** -21 + 2 * (hd / 8) * 2.0 ** -22 * size[..., None] + (n / 16 + 8) * 2.0 ** -22
    return 2.0 ** -8 * out.abs() + (1 + 2.0 ** -8) * weight * spread


def f32_bound(out, spread, size, n, hd):
    """How far an fp32 result may be off, elementwise.  A product in two tf32 parts a side: 2^-21 of itself (2^-22 for the
    product of the small parts, 2^-23 for what each side's parts leave out).  Eight of them in the tensor core, each cut
    off at 2^-23 of the largest: 2^-20 of their sizes' sum.  Sums of hd in hd / 8 rounded steps and one for scale * q:
    2^-24 each.  Weights: e to the score's error, and 2^-22 for the exponential; in numerator and denominator.  Sums over
    n tokens in n / 8 rounded steps, and eight for the joins."""
    product = 2.0 ** -21 + 2.0 ** -20
    weight = torch.expm1(size[..., None] * (product + (hd / 8 + 1) * 2.0 ** -24)) + 2.0 ** -22
    return (2 * weight + product + (n / 8 + 8) * 2.0 ** -24) * spread + 2.0 ** -23 * out.abs()
