"""Plain 64-bit forms of the serving operators, and the error bounds their tests use.

Bounds count roundings, with u = eps / 2 of a type.  Of an attention output
sum_j p_j V_j with p = softmax(s), to first order:
  * an error of at most ds in every score moves each p_j by a factor within
    e^(+-2 ds) and the log sum by at most ds;
  * a relative error r in every exponential or weight moves the output by at
    most 2 r A, A = sum_j p_j |V_j| (once in the sum of weights, once in the
    weighted sum), and the log sum by r;
  * fp32 sums of n terms: n 2^-24 relative to the sum of magnitudes;
  * rounding the output: u |out|.
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}     # half a subnormal step
EXP = 2.0 ** -16          # relative error allowed to a kernel's own exponential


def softmax_rows(x):
    """Weights and log sums of rows that may be -inf throughout (weights 0, log sum
    -inf).  The maximum leaves before the sum, whose logarithm a maximum of the lowest
    fp32 values would absorb."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total), (m + torch.log(total))[..., 0]


def prompt(q, K, V, cu_q, cu_k, u_weights):
    """out, lse and their bounds for packed prompts (rows of no sequence: NaN)."""
    hq, total, d = q.shape
    group = hq // K.shape[0]
    out = torch.full((hq, total, d), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((hq, total), math.nan, dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for a, z, ka, kz in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        if z <= a:
            continue
        n = kz - ka
        i = torch.arange(z - a, device=q.device)[:, None] + n - (z - a)
        seen = torch.arange(n, device=q.device)[None] <= i
        for h in range(hq):
            if n == 0:
                out[h, a:z], lse[h, a:z] = 0.0, -math.inf
                continue
            qq, k, v = (t.double() for t in (q[h, a:z], K[h // group, ka:kz], V[h // group, ka:kz]))
            x = torch.where(seen, qq @ k.T / math.sqrt(d), -math.inf)
            p, lse[h, a:z] = softmax_rows(x)
            out[h, a:z] = p @ v
            # products of two 16-bit values are exact in fp32; d sums and two scalings
            mag = qq.abs() @ k.abs().T / math.sqrt(d)
            ds = (d + 4) * 2.0 ** -24 * torch.where(seen, mag, 0.0).amax(1, keepdim=True)
            rel = EXP + n * 2.0 ** -24 + ds
            tol[h, a:z] = (2 * rel + 2 * u_weights) * (p @ v.abs()) + U[q.dtype] * out[h, a:z].abs() + TINY[q.dtype]
            tol_lse[h, a:z] = rel[:, 0] + 2.0 ** -22 * lse[h, a:z].abs().nan_to_num(posinf=0.0)
    return out, lse, tol, tol_lse


def rotation(d, signs):
    """H diag(signs) / sqrt(d) in 64 bits."""
    h = torch.ones((1, 1), dtype=torch.float64, device=signs.device)
    while h.shape[0] < d:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h * signs.double()[None] / math.sqrt(d)


def unpack(idx, d, b):
    """Codes (..., d) of packed rows, bit by bit from the layout's definition."""
    bits = (idx[..., :, None].to(torch.int64) >> torch.arange(8, device=idx.device)) & 1
    bits = bits.reshape(idx.shape[:-1] + (d, b))
    return (bits << torch.arange(b, device=idx.device)).sum(-1)


def shared(q, pre, own, lengths, group, b, signs, cent, u_weights, u_cent):
    """out, lse and bounds; pre and own are (idx, norms, V); cent the codebook."""
    heads, n, d = pre[2].shape
    batch = len(lengths)
    rot = (q.double() @ rotation(d, signs).T).view(batch, heads, group, d) / math.sqrt(d)
    cent = cent.double()

    def keys(c, h, m):
        return cent[unpack(c[0][h, :m], d, b)] * c[1][h, :m].double()[:, None], c[2][h, :m].double()

    out = torch.zeros((batch, heads, group, d), dtype=torch.float64, device=q.device)
    lse = torch.zeros((batch, heads, group), dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    od = pre[2].dtype
    for h in range(heads):
        kp, vp = keys(pre, h, n)
        for s, m in enumerate(lengths):
            ko, vo = keys(own, s * heads + h, m)
            k, v = torch.cat([kp, ko]), torch.cat([vp, vo])
            if k.shape[0] == 0:
                lse[s, h] = -math.inf
                continue
            x = rot[s, h] @ k.T
            p, lse[s, h] = softmax_rows(x)
            out[s, h] = p @ v
            # the rotated query, each product, d sums, the norm: roundings of 2^-24, and
            # the rotation's own log2(d) additions of |q| sums
            mag = (rot[s, h].abs() @ k.abs().T).amax(1, keepdim=True)
            spread = rot[s, h].abs().amax(1, keepdim=True) * k.abs().sum(1).amax()
            ds = (d + 8) * 2.0 ** -24 * mag + u_cent * mag + 2.0 ** -21 * spread
            rel = EXP + k.shape[0] * 2.0 ** -24 + ds
            tol[s, h] = (2 * rel + 2 * u_weights) * (p @ v.abs()) + U[od] * out[s, h].abs() + TINY[od]
            tol_lse[s, h] = rel[:, 0] + 2.0 ** -22 * lse[s, h].abs()
    return out.view(-1, d), lse.view(-1), tol.view(-1, d), tol_lse.view(-1)


def weights(scores, start, group, lengths):
    """The sums after one step, and their bound."""
    out, tol = start.double().clone(), torch.zeros_like(start, dtype=torch.float64)
    for h, m in enumerate(lengths):
        if m == 0:
            continue
        p, _ = softmax_rows(scores[h * group:(h + 1) * group, :m].double())
        out[h, :m] += p.sum(0)
        # s - max rounds by 2^-24 |s - max|, which moves e^(s - max) by that much relatively
        x = scores[h * group:(h + 1) * group, :m].double()
        top = x.amax(1, keepdim=True)
        gap = torch.where(torch.isinf(x), torch.zeros_like(x), (x - torch.where(torch.isinf(top), 0.0, top)).abs())
        tol[h, :m] = (p * (2.0 ** -21 + 2.0 ** -23 * gap + 2 * m * 2.0 ** -24)).sum(0) + (group + 1) * 2.0 ** -24 * out[h, :m].abs()
    return out, tol


def evict(weights_h, length, keep, recent):
    """Rows of one head that stay, ascending (host arrays)."""
    if length <= keep:
        return list(range(length))
    old = length - recent
    rank = sorted(range(old), key=lambda t: (math.isnan(weights_h[t]), -weights_h[t] if not math.isnan(weights_h[t]) else 0.0, t))
    return sorted(rank[:keep - recent]) + list(range(old, length))
