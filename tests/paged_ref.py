"""Plain 64-bit forms of the paged-cache operators and the error bounds that
their kernels' arithmetic allows, for the tests.

Half a step of a type t is eps(t) / 2 relative (torch.finfo(t).eps / 2).
Binary32 sums are counted at 2^-23 for each addition: twice the half step, so
that a matrix unit that truncates is covered too."""
import torch

F32 = 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def slots(table_row, n, page, device):
    t = torch.arange(n, device=device)
    return table_row.to(torch.int64)[t // page] * page + t % page


def rotate(x, cos_sin, pos, interleaved):
    """x [n, heads, d] float64, turned by rows `pos` of cos_sin; also the sum
    of the two products' magnitudes (for the bound)."""
    r = cos_sin.shape[1]
    cs = cos_sin.double()[pos]
    c, s = cs[:, None, : r // 2], cs[:, None, r // 2:]
    y, mag = x.clone(), torch.zeros_like(x)
    i = torch.arange(r // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = (a * c).abs() + (b * s).abs()
    mag[..., ib] = (b * c).abs() + (a * s).abs()
    return y, mag


def rotate_bound(y, mag, dtype):
    """One rounding to dtype of a value within 2 binary32 roundings of y: a
    product, then a fused product and sum.  2^-25: half a binary16 subnormal
    step."""
    return half_step(dtype) * (y.abs() + 2 * F32 * mag) + 2 * F32 * mag + 2.0 ** -25


def attend(q, k, v, pos, scale, window, cache_dtype, out_dtype, shift=14):
    """q [n, h, d], k, v [m, hk, d] (any type), pos [n] -> out, lse and their
    bounds, all float64.  Hidden tokens take no part, whatever they hold.
    shift: the power of two by which the kernel scales binary16 probabilities,
    14 for single tokens in 16-row tiles, 11 in the larger tiles."""
    n, h, d = q.shape
    m, hk, _ = k.shape
    g = h // hk
    q, k, v = q.double(), k.double(), v.double()
    out = torch.zeros((n, h, d), dtype=torch.float64, device=q.device)
    lse = torch.full((n, h), float("-inf"), dtype=torch.float64, device=q.device)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for i in range(n):
        p = int(pos[i])
        lo = max(0, p + 1 - window) if window else 0
        if p < 0:
            continue
        for j in range(hk):
            kk, vv = k[lo:p + 1, j], v[lo:p + 1, j]
            qq = q[i, j * g:(j + 1) * g]
            s = (qq[:, None, :] * kk[None]).sum(-1) * scale
            mag = (qq.abs()[:, None, :] * kk.abs()[None]).sum(-1) * abs(scale)
            e = torch.logsumexp(s, -1, keepdim=True)
            w = torch.exp(s - e)
            out[i, j * g:(j + 1) * g] = (w[..., None] * vv[None]).sum(1)
            lse[i, j * g:(j + 1) * g] = e[:, 0]
            # score: d products summed, the scale (times log2 e) rounded and
            # multiplied, the maximum subtracted and a constant added; q of a
            # bfloat16 model below binary16's normal range: 2^-25 absolute
            ds = (d + 6) * F32 * mag + 4 * F32 * (s - s.amax(-1, keepdim=True)).abs()
            ds = ds + 2.0 ** -25 * abs(scale) * kk.abs().sum(-1)[None] * (cache_dtype != out_dtype)
            cnt = p + 1 - lo
            # probability: the score's error, exp2 (4 steps), one rounding to
            # the cache's type; the sums: cnt terms and the rescalings
            rel = 2 * ds + 8 * F32 + half_step(cache_dtype) + 2 * cnt * F32
            mean = (w * ds).sum(-1, keepdim=True) + (2 * cnt + 8) * F32
            # binary16 probabilities below the normal range: half a step of
            # 2^-24 at a scale of 2^shift, against the probability at the
            # kernel's reference, which is at most the largest one: 2^-39 of
            # it at a shift of 14, 2^-36 at 11
            tail = 2.0 ** (-25 - shift) * w.amax(-1, keepdim=True)
            a = (((w * (rel + mean) + tail)[..., None]) * vv.abs()[None]).sum(1)
            o = out[i, j * g:(j + 1) * g]
            b_out[i, j * g:(j + 1) * g] = (a * 1.01 + half_step(out_dtype) * (o.abs() + a)
                                           + 2.0 ** -25)
            b_lse[i, j * g:(j + 1) * g] = (ds.amax(-1) + (2 * cnt + 8) * F32
                                           + 8 * F32 * (e[:, 0].abs() + 40))
    return out, lse, b_out, b_lse
