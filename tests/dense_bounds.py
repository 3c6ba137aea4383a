"""Bounds for long contexts, where the worst case of every key's rounding at once
(dense_cases.reference's tolerance) is wider than the results: keys' roundings
are independent, so what is checked is their rms.

``check_rms``: the error's rms over all outputs is at most twice that of rounding the
exact result once to bf16.  A probability held like a bf16 is off by as much,
relative to itself, as the output's own rounding; where few keys carry a row that
is as much again, sqrt(2) in all, and less where many do.

``check_units``: for every unit of 32 keys, the error's component along what the unit adds
to the result (sum p (v - out) over its keys) is a quarter of that at most, where an error
of the rms that check_rms allows makes it a tenth or less by chance; a unit left out gives -1, one taken twice +1.

``check_elements``: each output within its own half step of bf16 (2^-8 of itself) and the
same of sum_j p_j |v_j| for its probabilities, with what fp32 scores add (``ds``: their
absolute error, in the probability and in its normaliser; 2^-20 for exp2 and sums), and
with ``noise``: over FP8 caches a probability is held in two e4m3 parts whose last step is
2^-9 where the largest p x scale of a block is 2^7 to 2^9.  What lies below that step is
rounded to it, right on average, with a variance of at most a quarter of the step squared,
2^-20, a key, 2^-13 a block.  The kernel lowers its reference before such blocks number
64 sum (P / 2^7)^2 over the blocks' largest P (2^-21 of sum P^2, and as much again after it
fell), unless one within 2^2 of the reference came by in the last 8 blocks (P >= 2^5 then:
sum P^2 >= 2^10 in 8 blocks against a variance of 8 x 2^-13 = 2^-10, 2^-20 of it).  So the rms of
the sum of all roundings is at most 2^-10 sqrt(sum p^2) rms(v); six times that is not met once
in 10^8 outputs.
"""
import math

import torch


def rms(x):
    return math.sqrt(float((x.double() ** 2).mean()))


def check_rms(out, ref):
    err, once = rms(out.double() - ref), rms(ref.to(torch.bfloat16).double() - ref)
    assert err <= 2 * once, "rms error %.3e, %.2f times one rounding's" % (err, err / once)


def check_units(out, ref, p, v, unit=32):
    """out, ref: [heads, d_v] of one row; p: [heads, keys]; v: [keys, d_v]."""
    # in units of the output's own rounding, so that all heads count
    w = 1.0 / (ref.abs() + ref.pow(2).mean(-1, keepdim=True).sqrt())
    err = (out.double() - ref) * w
    noise = 2 * rms((ref.to(torch.bfloat16).double() - ref) * w)
    n = p.shape[1]
    tested = 0
    for j in range(0, n, unit):
        q = p[:, j:j + unit]
        d = (q @ v[j:j + unit] - q.sum(-1, keepdim=True) * ref) * w
        size = float((d ** 2).sum())
        if noise > 0.1 / 6 * math.sqrt(size):                # six sigma of chance past a tenth
            continue
        tested += 1
        a = float((err * d).sum()) / size
        assert abs(a) <= 0.25, "keys %d to %d: %.2f of what they add" % (j, min(j + unit, n) - 1, a)
    return tested


def seen_of(c, b, i, window=None, sinks=0):
    """(p [heads, keys], v [keys, d_v], out) in 64 bits of new token i of sequence b over the keys it sees."""
    L, n = c.lens[b], c.news[b]
    vis = min(max(L - n + i + 1, 0), L)
    pos = torch.arange(vis, device=c.q.device)
    if window is not None:
        pos = pos[(pos >= vis - window) | (pos < sinks)]
    k = c.lat.rows[b][pos]
    p = torch.softmax(c.scale * (c.q[sum(c.news[:b]) + i].double() @ k.T), -1)
    return p, k[:, :c.d_v], p @ k[:, :c.d_v]


def check_elements(out, lse, ref, z, mag, noise, ds):
    e = (out.double() - ref).abs() - (2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * ds + 2.0 ** -20) * mag + 6 * noise)
    assert bool((e <= 0).all()), "out: %.3e beyond its bound, %.1e of the rms" % (float(e.max()), float(e.max()) / rms(ref))
    e = (lse.double() - z).abs() - (ds + 2.0 ** -20 + 2.0 ** -22 * z.abs())
    assert bool((e <= 0).all()), "lse: %.3e beyond its bound" % float(e.max())


def exact_rows(c, rows):
    """(out, lse, sum p |v|, noise, ds) in 64 bits of some rows of a one-sequence call."""
    k = c.lat.rows[0]
    L, n = c.lens[0], c.rows
    res = []
    ds = 0.0
    for i in rows:
        x = k[:L - n + i + 1]
        q = c.q[i].double()
        s = c.scale * (q @ x.T)
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - z[:, None])
        size = p.pow(2).sum(-1).sqrt()[:, None] * x[:, :c.d_v].pow(2).mean(0).sqrt()
        res.append((p @ x[:, :c.d_v], z, p @ x[:, :c.d_v].abs(), 2.0 ** -10 * size if c.lat.fmt == 0 else 0 * size))
        ds = max(ds, abs(c.scale) * c.lat.D * 2.0 ** -23 * float((q.abs() @ x.abs().T).max()))
        if c.lat.fmt == 0:          # q in two e4m3 parts
            ds = max(ds, ds + abs(c.scale) * 2.0 ** -17 * float((q.abs().amax(-1) * x.abs().sum(-1).amax()).max()))
    return tuple(torch.stack(t) for t in zip(*res)) + (ds,)
