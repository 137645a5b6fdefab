"""Plain 64-bit implementations of the bounded-cache operators, and the error bounds their
tests hold the kernels to.  Written from the definitions in include/pagedkv.h with torch
double arithmetic on the CPU; no code of the library.

Error bound of an attention output o = sum_t p_t v_t / sum_t p_t, with A = sum_t p_t |v_t| /
sum_t p_t (computed per element in 64 bits):
  |got - o| <= u_out |o| + (u_p + 4 d + 2 n 2^-23) A + n 2^-24 max|v| [fp16 P only]
  u_out  half a step of the output type (bf16 2^-8, fp16 2^-11) for the one final rounding;
  u_p    half a step of what P is held in when it meets V (stated by each test);
  d      error of a score in the exponent: D products summed in 32 bits, each step off by at
         most 2^-23 of the sum of magnitudes S = |scale| sum_d |q_d k_d|, plus the rounding of
         the scaled score and exp's own 2^-22: d = (D + 4) 2^-23 max_t S_t + 2^-22; it enters
         numerator and denominator, and twice that covers the reference maximum's rounding;
  n 2^-23  the 32-bit sums over n positions of the numerator and of the denominator;
  n 2^-24 max|v|  fp16 weights below the type's normal range (half a step 2^-25, and the
         largest weight is at least 1/2).
"""
from __future__ import annotations

import torch

U_OUT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def visible(p, t, window, num_sinks):
    """bool [len(p), len(t)]: the token at position p sees position t."""
    p, t = p[:, None], t[None, :]
    return (t <= p) & ((t > p - window) | (t < num_sinks))


def attend(q, k, v, pos, window, num_sinks, scale, u_p, dtype):
    """One sequence: q [n, Hq, D] at positions pos [n], k and v [T, Hkv, D], all double.
    (out, bound), both [n, Hq, D]; a token that sees nothing has a zero row, exactly."""
    n, Hq, D = q.shape
    T, Hkv, _ = k.shape
    out = torch.zeros_like(q)
    bound = torch.zeros_like(q)
    if n == 0 or T == 0:
        return out, bound
    see = visible(pos, torch.arange(T), window, num_sinks)
    any_seen = see.any(0)
    # what nothing sees takes no part, whatever it holds
    k = torch.where(any_seen[:, None, None], k, torch.zeros_like(k))
    v = torch.where(any_seen[:, None, None], v, torch.zeros_like(v))
    g = Hq // Hkv
    for h in range(Hq):
        kh, vh = k[:, h // g], v[:, h // g]
        x = scale * (q[:, h] @ kh.T)
        x = torch.where(see, x, torch.full_like(x, -torch.inf))
        m = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
        z = e.sum(1, keepdim=True)
        ok = z > 0
        z = torch.where(ok, z, torch.ones_like(z))
        o = e @ vh / z
        a = e @ vh.abs() / z
        s = abs(scale) * (q[:, h].abs() @ kh.abs().T)      # magnitudes: a negative scale too
        s = torch.where(see, s, torch.zeros_like(s)).amax(1, keepdim=True)
        d = (D + 4) * 2.0 ** -23 * s + 2.0 ** -22
        cnt = see.sum(1, keepdim=True).double()
        b = U_OUT[dtype] * o.abs() + (u_p + 4 * d + 2 * cnt * 2.0 ** -23) * a
        if u_p >= 2.0 ** -11 and dtype == "f16":
            b = b + cnt * 2.0 ** -24 * vh.abs().amax()
        out[:, h] = torch.where(ok, o, torch.zeros_like(o))
        bound[:, h] = torch.where(ok, b * (1 + 2.0 ** -6), torch.zeros_like(b))
    return out, bound


def check(got, ref, bound, what=""):
    got = got.detach().double().cpu()
    err = (got - ref).abs()
    bad = ~(err <= bound)                        # a NaN is bad
    assert not bad.any(), "%s: %d of %d outside the bound, worst %.3g times it, at %s" % (
        what, int(bad.sum()), bad.numel(),
        float((err / bound.clamp(min=1e-30)).nan_to_num(1e30).max()), bad.nonzero()[0].tolist())
    return float((err / bound.clamp(min=1e-30)).max()) if err.numel() else 0.0


def block_scale(amax):
    """Smallest power of two s with amax / 448 <= s / 8 (amax / 448 rounded to binary32)."""
    y = float(torch.tensor(amax, dtype=torch.float32) / 448)
    if y == 0:
        return 1.0
    s = 2.0 ** -126
    while not y <= s / 8:
        s *= 2
    return s


def quantise_e4m3(x):
    """E4M3 number nearest to x (double tensor), ties to even, clamped to 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)
