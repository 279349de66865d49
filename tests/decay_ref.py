"""Plain fp64 implementation of the linear attention with a decay per head over
packed sequences, with elementwise error bounds, written from the formulas (no
code of the library).

Bounds: each rounding to bf16 that the operator documents at most half a step
(2^-8 relative).  The state's update splits its operand into bf16 hi + lo (half
a step of a half step: 2^-16), its weights are 2-ulp exponentials of fp32
arguments of at most 2^7 (2^7 * 2^-23 = 2^-16), and its fp32 sum over 16
tokens at a time loses at most tokens / 16 * 2^-23 (2^-15 for 4096 tokens):
below 2^-14 of the sum of the terms' magnitudes, as is every other fp32 step."""
import math

import torch

HALF = 2.0 ** -8
SLACK = 2.0 ** -13
STATE = 2.0 ** -14
CHUNK = 128


def walk(a, b, c, log_decay, cu, first, back, w_scale=1.0, p_scale=1.0, s_scale=1.0):
    """out_i = p_scale sum_j lam^|i-j| (a_i.b_j) c_j + s_scale lam^e a_i first, j <= i and e = i + 1 (j >= i and
    e = n - 1 - i backwards); last = lam^n first + w_scale sum_j lam^(n-1-j) b_j^T c_j (lam^(j+1) backwards).
    Everything fp64 [total, h, d] / [n_seq, h, d, d]; rows of no sequence are NaN.  Returns out, tol, last, last_tol."""
    out, tol = torch.full_like(a, math.nan), torch.full_like(a, math.nan)
    last, last_tol = torch.zeros_like(first), torch.zeros_like(first)
    for s in range(len(cu) - 1):
        rows = slice(int(cu[s]), int(cu[s + 1]))
        n = rows.stop - rows.start
        i = torch.arange(n, dtype=torch.float64)
        for h in range(a.shape[1]):
            ld, x = log_decay[h].double().item(), first[s, h]
            power = lambda e: torch.where(e == 0, 1.0, torch.exp(ld * e)) if ld == -math.inf else torch.exp(ld * e)  # noqa: E731
            ah, bh, ch = a[rows, h], b[rows, h], c[rows, h]
            dist = (i[None] - i[:, None]) if back else (i[:, None] - i[None])
            m = torch.where(dist >= 0, power(dist.clamp_min(0)), 0.0)
            sc = ah @ bh.t() * m * p_scale
            e = power(n - 1 - i if back else i + 1)[:, None] * s_scale
            w = (power(i + 1 if back else n - 1 - i) * w_scale)[:, None]
            o = sc @ ch + e * (ah @ x)
            mag = (ah.abs() @ bh.abs().t() * m * abs(p_scale)) @ ch.abs() + e.abs() * (ah.abs() @ x.abs())
            t = SLACK * mag
            inside = (i[:, None] // CHUNK) == (i[None] // CHUNK)
            t = t + HALF * (sc.abs() * inside) @ ch.abs()
            for k0 in range(0, n, CHUNK):                 # the state at each chunk, as rounded to bf16
                k1 = min(n, k0 + CHUNK)
                if back:
                    y = power(torch.tensor(n - k1, dtype=torch.float64)) * x + ((power(i[k1:] + 1 - k1)[:, None] * bh[k1:]).t() @ ch[k1:]) * w_scale
                    f = power(k1 - 1 - i[k0:k1])
                else:
                    y = power(torch.tensor(k0, dtype=torch.float64)) * x + ((power(k0 - 1 - i[:k0])[:, None] * bh[:k0]).t() @ ch[:k0]) * w_scale
                    f = power(i[k0:k1] + 1 - k0)
                t[k0:k1] += HALF * abs(s_scale) * f[:, None] * (ah[k0:k1].abs() @ y.abs())
            out[rows, h], tol[rows, h] = o, t + HALF * (o.abs() + t)
            lam_n = power(torch.tensor(n, dtype=torch.float64))
            last[s, h] = lam_n * x + (bh * w).t() @ ch
            last_tol[s, h] = STATE * (lam_n * x.abs() + (bh.abs() * w.abs()).t() @ ch.abs())
    return out, tol, last, last_tol


def decay_attention(q, k, v, log_decay, cu, scale, state_in=None, dout=None, dstate_out=None):
    """Results and bounds (`*_tol`) of the forward and, with dout, of the gradients."""
    q, k, v = q.double(), k.double(), v.double()
    n, (h, d) = len(cu) - 1, q.shape[1:]
    zero = torch.zeros(n, h, d, d, dtype=torch.float64)
    s0 = zero if state_in is None else state_in.double()
    r = {}
    r["out"], r["out_tol"], r["state_out"], r["state_out_tol"] = walk(q, k, v, log_decay, cu, s0, False, 1.0, scale, scale)
    if dout is None:
        return r
    g = dout.double()
    r1 = zero if dstate_out is None else dstate_out.double()
    t = lambda x: x.transpose(-1, -2)  # noqa: E731
    r["dq"], r["dq_tol"], _, _ = walk(g, v, k, log_decay, cu, t(s0), False, 1.0, scale, scale)
    r["dk"], r["dk_tol"], _, _ = walk(v, g, q, log_decay, cu, t(r1), True, scale, scale, 1.0)
    r["dv"], r["dv_tol"], r["dstate_in"], r["dstate_in_tol"] = walk(k, q, g, log_decay, cu, r1, True, scale, scale, 1.0)
    return r


def recurrence(q, k, v, log_decay, cu, scale, state_in):
    """The definition, token by token, in fp64: out and the last states."""
    q, k, v = q.double(), k.double(), v.double()
    lam = torch.exp(log_decay.double())[:, None, None]
    out, last = torch.full_like(q, math.nan), state_in.double().clone()
    for s in range(len(cu) - 1):
        for t in range(int(cu[s]), int(cu[s + 1])):
            last[s] = lam * last[s] + k[t][:, :, None] * v[t][:, None, :]
            out[t] = scale * (q[t][:, None, :] @ last[s])[:, 0]
    return out, last
