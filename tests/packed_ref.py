"""Plain fp64 implementations of the operators over packed sequences, with
elementwise error bounds, written from the formulas (no code of the library).

Bounds count the roundings that the operators document, each at most half a
step (bf16: 2^-8 relative), and fp32 arithmetic as SLACK = 2^-13 of the sum of
the terms' magnitudes (a 128-term fp32 dot product and a 2-ulp exp2 of an
argument below 2^5 stay below 160 * 2^-24 + 2^5 * 2^-22 < 2^-14)."""
import math

import torch

HALF = 2.0 ** -8          # bf16: half a step, relative
SLACK = 2.0 ** -13


def cu_of(lens, first=0):
    return torch.tensor([first] + [first + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)


def attention(q, k, v, cu_q, cu_k, causal, dout=None):
    """q [tq, hq, d], k, v [tk, hk, d] in fp64; returns a dict of results and of elementwise bounds (`*_tol`).
    Rows of no sequence are NaN in every result."""
    q, k, v = q.double(), k.double(), v.double()
    hq, hk, d = q.shape[1], k.shape[1], q.shape[2]
    g, c = hq // hk, 1 / math.sqrt(d)
    nan = lambda x: torch.full_like(x, math.nan)  # noqa: E731
    r = dict(out=nan(q), out_tol=nan(q), out32_tol=nan(q), lse=nan(q[..., 0]), lse_tol=nan(q[..., 0]))
    if dout is not None:
        dout = dout.double()
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            r[n], r[n + "_tol"] = nan(x), nan(x)
    for i in range(len(cu_q) - 1):
        sq, sk = slice(int(cu_q[i]), int(cu_q[i + 1])), slice(int(cu_k[i]), int(cu_k[i + 1]))
        nq, nk = sq.stop - sq.start, sk.stop - sk.start
        if dout is not None:
            for n in ("dk", "dv", "dk_tol", "dv_tol"):
                r[n][sk] = 0.0
        lim = torch.arange(nq, device=q.device) + (nk - nq) if causal else torch.full((nq,), nk, device=q.device)
        sees = torch.arange(nk, device=q.device)[None] <= lim[:, None]
        for h in range(hq):
            qh, kh, vh = q[sq, h], k[sk, h // g], v[sk, h // g]
            s = (qh @ kh.t() * c).masked_fill(~sees, -math.inf)
            mags = (qh.abs() @ kh.abs().t() * c).masked_fill(~sees, 0.0)
            m = s.amax(1, keepdim=True) if nk else torch.full((nq, 1), -math.inf, dtype=q.dtype, device=q.device)
            m = torch.where(torch.isfinite(m), m, 0.0)
            e = torch.exp(s - m)
            l = e.sum(1, keepdim=True)
            p = torch.where(l > 0, e / l.clamp_min(1e-300), 0.0)
            o, mag = p @ vh, p @ vh.abs()
            r["out"][sq, h], r["lse"][sq, h] = o, (torch.log2(l) + m / math.log(2))[:, 0]
            r["out32_tol"][sq, h] = (HALF + SLACK) * mag
            r["out_tol"][sq, h] = (HALF + SLACK) * mag + HALF * (o.abs() + (HALF + SLACK) * mag)
            most = mags.amax(1) if nk else torch.zeros(nq, dtype=q.dtype, device=q.device)
            r["lse_tol"][sq, h] = (d + 8) * 2.0 ** -24 * most / math.log(2) + 2.0 ** -19
            if dout is None:
                continue
            go = dout[sq, h]
            dp = go @ vh.t()
            delta = (go * o).sum(1, keepdim=True)
            ds = p * (dp - delta)
            # dS in the kernel: P and dP in fp32, D from the forward's fp32 output (whose P was bf16), dS rounded to bf16
            ds_tol = (HALF * ds.abs() + p * (go.abs() @ vh.abs().t() + (go.abs() * mag).sum(1, keepdim=True)) * 4 * SLACK
                      + p * (HALF + SLACK) * (go.abs() * mag).sum(1, keepdim=True))
            p_tol = (HALF + 4 * SLACK) * p
            kv = h // g
            r["dq"][sq, h] = ds @ kh * c
            r["dq_tol"][sq, h] = ds_tol @ kh.abs() * c
            r["dk"][sk, kv] += ds.t() @ qh * c
            r["dk_tol"][sk, kv] += ds_tol.t() @ qh.abs() * c
            r["dv"][sk, kv] += p.t() @ go
            r["dv_tol"][sk, kv] += p_tol.t() @ go.abs()
        if dout is not None:
            for n, sl in (("dq", sq), ("dk", sk), ("dv", sk)):
                t = r[n + "_tol"][sl]
                r[n + "_tol"][sl] = t + HALF * (r[n][sl].abs() + t)
    return r


def check(got, want, tol, what=""):
    """Every element within its bound, and where `want` is NaN (rows of no sequence) nothing."""
    got, want, tol = got.double().cpu(), want.cpu(), tol.cpu()
    own = ~torch.isnan(want)
    bad = own & ~((got == want) | ((got - want).abs() <= tol + 1e-30))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], tol[bad][:4])
