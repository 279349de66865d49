"""Linear attention with a decay per head over long sequences: parts of several
chunks, several sums to a part, many borders to a sequence and walks of several
chunks one after another in a CTA, against a chunked fp64 form on the device."""
import math

import pytest
import torch

from decay_ref import CHUNK, HALF, SLACK, walk
from packed_ref import check, cu_of
from test_decay_attn import inputs, run, workspace
from test_packed_attn import ops  # noqa: F401  (a fixture)


def chunked_walk(a, b, c, log_decay, cu, first, back, w_scale=1.0, p_scale=1.0, s_scale=1.0):
    """What decay_ref.walk gives, with its bounds, for all heads at once and chunk by chunk (finite decays)."""
    out, tol, last, last_mag = torch.full_like(a, math.nan), torch.full_like(a, math.nan), first.clone(), first.abs()
    ld = log_decay.double()[:, None, None]
    for s in range(len(cu) - 1):
        lo, hi = int(cu[s]), int(cu[s + 1])
        starts = list(range(lo, hi, CHUNK))
        y, mag = last[s], last_mag[s]
        for k0 in reversed(starts) if back else starts:
            rows = slice(k0, min(hi, k0 + CHUNK))
            ah, bh, ch = (x[rows].transpose(0, 1) for x in (a, b, c))
            m = rows.stop - k0
            i = torch.arange(m, device=a.device, dtype=torch.float64)[:, None]
            dist = i.t() - i if back else i - i.t()
            lam = torch.where(dist >= 0, torch.exp(ld * dist.clamp_min(0)), 0.0) * p_scale
            f = torch.exp(ld * (m - 1 - i if back else i + 1)) * s_scale
            w = torch.exp(ld * (i + 1 if back else m - 1 - i)) * w_scale
            sc = ah @ bh.transpose(1, 2) * lam
            o = sc @ ch + f * (ah @ y)
            t = SLACK * ((ah.abs() @ bh.abs().transpose(1, 2) * lam.abs()) @ ch.abs() + f.abs() * (ah.abs() @ mag))
            t = t + HALF * (sc.abs() @ ch.abs() + f.abs() * (ah.abs() @ y.abs()))
            out[rows], tol[rows] = o.transpose(0, 1), (t + HALF * (o.abs() + t)).transpose(0, 1)
            y = torch.exp(ld * m) * y + (bh * w).transpose(1, 2) @ ch
            mag = torch.exp(ld * m) * mag + (bh * w).abs().transpose(1, 2) @ ch.abs()
        last[s], last_mag[s] = y, mag
    return out, tol, last, last_mag


def chunked(q, k, v, ld, cu, scale, s0, g, r1):
    """Forward and gradients as decay_ref.decay_attention, by chunked_walk; for states the sums of magnitudes
    instead of bounds."""
    q, k, v, g, s0, r1 = (x.double() for x in (q, k, v, g, s0, r1))
    t = lambda x: x.transpose(-1, -2)  # noqa: E731
    r = {}
    r["out"], r["out_tol"], r["state_out"], r["state_out_mag"] = chunked_walk(q, k, v, ld, cu, s0, False, 1.0, scale, scale)
    r["dq"], r["dq_tol"], _, _ = chunked_walk(g, v, k, ld, cu, t(s0), False, 1.0, scale, scale)
    r["dk"], r["dk_tol"], _, _ = chunked_walk(v, g, q, ld, cu, t(r1), True, scale, scale, 1.0)
    r["dv"], r["dv_tol"], r["dstate_in"], r["dstate_in_mag"] = chunked_walk(k, q, g, ld, cu, r1, True, scale, scale, 1.0)
    return r


def test_reference_forms_agree():
    """The chunked form against the quadratic one (no GPU)."""
    gen = torch.Generator().manual_seed(0)
    a, b, c = (torch.randn(400, 2, 8, generator=gen, dtype=torch.float64) for _ in range(3))
    first, ld, cu = torch.randn(3, 2, 8, 8, generator=gen, dtype=torch.float64), torch.tensor([-0.01, -0.7]), cu_of([300, 0, 100])
    for args in ((False, 1.0, 0.3, 0.3), (True, 0.3, 0.3, 1.0)):         # as the forward's and the gradients' walks
        x, y = walk(a, b, c, ld, cu, first, *args), chunked_walk(a, b, c, ld, cu, first, *args)
        for got, want in zip(y[:3], x[:3]):
            assert torch.allclose(got, want, rtol=1e-10, atol=1e-13)
        assert torch.allclose(y[3] * 2.0 ** -14, x[3], rtol=1e-10)


def slow(heads):
    """Memories of some hundred to some thousand tokens."""
    return torch.log1p(-torch.exp2(-torch.linspace(8.0, 12.0, heads, dtype=torch.float64))).float().cuda()


# lengths, heads, d; what they are here for.  `parts`: the least tokens of a part, `borders`: the least borders of
# the longest sequence, as far as the workspace's size tells (which holds a state for each).
CASES = [
    dict(lens=[12011], h=1, d=64, borders=24),           # the scan takes 12 borders at a time
    dict(lens=[12011], h=1, d=128, borders=24),
    dict(lens=[15973], h=64, d=64, parts=1024),          # sums of 512 tokens, several to a part
    dict(lens=[15973], h=64, d=128, parts=1024),
    dict(lens=[8141], h=40, d=128, parts=1024),
    # some 400 walks of several chunks forward and 1200 backwards
    dict(lens=[1411, 300, 1500, 700, 0, 1283, 999, 1024, 385, 1355], h=40, d=128, parts=512),
    dict(lens=[1411, 300, 1500, 700, 0, 1283, 999, 1024, 385, 1355], h=64, d=64, parts=512),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c['lens'])}x{max(c['lens'])}-{c['h']}-{c['d']}")
def test_against_the_chunked_form(ops, case):  # noqa: F811
    lens, h, d = case["lens"], case["h"], case["d"]
    q, k, v, g, s0, r1 = inputs(lens, h, d, True)
    ld, cu = slow(h), cu_of(lens).cuda()
    ws = workspace(ops, q, cu)
    # the most borders that either direction has: the workspace holds one state each forward, two backwards
    states = (ws.numel() - 256) // (h * d * d * 4)
    assert states >= case.get("borders", 0) and sum(lens) // max(1, states // 2) >= case.get("parts", 0)
    got = run(ops, q, k, v, ld, cu, None, s0, g, r1, ws=ws)
    heads = sorted({0, h // 2, h - 1})
    want = chunked(*(x[:, heads] for x in (q, k, v)), ld[heads], cu.cpu(), d ** -0.5, *(x[:, heads] for x in (s0, g, r1)))
    for x in ("out", "dq", "dk", "dv"):
        check(got[x][:, heads], want[x], want[x + "_tol"], x)
    for x in ("state_out", "dstate_in"):
        check(got[x][:, heads], want[x], 2.0 ** -14 * want[x + "_mag"], x)
