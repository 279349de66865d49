"""Gradients of the softmax attention over packed sequences, against the plain
fp64 implementation (element by element with derived bounds) and against
differences of its forward."""
import math

import pytest
import torch

from packed_ref import attention, check, cu_of
from test_packed_attn import CASES, forward, ops, randn, workspace  # noqa: F401  (ops is a fixture)

pytestmark = pytest.mark.gpu


def grads(ops, q, k, v, g, cu_q, cu_k, causal, ws=None, stream=None, fwd=None):  # noqa: F811
    ws = workspace(ops, q, k, cu_q) if ws is None else ws
    _, out32, lse = fwd or forward(ops, q, k, v, cu_q, cu_k, causal)
    d = [torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in (q, k, v)]
    ops.vsa_packed_attn_bwd(q, k, v, out32, g, cu_q, cu_k, lse, *d, ws, causal=causal, stream=stream)
    assert ops.vsa_device_status(ws, stream) == 0
    return d


def check_grads(ops, q, k, v, g, cu_q, cu_k, causal):  # noqa: F811
    got = grads(ops, q, k, v, g, cu_q, cu_k, causal)
    r = attention(q.cpu(), k.cpu(), v.cpu(), cu_q.cpu(), cu_k.cpu(), causal, g.cpu())
    for x, n in zip(got, ("dq", "dk", "dv")):
        check(x, r[n], r[n + "_tol"], n)
        assert (x.cpu()[torch.isnan(r[n])] == 7).all(), n       # rows of no sequence keep what was there
    return got, r


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0][:4])}-{c[2]}x{c[3]}-{c[4]}-{c[5]}".replace(" ", ""))
def test_gradients(ops, case):  # noqa: F811
    lens_q, lens_k, hq, hk, d, causal = case
    lens_k = lens_q if lens_k is None else lens_k
    q, g = randn(1, sum(lens_q), hq, d), randn(4, sum(lens_q), hq, d)
    k, v = randn(2, sum(lens_k), hk, d), randn(3, sum(lens_k), hk, d)
    check_grads(ops, q, k, v, g, cu_of(lens_q).cuda(), cu_of(lens_k).cuda(), causal)


def test_gradients_against_differences(ops):  # noqa: F811
    """The derivative of sum(dout * out) along a direction, by central differences of the fp64 forward, whose own error
    (third derivatives times h^2 / 6, h = 2^-10) is far below the elementwise bounds summed over the direction."""
    lens_q, lens_k = [70, 3, 130], [100, 50, 130]
    q, g = randn(1, 203, 4, 64), randn(4, 203, 4, 64)
    k, v = randn(2, 280, 2, 64), randn(3, 280, 2, 64)
    cq, ck = cu_of(lens_q), cu_of(lens_k)
    got, r = check_grads(ops, q, k, v, g, cq.cuda(), ck.cuda(), True)
    x = [t.cpu().double() for t in (q, k, v)]
    h = 2.0 ** -10
    for i, n in enumerate(("dq", "dk", "dv")):
        u = torch.randn(x[i].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(9 + i))
        f = []
        for s in (h, -h):
            y = list(x)
            y[i] = x[i] + s * u
            f.append((attention(*y, cq, ck, True)["out"] * g.cpu().double()).sum().item())
        want = (f[0] - f[1]) / (2 * h)
        assert abs((got[i].cpu().double() * u).sum().item() - want) <= (r[n + "_tol"] * u.abs()).sum().item()


def test_gradients_fused_projection_and_rows_of_no_sequence(ops):  # noqa: F811
    """q, k, v and dq, dk, dv as slices of one projection and of its gradient; foreign rows hold NaN and Inf."""
    lens, hq, hk, d = [130, 0, 57], 10, 2, 128
    n = 20 + sum(lens) + 9
    x, g = randn(4, n, hq + 2 * hk, d), randn(5, n, hq, d)
    cu = cu_of(lens, first=20).cuda()
    for t in (x, g):
        t[:20], t[20 + sum(lens):] = math.nan, math.inf
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    want, _ = check_grads(ops, q, k, v, g, cu, cu, True)
    dx = torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = workspace(ops, q, k, cu)
    _, out32, lse = forward(ops, q, k, v, cu, cu)
    ops.vsa_packed_attn_bwd(q, k, v, out32, g, cu, cu, lse, dx[:, :hq], dx[:, hq:hq + hk], dx[:, hq + hk:], ws)
    assert torch.equal(dx, torch.cat(want, 1))


@pytest.mark.parametrize("lens_q", [[70, 190, 66], [5, 1, 9]])
def test_gradients_other_sequences_do_not_matter(ops, lens_q):  # noqa: F811
    lens_k = [70, 190, 66]
    q, g = randn(1, sum(lens_q), 6, 128), randn(4, sum(lens_q), 6, 128)
    k, v = randn(2, 326, 2, 128), randn(3, 326, 2, 128)
    cq, ck = cu_of(lens_q).cuda(), cu_of(lens_k).cuda()
    want = grads(ops, q, k, v, g, cq, ck, True)
    for x, n in ((q, lens_q[0]), (g, lens_q[0]), (k, 70), (v, 70)):
        x[:n] = math.nan
    for x, n in ((q, lens_q[2]), (g, lens_q[2]), (k, 66), (v, 66)):
        x[-n:] = math.inf
    got = grads(ops, q, k, v, g, cq, ck, True)
    rq, rk = slice(lens_q[0], lens_q[0] + lens_q[1]), slice(70, 260)
    for a, b, rows in zip(got, want, (rq, rk, rk)):
        assert torch.equal(a[rows], b[rows])


def test_gradients_with_a_common_component_of_the_keys(ops):  # noqa: F811
    """Keys and values that share a component far larger than their differences: dq is a small difference of large
    terms, which the bound follows."""
    q, g = randn(1, 300, 2, 64), randn(4, 300, 2, 64)
    k = (randn(2, 300, 2, 64).float() * 0.25 + 8).to(torch.bfloat16)
    v = (randn(3, 300, 2, 64).float() + 8).to(torch.bfloat16)
    cu = cu_of([300]).cuda()
    check_grads(ops, q, k, v, g, cu, cu, True)


def test_gradients_without_tokens(ops):  # noqa: F811
    e = lambda n, h: torch.empty(n, h, 64, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    none, cu = cu_of([0, 0]).cuda(), cu_of([2, 3]).cuda()
    grads(ops, e(0, 2), e(0, 1), e(0, 1), e(0, 2), none, none, True)
    x = lambda n, h: randn(1, n, h, 64)  # noqa: E731
    dq, _, _ = grads(ops, x(5, 2), e(0, 1), e(0, 1), x(5, 2), cu, none, True)
    assert (dq == 0).all()
    _, dk, dv = grads(ops, e(0, 2), x(5, 1), x(5, 1), e(0, 2), none, cu, True)
    assert (dk == 0).all() and (dv == 0).all()


def test_gradients_bad_borders_are_reported(ops):  # noqa: F811
    q, g = randn(1, 60, 2, 64), randn(4, 60, 2, 64)
    k, v = randn(2, 60, 1, 64), randn(3, 60, 1, 64)
    good = cu_of([20, 20, 20]).cuda()
    fwd = forward(ops, q, k, v, good, good)
    want = grads(ops, q, k, v, g, good, good, True, fwd=fwd)
    for bad in ([0, 20, 15, 60], [0, 20, 40, 61], [-1, 20, 40, 60], [0, 20, 2 ** 31 - 1, 60]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        ws = workspace(ops, q, k, cu)
        d = [torch.empty_like(x) for x in (q, k, v)]
        for a, b in ((cu, good), (good, cu)):
            ops.vsa_packed_attn_bwd(q, k, v, fwd[1], g, a, b, fwd[2], *d, ws)
            assert ops.vsa_device_status(ws) == 6              # VSA_ERR_DEVICE_CHECK
        got = grads(ops, q, k, v, g, good, good, True, ws=ws, fwd=fwd)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_training_step_captured(ops):  # noqa: F811
    """Forward and backward in one graph, replayed after the borders and the tensors changed; the same bits each time."""
    q, g = randn(1, 256, 4, 64), randn(4, 256, 4, 64)
    k, v = randn(2, 256, 2, 64), randn(3, 256, 2, 64)
    cu = cu_of([100, 156, 0]).cuda()
    ws = workspace(ops, q, k, cu)
    out, out32 = torch.zeros_like(q), torch.zeros(q.shape, device="cuda")
    lse = torch.zeros(4, 256, device="cuda")
    d = [torch.zeros_like(x) for x in (q, k, v)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ops.vsa_packed_attn_fwd(q, k, v, cu, cu, out, ws, out_f32=out32, lse=lse)
        ops.vsa_packed_attn_bwd(q, k, v, out32, g, cu, cu, lse, *d, ws)
    for lens in ([100, 156, 0], [1, 250, 5], [0, 0, 256]):
        cu.copy_(cu_of(lens))
        q.copy_(randn(sum(lens[:1]), 256, 4, 64))
        for x in d:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(d, grads(ops, q, k, v, g, cu, cu, True)))
    assert ops.vsa_device_status(ws) == 0


def test_gradients_on_another_stream(ops):  # noqa: F811
    q, g = randn(1, 500, 8, 128), randn(4, 500, 8, 128)
    k, v = randn(2, 500, 2, 128), randn(3, 500, 2, 128)
    cu = cu_of([499, 1]).cuda()
    want = grads(ops, q, k, v, g, cu, cu, False)
    fwd = forward(ops, q, k, v, cu, cu, False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = grads(ops, q, k, v, g, cu, cu, False, stream=s, fwd=fwd)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
