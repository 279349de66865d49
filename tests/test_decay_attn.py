"""Linear attention with a decay per head over packed sequences: forward,
gradients and the recurrent step, against the plain fp64 implementation,
element by element with derived bounds."""
import math

import pytest
import torch

from decay_ref import decay_attention, recurrence
from packed_ref import HALF, check, cu_of
from test_packed_attn import ops, randn  # noqa: F401  (ops is a fixture)

gpu = pytest.mark.gpu


def decays(heads):
    """From a memory of a few tokens to one of thousands."""
    e = torch.linspace(1.0, 12.0, heads, dtype=torch.float64) if heads > 1 else torch.tensor([6.0], dtype=torch.float64)
    return torch.log1p(-torch.exp2(-e)).float().cuda()


def states(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda() * 4


def workspace(ops, q, cu):  # noqa: F811
    n = ops.vsa_decay_attn_workspace_bytes(q.shape[0], cu.numel() - 1, q.shape[1], q.shape[2])
    assert n > 0
    return ops.new_workspace_bytes(n)


def run(ops, q, k, v, ld, cu, scale=None, s0=None, g=None, r1=None, ws=None, stream=None, want_states=True):  # noqa: F811
    """Forward and, with g, gradients; every output filled with a sentinel before."""
    ws = workspace(ops, q, cu) if ws is None else ws
    n, (h, d) = cu.numel() - 1, q.shape[1:]
    full = lambda shape, t: torch.full(shape, 7.0, dtype=t, device="cuda")  # noqa: E731
    r = dict(out=full(q.shape, torch.bfloat16))
    if want_states:
        r["state_out"] = full((n, h, d, d), torch.float32)
    ops.vsa_decay_attn_fwd(q, k, v, ld, cu, r["out"], ws, scale=scale, state_in=s0, state_out=r.get("state_out"), stream=stream)
    if g is not None:
        for x in ("dq", "dk", "dv"):
            r[x] = full(q.shape, torch.bfloat16)
        if want_states:
            r["dstate_in"] = full((n, h, d, d), torch.float32)
        ops.vsa_decay_attn_bwd(q, k, v, g, ld, cu, r["dq"], r["dk"], r["dv"], ws, scale=scale, state_in=s0, dstate_out=r1,
                               dstate_in=r.get("dstate_in"), stream=stream)
    assert ops.vsa_device_status(ws, stream) == 0
    return r


def compare(got, want):
    for x in got:
        check(got[x], want[x], want[x + "_tol"], x)
        assert (got[x].cpu()[torch.isnan(want[x])] == 7).all(), x       # rows of no sequence keep what was there


def inputs(lens, h, d, with_state, extra=0):
    n = sum(lens) + extra
    q, k, v, g = (randn(s, n, h, d) for s in (1, 2, 3, 4))
    s0 = states(5, len(lens), h, d, d) if with_state else None
    r1 = states(6, len(lens), h, d, d) if with_state else None
    return q, k, v, g, s0, r1


def cpu(*x):
    return [None if t is None else t.cpu() for t in x]


CASES = [
    # lengths, heads, d, states
    ([1], 1, 64, True),
    ([1], 3, 128, False),
    ([127, 128, 129], 2, 128, True),
    ([255, 1, 0, 257, 256], 3, 64, True),
    ([0, 0, 5], 2, 64, True),
    ([5, 0], 2, 128, False),
    ([1000], 1, 128, True),                      # several segments
    ([900, 3, 1100], 2, 64, True),
    ([640, 0, 770, 128], 2, 128, False),
    ([2] * 150, 1, 64, True),
]


def test_reference_forms_agree():
    """The quadratic form of the reference against the definition, token by token (no GPU)."""
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(9, 2, 4, generator=g, dtype=torch.float64) for _ in range(3))
    s0 = torch.randn(3, 2, 4, 4, generator=g, dtype=torch.float64)
    ld = torch.tensor([-0.3, -2.0])
    cu = cu_of([5, 0, 4])
    r = decay_attention(q, k, v, ld, cu, 0.5, s0)
    out, last = recurrence(q, k, v, ld, cu, 0.5, s0)
    assert torch.allclose(r["out"], out, rtol=1e-12) and torch.allclose(r["state_out"], last, rtol=1e-12)


def test_reference_gradients_against_differences():
    """The reference's gradients against central differences of its forward (no GPU): the loss is linear in q, in v and
    in the state and quadratic at most in k together with the others, so the differences are exact up to rounding."""
    gen = torch.Generator().manual_seed(0)
    q, k, v, g = (torch.randn(7, 1, 3, generator=gen, dtype=torch.float64) for _ in range(4))
    s0, r1 = (torch.randn(2, 1, 3, 3, generator=gen, dtype=torch.float64) for _ in range(2))
    ld, cu = torch.tensor([-0.2]), cu_of([3, 4])
    r = decay_attention(q, k, v, ld, cu, 0.7, s0, g, r1)

    def loss(q, k, v, s0):
        f = decay_attention(q, k, v, ld, cu, 0.7, s0)
        return ((f["out"] * g).sum() + (f["state_out"] * r1).sum()).item()

    x = [q, k, v, s0]
    for i, n in enumerate(("dq", "dk", "dv", "dstate_in")):
        u = torch.randn(x[i].shape, generator=gen, dtype=torch.float64)
        lo, hi = list(x), list(x)
        lo[i], hi[i] = x[i] - u, x[i] + u
        assert math.isclose((loss(*hi) - loss(*lo)) / 2, (r[n] * u).sum().item(), rel_tol=1e-10, abs_tol=1e-10)


@gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0][:4])}-{c[1]}-{c[2]}-{c[3]}".replace(" ", ""))
def test_forward_and_gradients(ops, case):  # noqa: F811
    lens, h, d, with_state = case
    q, k, v, g, s0, r1 = inputs(lens, h, d, with_state)
    ld, cu = decays(h), cu_of(lens).cuda()
    got = run(ops, q, k, v, ld, cu, None, s0, g, r1)
    compare(got, decay_attention(*cpu(q, k, v, ld, cu), d ** -0.5, *cpu(s0, g, r1)))


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_without_state_outputs(ops, d):  # noqa: F811
    """The last chunk's update is left out; nothing else changes."""
    q, k, v, g, s0, r1 = inputs([300, 128], 2, d, True)
    ld, cu = decays(2), cu_of([300, 128]).cuda()
    full, less = run(ops, q, k, v, ld, cu, 0.3, s0, g, r1), run(ops, q, k, v, ld, cu, 0.3, s0, g, r1, want_states=False)
    assert all(torch.equal(full[x], less[x]) for x in less)
    compare(full, decay_attention(*cpu(q, k, v, ld, cu), 0.3, *cpu(s0, g, r1)))


@gpu
def test_extreme_decays(ops):  # noqa: F811
    """No memory at all (-inf), a memory that dies within a chunk, and no decay."""
    q, k, v, g, s0, r1 = inputs([300, 5], 4, 64, True)
    ld, cu = torch.tensor([-math.inf, -3.0, -0.05, 0.0]).cuda(), cu_of([300, 5]).cuda()
    compare(run(ops, q, k, v, ld, cu, None, s0, g, r1), decay_attention(*cpu(q, k, v, ld, cu), 0.125, *cpu(s0, g, r1)))


@gpu
def test_fused_projection_and_rows_of_no_sequence(ops):  # noqa: F811
    lens, h, d = [130, 0, 57], 3, 128
    n = 20 + sum(lens) + 9
    x, g = randn(4, n, 3 * h, d), randn(5, n, h, d)
    x[:20], x[20 + sum(lens):], g[:20], g[20 + sum(lens):] = math.nan, math.inf, math.inf, math.nan
    ld, cu = decays(h), cu_of(lens, first=20).cuda()
    q, k, v = x[:, :h], x[:, h:2 * h], x[:, 2 * h:]
    s0, r1 = states(5, 3, h, d, d), states(6, 3, h, d, d)
    got = run(ops, q, k, v, ld, cu, None, s0, g, r1)
    compare(got, decay_attention(*cpu(q, k, v, ld, cu), d ** -0.5, *cpu(s0, g, r1)))
    dx = torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ops.vsa_decay_attn_bwd(q, k, v, g, ld, cu, dx[:, :h], dx[:, h:2 * h], dx[:, 2 * h:], workspace(ops, q, cu), state_in=s0,
                           dstate_out=r1)
    assert torch.equal(dx, torch.cat([got["dq"], got["dk"], got["dv"]], 1))


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_other_sequences_do_not_matter(ops, d):  # noqa: F811
    lens = [70, 700, 66]
    q, k, v, g, s0, r1 = inputs(lens, 2, d, True)
    ld, cu = decays(2), cu_of(lens).cuda()
    want = run(ops, q, k, v, ld, cu, None, s0, g, r1)
    for x in (q, k, v, g):
        x[:70], x[-66:] = math.nan, math.inf
    for x in (s0, r1):
        x[0], x[2] = math.inf, math.nan
    got = run(ops, q, k, v, ld, cu, None, s0, g, r1)
    for n in got:
        rows = 1 if "state" in n else slice(70, 770)
        assert torch.equal(got[n][rows], want[n][rows]), n


@gpu
def test_a_prompt_in_pieces_and_tokens_one_by_one(ops):  # noqa: F811
    """As they are used together: a prompt's first part, its continuation with the state carried over, then single
    tokens by the recurrent step, against the whole sequences in fp64."""
    h, d, lens, more = 3, 64, [200, 77], 4
    ld = decays(h)
    whole = [n + more for n in lens]
    q, k, v = (randn(s, sum(whole), h, d) for s in (1, 2, 3))
    start = [0, whole[0]]
    take = lambda x, a, b: torch.cat([x[s + lo:s + hi] for s, lo, hi in zip(start, a, b)])  # noqa: E731
    state = torch.zeros(2, h, d, d, device="cuda")
    outs = []
    for a, b in (([0, 0], [130, 50]), ([130, 50], lens)):
        cu = cu_of([y - x for x, y in zip(a, b)]).cuda()
        r = run(ops, take(q, a, b), take(k, a, b), take(v, a, b), ld, cu, None, state)
        state = r["state_out"]
        outs.append((a, b, r["out"]))
    for t in range(more):
        a, b = [n + t for n in lens], [n + t + 1 for n in lens]
        out = torch.full((2, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
        ops.vsa_decay_attn_step(take(q, a, b), take(k, a, b), take(v, a, b), ld, state, out)
        outs.append((a, b, out))
    want, last = recurrence(*cpu(q, k, v, ld, cu_of(whole)), d ** -0.5, torch.zeros(2, h, d, d))
    r = decay_attention(*cpu(q, k, v, ld, cu_of(whole)), d ** -0.5)
    for a, b, out in outs:
        # a piece may be chunked otherwise than the whole: both roundings (scores, state) at most, so twice the bound
        check(out, take(want, a, b), 2 * take(r["out_tol"], a, b))
    check(state, last, 2 * r["state_out_tol"])


@gpu
@pytest.mark.parametrize("case", [(1, 1, 64), (1, 12, 128), (3, 5, 64), (67, 3, 128)])
def test_step(ops, case):  # noqa: F811
    n, h, d = case
    x = randn(1, n, 3 * h, d)
    q, k, v = x[:, :h], x[:, h:2 * h], x[:, 2 * h:]      # strided rows
    state, ld = states(2, n, h, d, d), decays(h)
    new, out = torch.full_like(state, 7.0), torch.full((n, 2 * h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    before = state.clone()
    ops.vsa_decay_attn_step(q, k, v, ld, state, out[:, :h], scale=0.2, state_out=new)
    assert torch.equal(state, before) and (out[:, h:] == 7).all()
    want, last = recurrence(*cpu(q, k, v, ld, torch.arange(n + 1)), 0.2, before.cpu())
    mags = ((before.double() * torch.exp(ld.double())[:, None, None]).abs() + (k.double()[..., None] * v.double()[..., None, :]).abs()).cpu()
    check(new, last, 2.0 ** -21 * mags)                  # a 2-ulp exponential, a product and an fma
    t = 0.2 * 2.0 ** -16 * (q.double().abs()[..., None, :].cpu() @ mags)[..., 0, :]      # d + 8 fp32 steps: 136 * 2^-24
    check(out[:, :h], want, t + HALF * (want.abs() + t))
    again = out.clone()
    ops.vsa_decay_attn_step(q, k, v, ld, state, again[:, :h], scale=0.2)                 # in place
    assert torch.equal(state, new) and torch.equal(again, out)


@gpu
def test_step_without_memory_and_without_sequences(ops):  # noqa: F811
    q, k, v = (randn(s, 2, 1, 64) for s in (1, 2, 3))
    state, out = states(2, 2, 1, 64, 64), torch.zeros_like(q)
    ops.vsa_decay_attn_step(q, k, v, torch.tensor([-math.inf]).cuda(), state, out)
    assert torch.equal(state, k.float()[..., None] * v.float()[..., None, :])
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    ops.vsa_decay_attn_step(e, e, e, decays(1), torch.empty(0, 1, 64, 64, device="cuda"), e)


@gpu
def test_without_tokens(ops):  # noqa: F811
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    s0, r1 = states(1, 3, 2, 64, 64), states(2, 3, 2, 64, 64)
    cu = cu_of([0, 0, 0]).cuda()
    got = run(ops, e, e, e, decays(2), cu, None, s0, e, r1)
    assert torch.equal(got["state_out"], s0) and torch.equal(got["dstate_in"], r1)
    got = run(ops, e, e, e, decays(2), cu, None, None, e, None)
    assert (got["state_out"] == 0).all() and (got["dstate_in"] == 0).all()


@gpu
def test_bad_borders_are_reported(ops):  # noqa: F811
    q, k, v, g, s0, r1 = inputs([20, 600, 20], 2, 64, True)
    ld, good = decays(2), cu_of([20, 600, 20]).cuda()
    want = run(ops, q, k, v, ld, good, None, s0, g, r1)
    for bad in ([0, 20, 15, 640], [0, 20, 40, 641], [-1, 20, 40, 640], [0, 20, 2 ** 31 - 1, 640]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        ws = workspace(ops, q, cu)
        d = [torch.zeros_like(q) for _ in range(4)]
        ops.vsa_decay_attn_fwd(q, k, v, ld, cu, d[0], ws, state_in=s0)
        assert ops.vsa_device_status(ws) == 6                  # VSA_ERR_DEVICE_CHECK
        ops.vsa_decay_attn_bwd(q, k, v, g, ld, cu, *d[1:], ws, state_in=s0, dstate_out=r1)
        assert ops.vsa_device_status(ws) == 6
        got = run(ops, q, k, v, ld, good, None, s0, g, r1, ws=ws)
        assert all(torch.equal(got[x], want[x]) for x in got)


@gpu
def test_captured_with_changing_borders_and_repeatable(ops):  # noqa: F811
    q, k, v, g, s0, r1 = inputs([500, 268, 0], 2, 128, True)
    ld, cu = decays(2), cu_of([500, 268, 0]).cuda()
    ws = workspace(ops, q, cu)
    out, d = torch.zeros_like(q), [torch.zeros_like(q) for _ in range(3)]
    s1, r0 = torch.zeros_like(s0), torch.zeros_like(s0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ops.vsa_decay_attn_fwd(q, k, v, ld, cu, out, ws, state_in=s0, state_out=s1)
        ops.vsa_decay_attn_bwd(q, k, v, g, ld, cu, *d, ws, state_in=s0, dstate_out=r1, dstate_in=r0)
    for lens in ([500, 268, 0], [1, 750, 17], [0, 0, 768]):
        cu.copy_(cu_of(lens))
        q.copy_(randn(lens[0], 768, 2, 128))
        graph.replay()
        torch.cuda.synchronize()
        want = run(ops, q, k, v, ld, cu, None, s0, g, r1)
        for x, n in zip((out, s1, *d, r0), ("out", "state_out", "dq", "dk", "dv", "dstate_in")):
            assert torch.equal(x, want[n]), (lens, n)
    assert ops.vsa_device_status(ws) == 0


@gpu
def test_on_another_stream(ops):  # noqa: F811
    q, k, v, g, s0, r1 = inputs([900], 2, 64, True)
    ld, cu = decays(2), cu_of([900]).cuda()
    want = run(ops, q, k, v, ld, cu, None, s0, g, r1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(ops, q, k, v, ld, cu, None, s0, g, r1, stream=s)
    s.synchronize()
    assert all(torch.equal(got[x], want[x]) for x in got)
