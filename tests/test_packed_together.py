"""The operators over packed sequences as a model uses them together: a softmax
branch and a linear branch with decays over the same packed batch, one
workspace for all calls, for training and for generating token by token."""
import pytest
import torch

from decay_ref import decay_attention
from packed_ref import attention, check, cu_of
from test_packed_attn import ops, randn  # noqa: F401  (ops is a fixture)

pytestmark = pytest.mark.gpu


def bf16(shape):
    return torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")


def workspace(ops, total_q, total_k, n_seq, hq, hk, d):  # noqa: F811
    return ops.new_workspace_bytes(max(ops.vsa_packed_attn_workspace_bytes(total_q, total_k, n_seq, hq, hk, d),
                                       ops.vsa_decay_attn_workspace_bytes(total_k, n_seq, hk, d)))


@pytest.mark.parametrize("d", [64, 128])
def test_training_step_of_both_branches(ops, d):  # noqa: F811
    """Slices of one projection feed both branches (the linear one takes the kv heads' queries); eager, and captured
    with the calls of both branches interleaved on one workspace: the same bits."""
    lens, hq, hk = [150, 0, 333, 7], 4, 2
    n = sum(lens)
    x, g, gl = randn(1, n, hq + 2 * hk, d), randn(2, n, hq, d), randn(3, n, hk, d)
    q, k, v, ql = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], x[:, :hk]
    ld, cu = torch.tensor([-0.01, -0.2]).cuda(), cu_of(lens).cuda()
    ws = workspace(ops, n, n, len(lens), hq, hk, d)
    soft = dict(out=bf16(q.shape), dq=bf16(q.shape), dk=bf16(k.shape), dv=bf16(k.shape))
    lin = dict(out=bf16(ql.shape), dq=bf16(ql.shape), dk=bf16(ql.shape), dv=bf16(ql.shape))
    out32, lse = torch.empty(n, hq, d, device="cuda"), torch.empty(hq, n, device="cuda")

    def step():
        ops.vsa_packed_attn_fwd(q, k, v, cu, cu, soft["out"], ws, out_f32=out32, lse=lse)
        ops.vsa_decay_attn_fwd(ql, k, v, ld, cu, lin["out"], ws)
        ops.vsa_decay_attn_bwd(ql, k, v, gl, ld, cu, lin["dq"], lin["dk"], lin["dv"], ws)
        ops.vsa_packed_attn_bwd(q, k, v, out32, g, cu, cu, lse, soft["dq"], soft["dk"], soft["dv"], ws)

    step()
    assert ops.vsa_device_status(ws) == 0
    rs = attention(q.cpu(), k.cpu(), v.cpu(), cu.cpu(), cu.cpu(), True, g.cpu())
    rl = decay_attention(ql.cpu(), k.cpu(), v.cpu(), ld.cpu(), cu.cpu(), d ** -0.5, None, gl.cpu())
    for got, r in ((soft, rs), (lin, rl)):
        for name in got:
            check(got[name], r[name], r[name + "_tol"], name)
    want = [t.clone() for r in (soft, lin) for t in r.values()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for _ in range(3):
        for r in (soft, lin):
            for t in r.values():
                t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([t for r in (soft, lin) for t in r.values()], want))
    assert ops.vsa_device_status(ws) == 0


def test_generation_with_a_cache_and_a_state(ops):  # noqa: F811
    """Prompts, then a piece of several tokens, then single tokens: the softmax branch reads a cache of keys and values
    that grows in place (a slice of a larger buffer, sequence after sequence), the linear branch carries its state."""
    hq, hk, d, prompt, piece, singles = 6, 2, 64, [200, 1, 77], 5, 3
    n_seq, room = len(prompt), 300
    whole = [p + piece + singles for p in prompt]
    x = randn(1, sum(whole), hq + 2 * hk, d)
    start = [sum(whole[:i]) for i in range(n_seq)]
    ld = torch.tensor([-0.02, -0.5]).cuda()
    cache_k, cache_v = bf16((n_seq, room, hk, d)), bf16((n_seq, room, hk, d))
    state = torch.zeros(n_seq, hk, d, d, device="cuda")
    ws = workspace(ops, sum(whole), sum(whole), n_seq, hq, hk, d)
    outs = []
    done = [0] * n_seq
    for count in [prompt, [piece] * n_seq] + [[1] * n_seq] * singles:
        rows = torch.cat([torch.arange(s + a, s + a + c) for s, a, c in zip(start, done, count)]).cuda()
        q, k, v = x[rows, :hq], x[rows, hq:hq + hk].contiguous(), x[rows, hq + hk:].contiguous()
        at = 0
        for i, c in enumerate(count):
            cache_k[i, done[i]:done[i] + c], cache_v[i, done[i]:done[i] + c] = k[at:at + c], v[at:at + c]
            at += c
        done = [a + c for a, c in zip(done, count)]
        keys = torch.cat([cache_k[i, :done[i]] for i in range(n_seq)])
        values = torch.cat([cache_v[i, :done[i]] for i in range(n_seq)])
        cu_q, cu_k = cu_of(count).cuda(), cu_of(done).cuda()
        soft, lin, new = bf16(q.shape), bf16(k.shape), torch.empty_like(state)
        ops.vsa_packed_attn_fwd(q, keys, values, cu_q, cu_k, soft, ws)
        if max(count) > 1:
            ops.vsa_decay_attn_fwd(q[:, :hk], k, v, ld, cu_q, lin, ws, state_in=state, state_out=new)
            state = new
        else:
            ops.vsa_decay_attn_step(q[:, :hk], k, v, ld, state, lin)
        assert ops.vsa_device_status(ws) == 0
        outs.append((rows.cpu(), soft, lin))
    cu = cu_of(whole)
    q, k, v = x[:, :hq].cpu(), x[:, hq:hq + hk].cpu(), x[:, hq + hk:].cpu()
    rs = attention(q, k, v, cu, cu, True)
    rl = decay_attention(q[:, :hk], k, v, ld.cpu(), cu, d ** -0.5)
    for rows, soft, lin in outs:
        check(soft, rs["out"][rows], rs["out_tol"][rows], "softmax branch")
        # pieces are chunked otherwise than the whole: both roundings (scores, state) at most, so twice the bound
        check(lin, rl["out"][rows], 2 * rl["out_tol"][rows], "linear branch")
    check(state, rl["state_out"], 2 * rl["state_out_tol"], "state")


def test_long_strides(ops):  # noqa: F811
    """Row offsets past 2^32 bytes in every tensor of both branches: all of them are slices of one buffer whose rows lie
    2 MB apart; the same bits as from dense copies."""
    n, d, lens = 2400, 64, [100, 2200, 100]
    big = torch.empty(n, 1 << 20, dtype=torch.bfloat16, device="cuda")           # 5 GB
    at = iter(range(0, 1 << 14, 128))

    def part(heads, seed=None):
        c = next(at) * 8
        x = big[:, c:c + heads * d].unflatten(1, (heads, d))
        x.copy_(randn(seed, n, heads, d)) if seed else x.fill_(7)
        return x

    q, k, v, g, ql, gl = part(2, 1), part(1, 2), part(1, 3), part(2, 4), part(1, 5), part(1, 6)
    ld, cu = torch.tensor([-0.03]).cuda(), cu_of(lens).cuda()
    ws = workspace(ops, n, n, len(lens), 2, 1, d)
    out32, lse = torch.empty(n, 2, d, device="cuda"), torch.empty(2, n, device="cuda")

    def run(q, k, v, g, ql, gl, new):
        r = [new(2), new(2), new(1), new(1), new(1), new(1), new(1), new(1)]
        ops.vsa_packed_attn_fwd(q, k, v, cu, cu, r[0], ws, out_f32=out32, lse=lse)
        ops.vsa_packed_attn_bwd(q, k, v, out32, g, cu, cu, lse, *r[1:4], ws)
        ops.vsa_decay_attn_fwd(ql, k, v, ld, cu, r[4], ws)
        ops.vsa_decay_attn_bwd(ql, k, v, gl, ld, cu, *r[5:], ws)
        assert ops.vsa_device_status(ws) == 0
        return r

    far = run(q, k, v, g, ql, gl, part)
    near = run(*[x.contiguous() for x in (q, k, v, g, ql, gl)], lambda h: bf16((n, h, d)))
    assert all(torch.equal(a, b) for a, b in zip(far, near))
    step = part(1), part(1)
    state = torch.randn(n, 1, d, d, device="cuda")
    a, b = state.clone(), state.clone()
    ops.vsa_decay_attn_step(ql, k, v, ld, a, step[0])
    dense = bf16((n, 1, d))
    ops.vsa_decay_attn_step(ql.contiguous(), k.contiguous(), v.contiguous(), ld, b, dense)
    assert torch.equal(step[0], dense) and torch.equal(a, b)


def many_borders():
    lens = torch.tensor([0, 0, 1, 2, 3, 5])[torch.randint(6, (1100,), generator=torch.Generator().manual_seed(3))]
    lens[::97] = 131
    return cu_of(lens.tolist(), first=4)


def test_many_short_sequences(ops):  # noqa: F811
    """More sequences than two steps of the search for a tile cover, with runs of empty ones, and rows of none."""
    cu = many_borders().cuda()
    n, d = int(cu[-1]) + 3, 64
    q, g, k, v = randn(1, n, 2, d), randn(2, n, 2, d), randn(3, n, 1, d), randn(4, n, 1, d)
    ws = workspace(ops, n, n, 1100, 2, 1, d)
    ld = torch.tensor([-0.1]).cuda()
    soft = dict(out=bf16(q.shape), dq=bf16(q.shape), dk=bf16(k.shape), dv=bf16(k.shape))
    lin = dict(out=bf16(k.shape), dq=bf16(k.shape), dk=bf16(k.shape), dv=bf16(k.shape))
    out32, lse = torch.empty(n, 2, d, device="cuda"), torch.empty(2, n, device="cuda")
    ops.vsa_packed_attn_fwd(q, k, v, cu, cu, soft["out"], ws, out_f32=out32, lse=lse)
    ops.vsa_packed_attn_bwd(q, k, v, out32, g, cu, cu, lse, soft["dq"], soft["dk"], soft["dv"], ws)
    ops.vsa_decay_attn_fwd(q[:, :1], k, v, ld, cu, lin["out"], ws)
    ops.vsa_decay_attn_bwd(q[:, :1], k, v, g[:, :1], ld, cu, lin["dq"], lin["dk"], lin["dv"], ws)
    assert ops.vsa_device_status(ws) == 0
    rs = attention(q.cpu(), k.cpu(), v.cpu(), cu.cpu(), cu.cpu(), True, g.cpu())
    rl = decay_attention(q[:, :1].cpu(), k.cpu(), v.cpu(), ld.cpu(), cu.cpu(), d ** -0.5, None, g[:, :1].cpu())
    for got, r in ((soft, rs), (lin, rl)):
        for name in got:
            check(got[name], r[name], r[name + "_tol"], name)
            assert (got[name].cpu()[torch.isnan(r[name])] == 7).all(), name


def test_bad_borders_among_many_are_reported(ops):  # noqa: F811
    good = many_borders()
    n, d = int(good[-1]) + 3, 64
    q, k, v = randn(1, n, 2, d), randn(3, n, 1, d), randn(4, n, 1, d)
    ws = workspace(ops, n, n, 1100, 2, 1, d)
    ld, out32, lse = torch.tensor([-0.1]).cuda(), torch.zeros(n, 2, d, device="cuda"), torch.zeros(2, n, device="cuda")
    o, b = torch.empty_like(q), [torch.empty_like(t) for t in (q, k, v)]
    good_d = good.cuda()
    for at, x in ((1, 2 ** 31 - 1), (778, -2 ** 31), (778, int(good[778]) + 200), (1100, n + 1)):
        bad = good.clone()
        bad[at] = x
        bad_d = bad.cuda()
        for cq, ck in ((bad_d, good_d), (good_d, bad_d)):
            ops.vsa_packed_attn_fwd(q, k, v, cq, ck, o, ws)
            assert ops.vsa_device_status(ws) == 6              # VSA_ERR_DEVICE_CHECK
            ops.vsa_packed_attn_bwd(q, k, v, out32, q, cq, ck, lse, *b, ws)
            assert ops.vsa_device_status(ws) == 6
        ops.vsa_decay_attn_fwd(q[:, :1], k, v, ld, bad_d, o[:, :1], ws)
        assert ops.vsa_device_status(ws) == 6
        ops.vsa_decay_attn_bwd(q[:, :1], k, v, q[:, 1:], ld, bad_d, *[t[:, :1] for t in b], ws)
        assert ops.vsa_device_status(ws) == 6
    ops.vsa_packed_attn_fwd(q, k, v, good_d, good_d, o, ws)
    assert ops.vsa_device_status(ws) == 0


def test_calls_at_once_on_two_streams(ops):  # noqa: F811
    """Both branches' steps side by side on two streams, a workspace each (kernels of both share SMs): the same bits
    as one after the other."""
    lens, hq, hk, d = [300, 1, 0, 700, 64], 8, 2, 64
    n = sum(lens)
    q, k, v, g = randn(1, n, hq, d), randn(2, n, hk, d), randn(3, n, hk, d), randn(4, n, hq, d)
    cu, ones = cu_of(lens).cuda(), cu_of([1] * len(lens)).cuda()
    ld = torch.linspace(-0.3, -0.001, hq).cuda()
    kq, vq = randn(5, n, hq, d), randn(6, n, hq, d)

    def buffers():
        f32 = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        return dict(ws=workspace(ops, n, n, len(lens), hq, hq, d), out=bf16(q.shape), o32=f32(n, hq, d), lse=f32(hq, n),
                    dq=bf16(q.shape), dk=bf16(k.shape), dv=bf16(k.shape), tok=bf16((len(lens), hq, d)), lin=bf16(q.shape),
                    ldq=bf16(q.shape), ldk=bf16(q.shape), ldv=bf16(q.shape), state=f32(len(lens), hq, d, d))

    def soft(b, s):
        ops.vsa_packed_attn_fwd(q, k, v, cu, cu, b["out"], b["ws"], out_f32=b["o32"], lse=b["lse"], stream=s)
        ops.vsa_packed_attn_bwd(q, k, v, b["o32"], g, cu, cu, b["lse"], b["dq"], b["dk"], b["dv"], b["ws"], stream=s)
        ops.vsa_packed_attn_fwd(q[:len(lens)], k, v, ones, cu, b["tok"], b["ws"], stream=s)

    def linear(b, s):
        ops.vsa_decay_attn_fwd(q, kq, vq, ld, cu, b["lin"], b["ws"], state_out=b["state"], stream=s)
        ops.vsa_decay_attn_bwd(q, kq, vq, g, ld, cu, b["ldq"], b["ldk"], b["ldv"], b["ws"], stream=s)

    want, x, y = buffers(), buffers(), buffers()
    soft(want, None)
    linear(want, None)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        soft(x, s)
        linear(y, t)
        linear(x, s)
        soft(y, t)
    torch.cuda.synchronize()
    for b in (x, y):
        assert ops.vsa_device_status(b["ws"]) == 0
        for name in want:
            assert name == "ws" or torch.equal(b[name], want[name]), name
