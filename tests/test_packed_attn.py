"""Softmax attention over packed sequences with grouped heads, against the
plain fp64 implementation, element by element with derived bounds."""
import math

import pytest
import torch

from packed_ref import attention, check, cu_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_30_b200 import build, ops
    build.build()
    return ops


def randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(torch.bfloat16).cuda()


def workspace(ops, q, k, cu_q):
    n = ops.vsa_packed_attn_workspace_bytes(q.shape[0], k.shape[0], cu_q.numel() - 1, q.shape[1], k.shape[1], q.shape[2])
    assert n > 0
    return ops.new_workspace_bytes(n)


def forward(ops, q, k, v, cu_q, cu_k, causal=True, ws=None):
    """out (bf16), out_f32, lse, every buffer filled with a sentinel before."""
    ws = workspace(ops, q, k, cu_q) if ws is None else ws
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    out32 = torch.full(q.shape, 7.0, dtype=torch.float32, device="cuda")
    lse = torch.full((q.shape[1], q.shape[0]), 7.0, dtype=torch.float32, device="cuda")
    ops.vsa_packed_attn_fwd(q, k, v, cu_q, cu_k, out, ws, causal=causal, out_f32=out32, lse=lse)
    assert ops.vsa_device_status(ws) == 0
    return out, out32, lse


def check_forward(ops, q, k, v, cu_q, cu_k, causal=True):
    out, out32, lse = forward(ops, q, k, v, cu_q, cu_k, causal)
    r = attention(q.cpu(), k.cpu(), v.cpu(), cu_q.cpu(), cu_k.cpu(), causal)
    check(out, r["out"], r["out_tol"], "out")
    check(out32, r["out"], r["out32_tol"], "out32")
    check(lse.t(), r["lse"], r["lse_tol"], "lse")
    alone = torch.isnan(r["out"])                       # rows of no sequence keep what was there
    assert (out.cpu()[alone] == 7).all() and (out32.cpu()[alone] == 7).all()
    return out, out32, lse


CASES = [
    # lens_q, lens_k (None: the same), heads_q, heads_kv, d, causal
    ([1], None, 1, 1, 64, True),
    ([1], None, 4, 1, 128, False),
    ([127, 128, 129], None, 2, 2, 128, True),
    ([255, 1, 0, 257, 256], None, 2, 1, 64, True),
    ([0, 0, 5], None, 3, 3, 64, True),
    ([300, 77], None, 10, 2, 128, True),                # group 5: 125 of 128 rows of a tile
    ([130, 64], None, 21, 3, 64, True),                 # group 7: 126 rows
    ([9, 3], None, 128, 1, 128, True),                  # group 128: one token per tile
    ([5], None, 100, 1, 64, False),                     # group 100
    ([700], None, 2, 2, 128, True),
    ([700], None, 2, 2, 64, False),
    ([40, 1, 200], [300, 129, 200], 4, 2, 128, True),   # continued prompts
    ([200, 5, 130, 1], [50, 0, 129, 0], 4, 2, 64, True),     # queries that see no key
    ([200, 5], [50, 0], 2, 2, 128, False),
    ([1] * 7, [1, 64, 127, 128, 129, 1000, 2500], 8, 2, 128, True),   # single tokens, split key axis
    ([1, 1], [4000, 3], 40, 8, 64, True),
    ([3, 0, 2], [1500, 700, 1], 6, 1, 128, True),       # few tokens, split key axis, 1 key for 2 queries
    ([2] * 150, [3] * 150, 2, 1, 64, True),             # more sequences than one scan step holds
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0][:4])}-{c[2]}x{c[3]}-{c[4]}-{c[5]}".replace(" ", ""))
def test_forward(ops, case):
    lens_q, lens_k, hq, hk, d, causal = case
    lens_k = lens_q if lens_k is None else lens_k
    q = randn(1, sum(lens_q), hq, d)
    k, v = randn(2, sum(lens_k), hk, d), randn(3, sum(lens_k), hk, d)
    check_forward(ops, q, k, v, cu_of(lens_q).cuda(), cu_of(lens_k).cuda(), causal)


def test_forward_large_scores(ops):
    """Scores that grow by hundreds along the keys (the running maximum is raised again and again) and fall."""
    q, k, v = randn(1, 900, 2, 128), randn(2, 900, 2, 128), randn(3, 900, 2, 128)
    ramp = torch.linspace(-8, 8, 900, device="cuda")[:, None, None]
    cu = cu_of([900]).cuda()
    for sign in (1, -1):
        check_forward(ops, (q.abs() * 2).to(torch.bfloat16), (k.abs() * 0.1 + sign * ramp).to(torch.bfloat16), v, cu, cu)


def test_forward_fused_projection_and_rows_of_no_sequence(ops):
    """q, k, v as slices of one projection; rows before the first and behind the last sequence hold NaN and Inf."""
    lens, hq, hk, d = [130, 0, 57], 6, 2, 128
    x = randn(4, 20 + sum(lens) + 9, hq + 2 * hk, d)
    x[:20], x[20 + sum(lens):] = math.nan, math.inf
    cu = cu_of(lens, first=20).cuda()
    check_forward(ops, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], cu, cu)
    check_forward(ops, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], cu, cu, causal=False)


def test_forward_strided_output(ops):
    q, k, v = randn(1, 100, 4, 64), randn(2, 100, 2, 64), randn(3, 100, 2, 64)
    cu = cu_of([60, 40]).cuda()
    want = forward(ops, q, k, v, cu, cu)[0]
    big = torch.full((100, 12, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.vsa_packed_attn_fwd(q, k, v, cu, cu, big[:, 4:8], workspace(ops, q, k, cu))
    assert torch.equal(big[:, 4:8], want)
    assert (big[:, :4] == 7).all() and (big[:, 8:] == 7).all()


@pytest.mark.parametrize("lens_q", [[70, 190, 66], [1, 1, 1]])
def test_forward_other_sequences_do_not_matter(ops, lens_q):
    """NaN and Inf in the sequences around one leave its results bit for bit."""
    lens_k = [70, 190, 66]
    q, k, v = randn(1, sum(lens_q), 4, 128), randn(2, 326, 2, 128), randn(3, 326, 2, 128)
    cq, ck = cu_of(lens_q).cuda(), cu_of(lens_k).cuda()
    want = forward(ops, q, k, v, cq, ck)
    for x, n in ((q, lens_q[0]), (k, 70), (v, 70)):
        x[:n] = math.nan
    for x, n in ((q, lens_q[2]), (k, 66), (v, 66)):
        x[-n:] = math.inf
    got = forward(ops, q, k, v, cq, ck)
    rows = slice(lens_q[0], lens_q[0] + lens_q[1])
    assert torch.equal(got[0][rows], want[0][rows]) and torch.equal(got[1][rows], want[1][rows])
    assert torch.equal(got[2][:, rows], want[2][:, rows])


def test_forward_nan_in_own_sequence_stays_nan(ops):
    q, k, v = randn(1, 64, 1, 64), randn(2, 64, 1, 64), randn(3, 64, 1, 64)
    cu = cu_of([64]).cuda()
    q[5] = math.nan
    out, out32, lse = forward(ops, q, k, v, cu, cu)
    assert torch.isnan(out[5]).all() and torch.isnan(lse[0, 5]) and torch.isfinite(out[torch.arange(64) != 5]).all()


def test_forward_long_strides(ops):
    """Row offsets past 2^32 bytes: a cache whose rows lie 2 MB apart."""
    n, hk, d = 2600, 1, 64
    cache = torch.empty(n, 1 << 20, dtype=torch.bfloat16, device="cuda")     # 5.4 GB
    k, v = cache[:, :64].unflatten(1, (1, 64)), cache[:, 64:128].unflatten(1, (1, 64))
    k.copy_(randn(2, n, hk, d)), v.copy_(randn(3, n, hk, d))
    check_forward(ops, randn(1, 3, 2, d), k, v, cu_of([1, 2]).cuda(), cu_of([100, 2500]).cuda())


def test_forward_without_tokens(ops):
    e = lambda n, h: torch.empty(n, h, 64, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    cu = cu_of([0, 0]).cuda()
    forward(ops, e(0, 2), e(0, 1), e(0, 1), cu, cu)
    out, out32, lse = forward(ops, randn(1, 5, 2, 64), e(0, 1), e(0, 1), cu_of([2, 3]).cuda(), cu)
    assert (out == 0).all() and (out32 == 0).all() and (lse == -math.inf).all()


def test_forward_bad_borders_are_reported(ops):
    q, k, v = randn(1, 60, 2, 64), randn(2, 60, 1, 64), randn(3, 60, 1, 64)
    good = cu_of([20, 20, 20]).cuda()
    want = forward(ops, q, k, v, good, good)[0]
    for bad in ([0, 20, 15, 60], [0, 20, 40, 61], [-1, 20, 40, 60], [0, 20, 2 ** 31 - 1, 60]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        ws = workspace(ops, q, k, cu)
        out = torch.zeros_like(q)
        ops.vsa_packed_attn_fwd(q, k, v, cu, good, out, ws)
        assert ops.vsa_device_status(ws) == 6                  # VSA_ERR_DEVICE_CHECK
        ops.vsa_packed_attn_fwd(q, k, v, good, cu, out, ws)
        assert ops.vsa_device_status(ws) == 6
        ops.vsa_packed_attn_fwd(q, k, v, good, good, out, ws)
        assert ops.vsa_device_status(ws) == 0 and torch.equal(out, want)


def test_forward_captured_with_changing_borders(ops):
    """One captured call replayed after the borders and the tensors changed."""
    q, k, v = randn(1, 256, 4, 64), randn(2, 256, 2, 64), randn(3, 256, 2, 64)
    cu = cu_of([100, 156, 0]).cuda()
    ws = workspace(ops, q, k, cu)
    out = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ops.vsa_packed_attn_fwd(q, k, v, cu, cu, out, ws)
    for lens in ([100, 156, 0], [1, 250, 5], [0, 0, 256]):
        cu.copy_(cu_of(lens))
        q.copy_(randn(sum(lens[:1]), 256, 4, 64))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, forward(ops, q, k, v, cu, cu)[0])
    assert ops.vsa_device_status(ws) == 0


def test_forward_on_another_stream_and_repeatable(ops):
    q, k, v = randn(1, 500, 8, 128), randn(2, 500, 2, 128), randn(3, 500, 2, 128)
    cu = cu_of([499, 1]).cuda()
    want = forward(ops, q, k, v, cu, cu)
    ws, out = workspace(ops, q, k, cu), torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ops.vsa_packed_attn_fwd(q, k, v, cu, cu, out, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want[0])


def test_forward_repeats_its_bits_with_many_short_works_per_cta(ops):
    """Sequences whose last pair of tiles has rows in one tile only, with longer ones around them: a tile that sits one
    piece of work out must not touch the other's operands.  (A fault of timing: the same call a few hundred times.)"""
    lens = [340, 22, 552, 76, 395, 207, 1056]
    q, k, v = randn(1, sum(lens), 24, 128), randn(2, sum(lens), 8, 128), randn(3, sum(lens), 8, 128)
    cu = cu_of(lens).cuda()
    ws = workspace(ops, q, k, cu)
    want = forward(ops, q, k, v, cu, cu, ws=ws)
    r = attention(q.cpu(), k.cpu(), v.cpu(), cu.cpu(), cu.cpu(), True)
    check(want[0], r["out"], r["out_tol"], "out")
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[2])
    differ = torch.zeros((), dtype=torch.bool, device="cuda")
    for _ in range(600):
        ops.vsa_packed_attn_fwd(q, k, v, cu, cu, out, ws, lse=lse)
        differ |= (out != want[0]).any() | (lse != want[2]).any()
    assert not differ and ops.vsa_device_status(ws) == 0
