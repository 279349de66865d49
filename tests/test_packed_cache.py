"""Softmax attention over a cache of keys and values that is kept in place: every
sequence has room to grow, and what it has not filled yet is passed as a
sequence without queries."""
import math

import pytest
import torch

from packed_ref import attention, check, cu_of
from test_packed_attn import ops, randn  # noqa: F401  (ops is a fixture)

pytestmark = pytest.mark.gpu


def borders(queries, keys, room):
    """cu_q, cu_k: each sequence's queries on its keys, and none on the rest of its room."""
    cu_k = [x for i, n in enumerate(keys) for x in (i * room, i * room + n)] + [len(keys) * room]
    return cu_of([x for n in queries for x in (n, 0)]).cuda(), torch.tensor(cu_k, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("room", [260, 2000])            # one share of the keys, and several
def test_generation_over_a_cache_in_place(ops, room, d):  # noqa: F811
    """Prompts, then single tokens, these by one captured call that is replayed while the cache grows under it: no key
    moves, and what the room holds before (NaN, infinity) reaches no result."""
    hq, hk, singles = 6, 2, 4
    prompt = [room - singles, 1, room // 2 + 3]          # the first one fills its room to the last row
    whole = [p + singles for p in prompt]
    n = len(prompt)
    x = randn(1, sum(whole), hq + 2 * hk, d)
    start = [sum(whole[:i]) for i in range(n)]
    cache = torch.full((2, n, room, hk, d), math.nan, dtype=torch.bfloat16, device="cuda")
    cache[:, :, ::3] = math.inf
    rows = torch.cat([torch.arange(s, s + p) for s, p in zip(start, prompt)]).cuda()
    for i in range(n):
        for j in range(2):
            cache[j, i, :prompt[i]] = x[start[i]:start[i] + prompt[i], hq + j * hk:hq + (j + 1) * hk]
    keys, values = cache.flatten(1, 2)
    ws = ops.new_workspace_bytes(ops.vsa_packed_attn_workspace_bytes(sum(prompt), n * room, 2 * n, hq, hk, d))
    first = torch.full((sum(prompt), hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.vsa_packed_attn_fwd(x[rows, :hq], keys, values, *borders(prompt, prompt, room), first, ws)
    outs = [(rows, first)]

    one = ops.new_workspace_bytes(ops.vsa_packed_attn_workspace_bytes(n, n * room, 2 * n, hq, hk, d))
    if room == 2000:
        assert one.numel() > 256 + 2 * n * hq * d * 4    # shares of the keys, joined
    q, out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    cu_q, cu_k = borders([1] * n, prompt, room)
    token = torch.tensor([s + p for s, p in zip(start, prompt)], device="cuda")
    place = torch.tensor([i * room + p for i, p in enumerate(prompt)], device="cuda")

    def step():
        new = x[token]
        q.copy_(new[:, :hq])
        keys[place], values[place] = new[:, hq:hq + hk], new[:, hq + hk:]
        token.add_(1)
        place.add_(1)
        cu_k[1::2] += 1
        ops.vsa_packed_attn_fwd(q, keys, values, cu_q, cu_k, out, one)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for _ in range(singles):
        at = token.clone()
        graph.replay()
        outs.append((at, out.clone()))
    assert ops.vsa_device_status(ws) == 0 and ops.vsa_device_status(one) == 0
    assert cu_k[1::2].tolist() == [i * room + w for i, w in enumerate(whole)]
    cu = cu_of(whole)
    r = attention(x[:, :hq].cpu(), x[:, hq:hq + hk].cpu(), x[:, hq + hk:].cpu(), cu, cu, True)
    for at, got in outs:
        check(got, r["out"][at.cpu()], r["out_tol"][at.cpu()])
