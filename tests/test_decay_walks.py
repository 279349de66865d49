"""Walks of one chunk, one after another in the CTAs of decay_out_kernel: what
batches of short sequences consist of."""
import os
import re

import pytest
import torch

from decay_ref import decay_attention
from packed_ref import HALF, SLACK, check, cu_of
from test_decay_attn import decays, inputs, run
from test_packed_attn import ops  # noqa: F401  (a fixture)

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_30_b200", "csrc",
                      "decay_attn.cu")


def table_barrier():
    """How the kernel's score warps meet before they read the table of powers: the barriers' number, the arrivals that
    complete a phase, and which barrier and parity walk k waits on, as the source has them."""
    text = open(SOURCE, encoding="utf-8").read()
    place, arrivals = re.search(r"mbar_init\(&bars->pow_ready(\[\w+\])?, (\d+)\)", text).groups()
    at, parity = re.search(r"mbar_wait\(&bars->pow_ready(?:\[([^\]]+)\])?, ([^,]+), abort_flag\)", text).groups()
    number = int(re.search(r"pow_ready\[(\d+)\]", text).group(1)) if place else 1
    return number, int(arrivals), lambda k: (eval(at, {"k": k}) if at else 0, eval(parity, {"k": k}))


def stuck(number, arrivals, wait, walks):
    """Whether some order of steps leaves the score warps standing for ever.  Two actors, the warps that write the table
    (64 threads) and a warp that only reads it (the others go as this one does); in each walk of one chunk they take
    the piece of work, arrive (a reader only where readers are counted), wait for the table, wait for the scores and hand
    over the weights.  A piece has a place in the queue once every warp has taken the one two before it; walk k's
    scores are formed once all weights of walk k - 1 are there."""
    counted = 2 if arrivals > 64 else 1
    PIECE, ARRIVE, TABLE, SCORES = range(4)
    seen, todo = set(), [((0, PIECE), (0, PIECE), (0,) * number, (0,) * number)]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        actors, phase, pending = state[:2], state[2], state[3]
        moved = False
        for i, (k, at) in enumerate(actors):
            other = actors[1 - i]
            ph, pe = list(phase), list(pending)
            if k == walks:
                continue
            place, parity = wait(k)
            if at == PIECE:
                can, new = other > (k - 2, PIECE), (k, ARRIVE if i < counted else TABLE)
            elif at == ARRIVE:
                can, new = True, (k, TABLE)
                pe[place] += 1
                if pe[place] == counted:
                    ph[place], pe[place] = ph[place] + 1, 0
            elif at == TABLE:                            # the phase of this parity is over: the one in progress has the other
                can, new = phase[place] % 2 != parity, (k, SCORES)
            else:
                can, new = k == 0 or other[0] >= k, (k + 1, PIECE)
            if can:
                moved = True
                todo.append((*[new if j == i else actors[j] for j in range(2)], tuple(ph), tuple(pe)))
        if not moved and any(k < walks for k, _ in actors):
            return True
    return False


def test_no_warp_is_left_behind():
    """No order of the warps' steps makes one of them miss the phase that it waits for (no GPU).  The search itself finds
    the orders that do: one barrier that the table's writers alone complete can be a whole phase ahead of a reader."""
    assert stuck(1, 64, lambda k: (0, k & 1), 6)
    assert not stuck(1, 256, lambda k: (0, k & 1), 6)
    assert not stuck(*table_barrier(), 6)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_many_walks_of_one_chunk(ops, d):  # noqa: F811
    """Some 30 walks a CTA forward and 90 backwards, of sequences of 1 to 128 tokens; twice, with the same bits."""
    lens = [1 + 61 * i % 128 for i in range(720)]
    h = 6
    q, k, v, g, s0, r1 = inputs(lens, h, d, True)
    ld, cu = decays(h), cu_of(lens).cuda()
    got = run(ops, q, k, v, ld, cu, None, s0, g, r1)
    again = run(ops, q, k, v, ld, cu, None, s0, g, r1)
    assert all(torch.equal(got[x], again[x]) for x in got)
    take = [0, 1, 359, 718, 719]                         # these against fp64, element by element
    start = [sum(lens[:i]) for i in take]
    rows = torch.cat([torch.arange(s, s + lens[i]) for i, s in zip(take, start)])
    part = lambda x: x.cpu()[rows]  # noqa: E731
    want = decay_attention(part(q), part(k), part(v), ld.cpu(), cu_of([lens[i] for i in take]), d ** -0.5, s0.cpu()[take], part(g),
                           r1.cpu()[take])
    for x in got:
        check(got[x].cpu()[take if "state" in x else rows], want[x], want[x + "_tol"], x)
    # and the outputs of all: with the weights and the state before the sequence rounded to bf16, and the result
    le, i = torch.tensor(lens, device="cuda"), torch.arange(128, device="cuda")
    here = i < le[:, None]
    zeros = torch.zeros(len(lens), 128, h, d, dtype=torch.float64, device="cuda")
    lay = lambda x: zeros.clone().masked_scatter_(here[..., None, None], x.double()).transpose(1, 2)  # noqa: E731
    lam = torch.exp(ld.double())[:, None, None]
    m = torch.where(i[:, None] >= i, lam ** (i[:, None] - i).clamp_min(0), 0.0) * d ** -0.5
    since = (lam ** (i + 1.0)[:, None]) * d ** -0.5
    a, b, c, x = lay(q), lay(k), lay(v), s0.double()
    w = a @ b.transpose(-1, -2) * m
    out = w @ c + since * (a @ x)
    state = since * (a.abs() @ x.abs())
    tol = HALF * (w.abs() @ c.abs() + state) + SLACK * ((a.abs() @ b.abs().transpose(-1, -2) * m) @ c.abs() + state)
    flat = lambda y: y.transpose(1, 2)[here]  # noqa: E731
    check(got["out"], flat(out), flat(tol + HALF * (out.abs() + tol)), "out of all")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_states_of_long_sequences_among_many_short_ones(ops, d):  # noqa: F811
    """More sequences than the rows have parts (the scan has a place per part's length, not per sequence), all their
    states wanted, and some of several parts: the first one, one that starts with a part's length of rows, two in a row
    and the last; the others of one part, of which two are full and one empty."""
    lens, h = [2] * 150, 2
    lens[0], lens[64], lens[80], lens[81], lens[149] = 300, 129, 515, 700, 257
    lens[1], lens[2], lens[100], lens[101] = 128, 0, 127, 1
    lens[63] = -sum(lens[:63]) % 128                     # sequence 64 starts at a multiple of 128
    q, k, v, g, s0, r1 = inputs(lens, h, d, True)
    ld, cu = decays(h), cu_of(lens).cuda()
    # the workspace holds a state for every 128 rows, twice: that is the length of a part here
    assert ops.vsa_decay_attn_workspace_bytes(sum(lens), len(lens), h, d) == 256 + 2 * (sum(lens) // 128) * h * d * d * 4
    assert sum(lens) // 128 < len(lens)
    got = run(ops, q, k, v, ld, cu, None, s0, g, r1)
    want = decay_attention(*[x.cpu() for x in (q, k, v, ld, cu)], d ** -0.5, *[x.cpu() for x in (s0, g, r1)])
    less = run(ops, q, k, v, ld, cu, None, s0, g, r1, want_states=False)   # and where no final states are wanted
    for r in (got, less):
        for x in r:
            check(r[x], want[x], want[x + "_tol"], x)
