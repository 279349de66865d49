"""States that leave the library (state_out, dstate_in) are good to fp32: the
weighted operand enters the products in three bf16 parts, one accumulator of
the tensor cores sums 512 tokens at most, and fp32 registers sum those.

Element by element, relative to the sum of the terms' magnitudes:
    weights      a 2-ulp exponential (2^-22) of an argument of which three
                 factors are rounded (3 * 2^-24 x of a weight 2^-x, 2^-21.9 on average
                 over weights of which the mean x is 1 / ln 2), times the operand (2^-24)
    three parts  2^-24
    accumulator  32 products of 16 tokens, each cut off at the 24th bit: 2^-18, and 2^-8 of that for the small parts
    registers    two additions per 512 tokens, 12 for 2816: 2^-20.4
    borders      two at most here, each 2^-22 for its factor and 2^-23 for its fma
which is below 2^-17.  Of a whole state's norm: an accumulator that is cut off 32
times loses half a last bit each time, 2^-25 to 2^-24 of what it holds by then.
The terms are independent, so that the sum's norm is as that of the last terms:
0.9e-6 (simulated below) at most, a weight's error 3.5e-7, two borders 7e-7: together 2^-19.
Two parts instead of three or one accumulator for a whole part are over that, by
the same simulation."""
import pytest
import torch

from decay_ref import CHUNK
from packed_ref import check, cu_of
from test_decay_attn import inputs, run, workspace
from test_decay_long import chunked, slow
from test_packed_attn import ops  # noqa: F401  (a fixture)

ELEMENT, NORM = 2.0 ** -17, 2.0 ** -19


def simulated(memory, tokens, parts, tokens_per_sum):
    """How far (of its norm) a state of `tokens` tokens is from its definition, with the weighted operand in so many
    bf16 parts and so many tokens to an accumulator that is cut off at its 24th bit.  The last tokens first."""
    gen = torch.Generator().manual_seed(0)
    bf16 = lambda x: x.to(torch.bfloat16).double()  # noqa: E731
    b, c = (bf16(torch.randn(tokens, 32, generator=gen)) for _ in range(2))
    w = (1 - 1 / memory) ** torch.arange(tokens, dtype=torch.float64)
    rest = (b * w[:, None]).float().double()
    split = []
    for _ in range(parts):
        split.append(bf16(rest))
        rest = rest - split[-1]

    def add(acc, x):
        m, e = torch.frexp(acc + x)
        return torch.ldexp(torch.trunc(m * 2.0 ** 24), e - 24)

    total = torch.zeros(32, 32)
    for t0 in range(0, tokens, tokens_per_sum):
        high, low = torch.zeros(2, 32, 32, dtype=torch.float64)
        for t in range(t0, min(tokens, t0 + tokens_per_sum), 16):
            high = add(high, split[0][t:t + 16].t() @ c[t:t + 16])
            for s in split[1:]:
                low = add(low, s[t:t + 16].t() @ c[t:t + 16])
        total = total + high.float() + low.float()
    exact = (b * w[:, None]).t() @ c
    return ((total.double() - exact).norm() / exact.norm()).item()


@pytest.mark.parametrize("memory", [256, 1024, 4096])
def test_the_bound_tells_the_forms_apart(memory):
    """(no GPU)"""
    assert simulated(memory, 22 * CHUNK, 3, 512) <= 0.95e-6
    assert simulated(memory, 22 * CHUNK, 2, 512) > NORM
    assert simulated(memory, 22 * CHUNK, 3, 22 * CHUNK) > NORM


@pytest.mark.gpu
@pytest.mark.parametrize("case", [([8141], 40, 64), ([8141], 40, 128), ([2816], 148, 64), ([2816], 148, 128)],
                         ids=lambda c: f"{c[0][0]}-{c[1]}-{c[2]}")
def test_states_are_good_to_fp32(ops, case):  # noqa: F811
    """A sequence of three parts of 22 chunks, and one that is one such part."""
    lens, h, d = case
    q, k, v, g, s0, r1 = inputs(lens, h, d, True)
    ld, cu = slow(h), cu_of(lens).cuda()
    ws = workspace(ops, q, cu)
    borders = (ws.numel() - 256) // (h * d * d * 4)      # of both directions
    assert borders // 2 == lens[0] // (22 * CHUNK)
    got = run(ops, q, k, v, ld, cu, None, s0, g, r1, ws=ws)
    heads = sorted({*range(0, h, 20), h - 1})
    want = chunked(*(x[:, heads] for x in (q, k, v)), ld[heads], cu.cpu(), d ** -0.5, *(x[:, heads] for x in (s0, g, r1)))
    for x in ("state_out", "dstate_in"):
        check(got[x][:, heads], want[x], ELEMENT * want[x + "_mag"], x)
        off = (got[x][:, heads].double() - want[x]).flatten(2).norm(dim=2) / want[x].flatten(2).norm(dim=2)
        assert (off <= NORM).all(), (x, off)
