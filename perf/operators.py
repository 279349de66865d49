"""Cases for the causal operators over packed sequences: softmax attention with
grouped heads (forward, training step, single tokens over a long cache) and
linear attention with a decay per head (chunked forward, training step, the
recurrent step for single tokens).

Tokens of all sequences lie one after another in [total, heads, d] tensors;
`cu` holds the sequence borders.  The plain forms pad the sequences to one
length and use elementary operations in 32 bits.
"""
import math
import random

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------ cases

def listed():
    return [
        # latency: four short text prompts (conditioning text of a small video model)
        dict(name="attn_short_prompts", op="attn", lens_q="77,12,120,33", lens_k="", heads=12, kv=12, d=64,
             causal=True, fused=True),
        # ordinary: a batch of prompts of very different lengths, grouped heads
        dict(name="attn_packed_prompts", op="attn", lens_q="1531,64,2048,1,777,300,1290,511,95,1000,2001,129",
             lens_k="", heads=40, kv=8, d=128, causal=True, fused=True),
        # largest: one 16 x 28 x 52 clip, every token after the ones before it
        dict(name="attn_clip_480p", op="attn", lens_q="23296", lens_k="", heads=12, kv=12, d=128, causal=True,
             fused=False),
        # serving: one new token for each of 24 sequences with long caches
        dict(name="attn_single_tokens", op="attn", lens_q=",".join(["1"] * 24),
             lens_k=",".join(str(16 + 347 * i) for i in range(24)), heads=40, kv=8, d=128, causal=True, fused=False),
        # training: a packed batch with grouped heads
        dict(name="attn_train_packed", op="attn_train", lens_q="1024,333,64,1800,7,900", lens_k="", heads=16, kv=4,
             d=64, causal=True, fused=True),
        # training: one long sequence
        dict(name="attn_train_long", op="attn_train", lens_q="8192", lens_k="", heads=12, kv=12, d=128, causal=True,
             fused=False),
        # ordinary: a packed batch that carries its state in and out
        dict(name="decay_packed_prompts", op="decay", lens_q="1531,64,2048,1,777,300,1290,511,95,1000,2001,129",
             heads=12, d=64, fused=True, state=True),
        # largest: one 20 x 28 x 52 clip
        dict(name="decay_clip_480p", op="decay", lens_q="29120", heads=40, d=128, fused=False, state=True),
        # training: packed sequences
        dict(name="decay_train_packed", op="decay_train", lens_q="1024,333,64,1800,7,900", heads=16, d=64, fused=True,
             state=True),
        # training: one 16 x 28 x 52 clip
        dict(name="decay_train_clip", op="decay_train", lens_q="23296", heads=12, d=128, fused=False, state=False),
        # serving: one sequence, one token
        dict(name="decay_step_single", op="decay_step", batch=1, heads=12, d=64),
        # serving: one token for each of 128 sequences
        dict(name="decay_step_batch", op="decay_step", batch=128, heads=40, d=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def _lens(rng, total, most):
    """Lengths (some of zero and one) of at most `most` sequences with about `total` tokens in all."""
    n = _log_int(rng, 1, most)
    cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if n > 3:
        lens[rng.randrange(n)] = rng.randrange(2)
    return lens


def draw(rng: random.Random):
    op = rng.choice(["attn", "attn", "attn_train", "decay", "decay_train", "decay_step"])
    d = rng.choice([64, 128])
    if op == "decay_step":
        heads = rng.choice([1, 5, 12, 16, 40])
        return dict(op=op, batch=_log_int(rng, 1, 128), heads=heads, d=d)
    if op in ("decay", "decay_train"):
        total = _log_int(rng, 64, 12000)
        return dict(op=op, lens_q=",".join(map(str, _lens(rng, total, 16))), heads=rng.choice([1, 3, 12, 16]), d=d,
                    fused=rng.random() < 0.5, state=rng.random() < 0.7)
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 5])
    lens = _lens(rng, _log_int(rng, 64, 4000), 8)
    case = dict(op=op, lens_q=",".join(map(str, lens)), lens_k="", heads=heads, kv=kv, d=d, causal=rng.random() < 0.8,
                fused=False)
    if op == "attn" and rng.random() < 0.5:      # queries that continue longer key sequences (some see no key)
        case["lens_k"] = ",".join(str(max(0, n + rng.randrange(-1 - n // 4, 3000))) for n in lens)
    else:
        case["fused"] = rng.random() < 0.5
    return case


def _ints(text):
    return [int(x) for x in text.split(",")]


# ----------------------------------------------------------------- inputs

def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _pad(lens):
    """Row of each position of the padded [n, longest] layout in the packed one (one extra row of zeros for
    padding), and the padded position of each packed row."""
    n, longest = len(lens), max(max(lens), 1)
    le = torch.tensor(lens, device="cuda")
    start = le.cumsum(0) - le
    pos = torch.arange(longest, device="cuda")
    total = sum(lens)
    rows = torch.where(pos[None] < le[:, None], start[:, None] + pos[None], total)
    back = torch.arange(n * longest, device="cuda").view(n, longest)[pos[None] < le[:, None]]
    return dict(rows=rows, back=back, len=le)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32).to(BF16)


def _qkv(g, total_q, total_k, hq, hkv, d, fused):
    """q, k, v; fused: slices of one [total, (hq + 2 hkv) d] projection, as a model has them."""
    if fused:
        x = _randn(g, total_q, hq + 2 * hkv, d)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return _randn(g, total_q, hq, d), _randn(g, total_k, hkv, d), _randn(g, total_k, hkv, d)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    heads, d = case["heads"], case["d"]
    if case["op"].startswith("decay"):
        # decays spread from 1 - 2^-5 to 1 - 2^-12 over the heads
        e = torch.linspace(5.0, 12.0, heads, dtype=F64)
        s["log_decay"] = torch.log1p(-torch.exp2(-e)).to(F32).cuda()
        s["scale"] = d ** -0.5
    if case["op"] == "decay_step":
        n = case["batch"]
        s["q"], s["k"], s["v"] = (_randn(g, n, heads, d) for _ in range(3))
        s["state"] = torch.randn(n, heads, d, d, generator=g, device="cuda", dtype=F32) * 4
        s["state_out"] = torch.empty_like(s["state"])
        s["out"] = torch.empty_like(s["q"])
        return s
    lens = _ints(case["lens_q"])
    lens_k = _ints(case["lens_k"]) if case.get("lens_k") else lens
    s["q"], s["k"], s["v"] = _qkv(g, sum(lens), sum(lens_k), heads, case.get("kv", heads), d, case["fused"])
    s["cu_q"], s["cu_k"] = _cu(lens), _cu(lens_k)
    s["pad_q"], s["pad_k"] = _pad(lens), _pad(lens_k)
    s["out"] = torch.empty(s["q"].shape, dtype=BF16, device="cuda")
    if case["op"].startswith("attn"):
        s["lse"] = torch.empty(heads, sum(lens), dtype=F32, device="cuda")
    elif case["state"]:
        s["state_in"] = torch.randn(len(lens), heads, d, d, generator=g, device="cuda", dtype=F32) * 4
        s["state_out"] = torch.empty_like(s["state_in"])
    if case["op"].endswith("train"):
        s["dout"] = _randn(g, sum(lens), heads, d)
        s["dq"], s["dk"], s["dv"] = (torch.empty(s[n].shape, dtype=BF16, device="cuda") for n in "qkv")
        if case["op"] == "attn_train":
            s["out_f32"] = torch.empty(s["q"].shape, dtype=F32, device="cuda")
        elif case["state"]:
            s["dstate_out"] = torch.randn(s["state_in"].shape, generator=g, device="cuda", dtype=F32)
            s["dstate_in"] = torch.empty_like(s["state_in"])
    return s


# ------------------------------------------------- plain forms (32 bits)

def _padded(x, pad):
    """[total, h, d] -> fp32 [n, h, longest, d], zeros behind each sequence."""
    x = torch.cat([x.to(F32), torch.zeros_like(x[:1], dtype=F32)])
    return x[pad["rows"]].transpose(1, 2)


def _packed(x, pad):
    """[n, h, longest, d] -> [total, h, d]."""
    return x.transpose(1, 2).flatten(0, 1)[pad["back"]]


def _hidden(s):
    """[n, 1, longest_q, longest_k]: whether a key is hidden from a query."""
    lq, lk = s["pad_q"]["len"], s["pad_k"]["len"]
    i = torch.arange(s["pad_q"]["rows"].shape[1], device="cuda")
    j = torch.arange(s["pad_k"]["rows"].shape[1], device="cuda")
    hidden = (j[None, None] >= lk[:, None, None]) | (i[None, :, None] >= lq[:, None, None])
    if s["case"]["causal"]:
        hidden = hidden | (j[None, None] > i[None, :, None] + (lk - lq)[:, None, None])
    return hidden[:, None]


def _plain_weights(s, q, k):
    """Softmax weights and log2 of the normaliser; rows that see no key have weights 0 and -inf."""
    x = (q * (q.shape[-1] ** -0.5 * math.log2(math.e))) @ k.transpose(-1, -2)
    x.masked_fill_(_hidden(s), -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    p = x.sub_(m).exp2_()
    l = p.sum(-1, keepdim=True)
    p.div_(l.clamp_min(1e-30))
    return p, (m + torch.log2(l)).squeeze(-1)


def _plain_attn(s):
    group = s["case"]["heads"] // s["case"]["kv"]
    q, k, v = _padded(s["q"], s["pad_q"]), _padded(s["k"], s["pad_k"]), _padded(s["v"], s["pad_k"])
    kx, vx = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    p, lse = _plain_weights(s, q, kx)
    o = p @ vx
    out = _packed(o, s["pad_q"]).to(BF16)
    lse = _packed(lse[..., None], s["pad_q"])[..., 0].t().contiguous()
    if s["case"]["op"] == "attn":
        return dict(out=out, lse=lse)
    go = _padded(s["dout"], s["pad_q"])
    dv = p.transpose(-1, -2) @ go
    ds = go @ vx.transpose(-1, -2)
    ds.sub_((go * o).sum(-1, keepdim=True)).mul_(p)
    c = q.shape[-1] ** -0.5
    dq, dk = ds @ kx * c, ds.transpose(-1, -2) @ q * c
    shared = lambda x: x.unflatten(1, (-1, group)).sum(2)  # noqa: E731
    return dict(out=out, dq=_packed(dq, s["pad_q"]).to(BF16), dk=_packed(shared(dk), s["pad_k"]).to(BF16),
                dv=_packed(shared(dv), s["pad_k"]).to(BF16))


CHUNK = 128


def _powers(log_decay, n):
    """fp32 decay^n for fp64 exponents n (negative: 0): [heads, 1, ...] against n's shape."""
    w = torch.exp(log_decay.to(F64).view(-1, *[1] * n.dim()) * n.clamp_min(0))
    return torch.where(n >= 0, w, 0.0).to(F32)


def _chunked(a, b, c, log_decay, backwards):
    """sum over j <= i (j >= i backwards) of decay^|i-j| (a_i . b_j) c_j, all [n, h, L, d], L a multiple of CHUNK:
    inside each chunk by its scores, across chunks by the chunks' states."""
    sign = -1 if backwards else 1
    i = torch.arange(CHUNK, device="cuda", dtype=F64)
    a, b, c = (x.unflatten(2, (-1, CHUNK)) for x in (a, b, c))             # [n, h, chunks, CHUNK, d]
    inside = (a @ b.transpose(-1, -2)).mul_(_powers(log_decay, sign * (i[:, None] - i[None]))[:, None]) @ c
    first, last = (CHUNK - 1 - i, i + 1) if not backwards else (i + 1, CHUNK - 1 - i)
    u = (b * _powers(log_decay, first)[:, None, :, None]).transpose(-1, -2) @ c
    t = torch.arange(a.shape[2], device="cuda", dtype=F64)
    across = _powers(log_decay, CHUNK * (sign * (t[:, None] - t[None]) - 1))   # [h, chunks, chunks]
    before = (across @ u.flatten(3)).view_as(u)
    return (inside + (a * _powers(log_decay, last)[:, None, :, None]) @ before).flatten(2, 3)


def _plain_decay(s):
    pad, ld, scale = s["pad_q"], s["log_decay"], s["scale"]
    longest = pad["rows"].shape[1]
    whole = lambda x: torch.nn.functional.pad(_padded(x, pad), (0, 0, 0, -longest % CHUNK))  # noqa: E731
    q, k, v = whole(s["q"]), whole(s["k"]), whole(s["v"])
    out = _chunked(q, k, v, ld, False)
    n = torch.arange(q.shape[2], device="cuda", dtype=F64)
    lens = pad["len"].to(F64)
    since = _powers(ld, n + 1)[None, :, :, None]                           # decay from the first state to token i
    until = _powers(ld, lens[:, None] - 1 - n[None]).transpose(0, 1)[..., None]   # from token i to the last state
    over = _powers(ld, lens).t()[..., None, None]                          # from the first state to the last
    got = {}
    if s["case"]["state"]:
        out = out + (q * since) @ s["state_in"]
        got["state_out"] = (k * until).transpose(-1, -2) @ v + over * s["state_in"]
    got["out"] = _packed(out[:, :, :longest] * scale, pad).to(BF16)
    if s["case"]["op"] == "decay":
        return got
    go = whole(s["dout"]) * scale
    dq = _chunked(go, v, k, ld, False)
    dk = _chunked(v, go, q, ld, True)
    dv = _chunked(k, q, go, ld, True)
    if s["case"]["state"]:
        dq = dq + (go * since) @ s["state_in"].transpose(-1, -2)
        dk = dk + (v * until) @ s["dstate_out"].transpose(-1, -2)
        dv = dv + (k * until) @ s["dstate_out"]
        got["dstate_in"] = (q * since).transpose(-1, -2) @ go + over * s["dstate_out"]
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        got[name] = _packed(x[:, :, :longest], pad).to(BF16)
    return got


def _plain_step(s):
    q, k, v = (s[n].to(F32) for n in "qkv")
    lam = torch.exp(s["log_decay"].to(F64)).to(F32)[:, None, None]
    state = s["state"] * lam + k[..., :, None] * v[..., None, :]
    out = (q[..., None, :] @ state)[..., 0, :] * s["scale"]
    return dict(out=out.to(BF16), state=state)


# ------------------------------------------------------ the framework's

_workspaces = {}


def _workspace(nbytes):
    """The program's one workspace, as large as any call so far needed."""
    from block_sparse_attention_30_b200 import ops
    if nbytes > _workspaces.get("bytes", 0):
        _workspaces.update(bytes=nbytes, ws=ops.new_workspace_bytes(nbytes))
    return _workspaces["ws"]


def _own_attn(s):
    from block_sparse_attention_30_b200 import ops
    c = s["case"]
    ws = _workspace(ops.vsa_packed_attn_workspace_bytes(s["q"].shape[0], s["k"].shape[0], s["cu_q"].numel() - 1,
                                                        c["heads"], c["kv"], c["d"]))
    if c["op"] == "attn":
        ops.vsa_packed_attn_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], ws, causal=c["causal"],
                                lse=s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    ops.vsa_packed_attn_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], ws, causal=c["causal"],
                            out_f32=s["out_f32"], lse=s["lse"])
    ops.vsa_packed_attn_bwd(s["q"], s["k"], s["v"], s["out_f32"], s["dout"], s["cu_q"], s["cu_k"], s["lse"], s["dq"],
                            s["dk"], s["dv"], ws, causal=c["causal"])
    return dict(out=s["out"], dq=s["dq"], dk=s["dk"], dv=s["dv"])


def _own_decay(s):
    from block_sparse_attention_30_b200 import ops
    c = s["case"]
    ws = _workspace(ops.vsa_decay_attn_workspace_bytes(s["q"].shape[0], s["cu_q"].numel() - 1, c["heads"], c["d"]))
    ops.vsa_decay_attn_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["cu_q"], s["out"], ws, scale=s["scale"],
                           state_in=s.get("state_in"), state_out=s.get("state_out"))
    got = dict(out=s["out"])
    if c["state"]:
        got["state_out"] = s["state_out"]
    if c["op"] == "decay":
        return got
    ops.vsa_decay_attn_bwd(s["q"], s["k"], s["v"], s["dout"], s["log_decay"], s["cu_q"], s["dq"], s["dk"], s["dv"], ws,
                           scale=s["scale"], state_in=s.get("state_in"), dstate_out=s.get("dstate_out"),
                           dstate_in=s.get("dstate_in"))
    got.update(dq=s["dq"], dk=s["dk"], dv=s["dv"])
    if c["state"]:
        got["dstate_in"] = s["dstate_in"]
    return got


def _own_step(s):
    from block_sparse_attention_30_b200 import ops
    ops.vsa_decay_attn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["out"], scale=s["scale"],
                            state_out=s["state_out"])
    return dict(out=s["out"], state=s["state_out"])


def run(state):
    op = state["case"]["op"]
    if op.startswith("attn"):
        return _own_attn(state) if own else _plain_attn(state)
    if op == "decay_step":
        return _own_step(state) if own else _plain_step(state)
    return _own_decay(state) if own else _plain_decay(state)


# ------------------------------------------------------------------- work

def _pairs(lens_q, lens_k, causal):
    """Visible (query, key) pairs: query i of nq sees the first i + 1 + nk - nq keys (causal) or all nk."""
    total = 0
    for nq, nk in zip(lens_q, lens_k):
        if not causal:
            total += nq * nk
        else:
            seen = min(nq, nk)                        # queries that see a key, the last one all nk
            total += seen * nk - seen * (seen - 1) // 2
    return total


def work(case):
    h, d = case["heads"], case["d"]
    if case["op"] == "decay_step":
        n = case["batch"] * h
        return dict(bytes=n * (8 * d * d + 8 * d), flops=5 * n * d * d)
    lens = _ints(case["lens_q"])
    total = sum(lens)
    if case["op"].startswith("attn"):
        lens_k = _ints(case["lens_k"]) if case["lens_k"] else lens
        pairs = _pairs(lens, lens_k, case["causal"]) * h
        q, kv = 2 * total * h * d, 4 * sum(lens_k) * case["kv"] * d
        if case["op"] == "attn":
            return dict(bytes=2 * q + kv + 4 * total * h, flops=4 * pairs * d)
        # q, k, v, dout, out, dq, dk, dv; 2 products forward and 5 backward
        return dict(bytes=4 * q + 2 * kv, flops=14 * pairs * d)
    x, states = 2 * total * h * d, 4 * len(lens) * h * d * d if case["state"] else 0
    # the recurrent form's products: k^T v and q S for each token
    if case["op"] == "decay":
        return dict(bytes=4 * x + 2 * states, flops=4 * total * h * d * d)
    # q, k, v, dout, out, dq, dk, dv; the states before and after, and their gradients
    return dict(bytes=8 * x + 4 * states, flops=12 * total * h * d * d)


# ------------------------------------------- the definition in 64 bits

def _exact_attn(s):
    c = s["case"]
    group = c["heads"] // c["kv"]
    q, k, v = s["q"].to(F64), s["k"].to(F64), s["v"].to(F64)
    train = c["op"] == "attn_train"
    go = s["dout"].to(F64) if train else None
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=F64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    scale = 1 / math.sqrt(c["d"])
    for n in range(len(cq) - 1):
        nq, nk = cq[n + 1] - cq[n], ck[n + 1] - ck[n]
        keys = slice(ck[n], ck[n + 1])
        for h in range(c["heads"]):
            for at in range(0, nq, 4096):
                rows = slice(cq[n] + at, cq[n] + min(nq, at + 4096))
                i = torch.arange(at, min(nq, at + 4096), device="cuda")[:, None] + (nk - nq)
                if not c["causal"]:
                    i = torch.full_like(i, nk)
                sees = torch.arange(nk, device="cuda")[None] <= i
                x = torch.einsum("id,jd->ij", q[rows, h], k[keys, h // group]) * scale
                x = torch.where(sees, x, -math.inf)
                z = torch.logsumexp(x, 1, keepdim=True) if nk else torch.full_like(i, -math.inf, dtype=F64)
                p = torch.where(sees, torch.exp(x - torch.where(torch.isfinite(z), z, 0.0)), 0.0)
                o = p @ v[keys, h // group]
                out[rows, h], lse[rows, h] = o, z[:, 0] / math.log(2)
                if train:
                    g = go[rows, h]
                    dp = torch.einsum("id,jd->ij", g, v[keys, h // group])
                    ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
                    dq[rows, h] = ds @ k[keys, h // group]
                    dk[keys, h // group] += torch.einsum("ij,id->jd", ds, q[rows, h])
                    dv[keys, h // group] += torch.einsum("ij,id->jd", p, g)
    if train:
        return dict(out=out, dq=dq, dk=dk, dv=dv)
    return dict(out=out, lse=lse.t().contiguous())


def _exact_decay(s):
    """The recurrence S_t = decay S_(t-1) + k_t^T v_t, o_t = scale q_t S_t, token by token for all sequences at once;
    its gradient by the recurrence backwards in time."""
    c, lens = s["case"], _ints(s["case"]["lens_q"])
    n, h, d, scale = len(lens), c["heads"], c["d"], s["scale"]
    lam = torch.exp(s["log_decay"].to(F64))[:, None, None]
    start = [sum(lens[:i]) for i in range(n)]
    order = sorted(range(n), key=lambda i: -lens[i])
    rank = torch.tensor(order, device="cuda")
    begin = torch.tensor(start, device="cuda")[rank]
    alive = [sum(x > t for x in lens) for t in range(max(lens))]
    q, k, v = (s[x].to(F64) for x in "qkv")
    state = s["state_in"].to(F64)[rank].clone() if c["state"] else torch.zeros(n, h, d, d, dtype=F64, device="cuda")
    train = c["op"] == "decay_train"
    go = s["dout"].to(F64) * scale if train else None
    out, dq = torch.zeros_like(q), torch.zeros_like(q)
    for t in range(max(lens)):
        m = alive[t]
        at = begin[:m] + t
        now = state[:m]
        now.mul_(lam)
        now.add_(k[at].unsqueeze(-1) * v[at].unsqueeze(-2))
        out[at] = (q[at].unsqueeze(-2) @ now).squeeze(-2) * scale
        if train:
            dq[at] = (now @ go[at].unsqueeze(-1)).squeeze(-1)
    back = torch.argsort(rank)
    got = dict(state_out=state[back]) if c["state"] else {}
    got["out"] = out
    if not train:
        return got
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    ds = s["dstate_out"].to(F64)[rank].clone() if c["state"] else torch.zeros_like(state)
    for t in range(max(lens) - 1, -1, -1):
        m = alive[t]
        at = begin[:m] + t
        now = ds[:m]                                  # the gradient of S_t
        now.add_(q[at].unsqueeze(-1) * go[at].unsqueeze(-2))
        dk[at] = (now @ v[at].unsqueeze(-1)).squeeze(-1)
        dv[at] = (k[at].unsqueeze(-2) @ now).squeeze(-2)
        now.mul_(lam)
    got.update(dq=dq, dk=dk, dv=dv)
    if c["state"]:
        got["dstate_in"] = ds[back]
    return got


def _exact_step(s):
    q, k, v = (s[x].to(F64) for x in "qkv")
    lam = torch.exp(s["log_decay"].to(F64))
    state = s["state"].to(F64) * lam[None, :, None, None] + torch.einsum("nha,nhc->nhac", k, v)
    return dict(out=torch.einsum("nha,nhac->nhc", q, state) * s["scale"], state=state)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("attn"):
        return _exact_attn(s)
    return _exact_step(s) if case["op"] == "decay_step" else _exact_decay(s)
