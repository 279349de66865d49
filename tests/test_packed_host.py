"""Host-side checks of the operators over packed sequences (no GPU work): bad
arguments are refused with the documented status codes before the device is
touched, and the torch front-end refuses tensors it cannot pass on."""
import pytest
import torch

from block_sparse_attention_30_b200 import _lib, build, ops

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation returns first


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


ATTN = dict(total_q=100, total_k=100, n_seq=3, heads_q=8, heads_kv=2, d=64)
DECAY = dict(total=100, n_seq=3, heads=4, d=64)

# argument names in the order of the C calls
FWD = ("q q_stride k k_stride v v_stride cu_q cu_k out out_stride out_f32 lse total_q total_k n_seq heads_q heads_kv d causal "
       "ws ws_bytes stream").split()
BWD = ("q q_stride k k_stride v v_stride out_f32 dout dout_stride cu_q cu_k lse dq dq_stride dk dk_stride dv dv_stride total_q "
       "total_k n_seq heads_q heads_kv d causal ws ws_bytes stream").split()
DFWD = ("q q_stride k k_stride v v_stride log_decay cu state_in state_out out out_stride scale total n_seq heads d ws ws_bytes "
        "stream").split()
DBWD = ("q q_stride k k_stride v v_stride dout dout_stride log_decay cu state_in dstate_out dq dq_stride dk dk_stride dv dv_stride "
        "dstate_in scale total n_seq heads d ws ws_bytes stream").split()
STEP = "q q_stride k k_stride v v_stride log_decay state state_out out out_stride scale batch heads d stream".split()


def call(L, name, order, **given):
    a = dict(scale=0.125, causal=1, ws=FAKE, ws_bytes=1 << 40, stream=None, state_in=None, state_out=None, dstate_out=None,
             dstate_in=None, batch=100, **(ATTN if "attn" in name and "decay" not in name else DECAY))
    if order is STEP:
        a.update(state=FAKE, state_out=FAKE)
    a.update({k: v for k, v in given.items() if k in ATTN or k in DECAY or k == "batch"})
    for n in order:
        if n.endswith("_stride"):
            heads = a["heads"] if "heads" in order else a["heads_kv"] if n[:-7] in ("k", "v", "dk", "dv") else a["heads_q"]
            a[n] = max(1, heads) * max(1, a["d"])
        elif n not in a:
            a[n] = FAKE
    a.update(given)
    return getattr(L, name)(*[a[n] for n in order])


CALLS = {"vsa_packed_attn_fwd": FWD, "vsa_packed_attn_bwd": BWD, "vsa_decay_attn_fwd": DFWD, "vsa_decay_attn_bwd": DBWD,
         "vsa_decay_attn_step": STEP}


@pytest.mark.parametrize("name", CALLS)
def test_shapes_are_refused(L, name):
    order = CALLS[name]
    bad = [(dict(d=96), UNSUPPORTED), (dict(d=0), INVALID)]
    if "packed" in name:
        bad += [(dict(n_seq=0), INVALID), (dict(total_q=-1), INVALID), (dict(total_k=-1), INVALID), (dict(heads_q=0), INVALID),
                (dict(heads_kv=0), INVALID), (dict(heads_q=7), INVALID), (dict(heads_q=258, heads_kv=2), UNSUPPORTED),
                (dict(total_q=1 << 30), UNSUPPORTED), (dict(total_k=1 << 30), UNSUPPORTED), (dict(n_seq=1 << 24), UNSUPPORTED),
                (dict(heads_q=1 << 16, heads_kv=1 << 16), UNSUPPORTED),
                (dict(total_q=(1 << 30) - 1, heads_q=128 * 64, heads_kv=64), UNSUPPORTED)]     # more CTAs than a grid holds
    elif order is STEP:
        bad += [(dict(batch=-1), INVALID), (dict(heads=0), INVALID), (dict(heads=1 << 16), UNSUPPORTED)]
    else:
        bad += [(dict(n_seq=0), INVALID), (dict(total=-1), INVALID), (dict(heads=0), INVALID), (dict(total=1 << 30), UNSUPPORTED),
                (dict(n_seq=1 << 24), UNSUPPORTED), (dict(heads=1 << 16), UNSUPPORTED),
                (dict(total=(1 << 30) - 1, heads=1000), UNSUPPORTED)]
    for change, code in bad:
        assert call(L, name, order, **change) == code, change


@pytest.mark.parametrize("name", CALLS)
def test_pointers_and_strides_are_refused(L, name):
    order = CALLS[name]
    for n in order:
        if n.endswith("_stride"):
            full = 4 * 64 if "heads" in order else (2 if n[:-7] in ("k", "v", "dk", "dv") else 8) * 64
            for stride in (full - 8, full + 4, 1 << 38, -full):
                assert call(L, name, order, **{n: stride}) == INVALID, (n, stride)
        elif n in ("q", "k", "v", "out", "dout", "dq", "dk", "dv", "out_f32", "lse", "state_in", "state_out", "dstate_out",
                   "dstate_in", "state"):
            assert call(L, name, order, **{n: FAKE + 4}) == INVALID, n
            optional = ("state_in", "state_out", "dstate_out", "dstate_in") if order is not STEP else ()
            optional += ("out_f32", "lse") if order is FWD else ()
            if n not in optional:
                assert call(L, name, order, **{n: None}) == INVALID, n
        elif n in ("cu_q", "cu_k", "cu", "log_decay"):
            assert call(L, name, order, **{n: None}) == INVALID and call(L, name, order, **{n: FAKE + 2}) == INVALID, n


def test_states_must_not_overlap(L):
    assert call(L, "vsa_decay_attn_fwd", DFWD, state_in=FAKE, state_out=FAKE) == INVALID
    assert call(L, "vsa_decay_attn_bwd", DBWD, dstate_in=FAKE, dstate_out=FAKE) == INVALID


def test_workspaces_are_refused(L):
    size = {"packed": L.vsa_packed_attn_workspace_bytes(*[ATTN[k] for k in ("total_q", "total_k", "n_seq", "heads_q", "heads_kv", "d")]),
            "decay": L.vsa_decay_attn_workspace_bytes(*[DECAY[k] for k in ("total", "n_seq", "heads", "d")])}
    assert all(n >= 256 for n in size.values())
    for name, order in CALLS.items():
        if order is STEP:
            continue
        for change in (dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=255), dict(ws_bytes=0)):
            assert call(L, name, order, **change) == WORKSPACE, (name, change)
    # single tokens over a long cache: the key axis is split, and the partial results need room
    few = dict(total_q=2, total_k=200000, n_seq=2, heads_q=8, heads_kv=2, d=128)
    n = L.vsa_packed_attn_workspace_bytes(*few.values())
    assert n > 256 + 2 * 8 * 128 * 4
    assert call(L, "vsa_packed_attn_fwd", FWD, **few, ws_bytes=n - 1) == WORKSPACE
    # one long sequence: states at the borders of its segments
    n = L.vsa_decay_attn_workspace_bytes(100000, 1, 4, 128)
    assert n > 256 + 4 * 128 * 128 * 4
    assert call(L, "vsa_decay_attn_fwd", DFWD, total=100000, n_seq=1, d=128, ws_bytes=255) == WORKSPACE


def test_workspace_bytes_of_invalid_shapes_are_zero(L):
    assert L.vsa_packed_attn_workspace_bytes(10, 10, 1, 7, 2, 64) == 0
    assert L.vsa_packed_attn_workspace_bytes(10, 10, 1, 8, 2, 80) == 0
    assert L.vsa_packed_attn_workspace_bytes(10, 10, 0, 8, 2, 64) == 0
    assert L.vsa_packed_attn_workspace_bytes(0, 0, 1, 8, 2, 64) >= 256
    assert L.vsa_decay_attn_workspace_bytes(10, 1, 4, 32) == 0
    assert L.vsa_decay_attn_workspace_bytes(-1, 1, 4, 64) == 0
    assert L.vsa_decay_attn_workspace_bytes(0, 5, 4, 64) >= 256


def test_calls_without_rows_need_no_device(L):
    assert call(L, "vsa_packed_attn_fwd", FWD, total_q=0, q=None, out=None) == OK
    assert call(L, "vsa_packed_attn_bwd", BWD, total_q=0, total_k=0, q=None, k=None, v=None, dout=None, dq=None, dk=None, dv=None,
                out_f32=None, lse=None) == OK
    assert call(L, "vsa_decay_attn_step", STEP, batch=0, q=None, k=None, v=None, out=None, state=None, state_out=None) == OK


def test_front_end_refuses_tensors():
    """Shapes, types and layouts that cannot be passed on fail with an assertion, before anything is called."""
    x, cu = torch.zeros(10, 2, 64, dtype=torch.bfloat16), torch.tensor([0, 10], dtype=torch.int32)
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(AssertionError):
        ops.vsa_packed_attn_fwd(x, x, x, cu, cu, x, ws)                        # not on a CUDA device
    with pytest.raises(AssertionError):
        ops.vsa_decay_attn_fwd(x, x, x, torch.zeros(2), cu, x, ws)
    with pytest.raises(AssertionError):
        ops.vsa_decay_attn_step(x, x, x, torch.zeros(2), torch.zeros(10, 2, 64, 64), x)
    with pytest.raises(AssertionError):
        ops._packed_shape(x[0])
    with pytest.raises(AssertionError):
        ops._borders(cu)


@pytest.mark.gpu
def test_front_end_refuses_cuda_tensors():
    x = torch.zeros(10, 4, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    ws = ops.new_workspace_bytes(ops.vsa_packed_attn_workspace_bytes(10, 10, 1, 4, 4, 64))
    ops.vsa_packed_attn_fwd(x, x, x, cu, cu, torch.empty_like(x), ws)
    bad = [dict(q=x.float()), dict(k=x[:, :, :32]), dict(k=x.transpose(0, 1).contiguous().transpose(0, 1)), dict(v=x[:9]),
           dict(cu_q=cu.long()), dict(cu_q=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(cu_k=cu.cpu()),
           dict(out=x[:9]), dict(workspace=ws.view(torch.float32)), dict(lse=torch.zeros(10, 4, device="cuda")),
           dict(out_f32=torch.zeros(10, 4, 64, device="cuda", dtype=torch.float16))]
    for change in bad:
        a = dict(q=x, k=x, v=x, cu_q=cu, cu_k=cu, out=torch.empty_like(x), workspace=ws)
        a.update(change)
        with pytest.raises(AssertionError):
            ops.vsa_packed_attn_fwd(**a)
    with pytest.raises(_lib.VSAError):                                          # 3 query heads on 2
        ops.vsa_packed_attn_fwd(x[:, :3], x[:, :2], x[:, :2], cu, cu, torch.empty_like(x)[:, :3], ws)
    with pytest.raises(_lib.VSAError):
        ops.vsa_packed_attn_fwd(x, x, x, cu, cu, torch.empty_like(x), ws[:128])
    torch.cuda.synchronize()
