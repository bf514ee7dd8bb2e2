"""The binding's checks of linear attention's calls and of the batch plan (no GPU): what is refused before the library is
called.  Tensors are CPU tensors that say they are on a device, and the library is a stand-in that notes its calls."""
import pytest
import torch

from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import workloads as wl

SHAPE = wl.LayerShape(nheads=2, head_dim=64, d_state=128, n_groups=1)
H, P, N, G = SHAPE.nheads, SHAPE.head_dim, SHAPE.d_state, SHAPE.n_groups
F32, I32, U8 = torch.float32, torch.int32, torch.uint8
DESC = bd.layer_desc(SHAPE)


class OnDevice:
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


class Stream:
    cuda_stream = 0


@pytest.fixture
def library(monkeypatch):
    fake = Library()
    monkeypatch.setattr(bd, "_lib", fake)
    return fake


def dev(*shape, dtype=torch.bfloat16):
    return OnDevice(torch.zeros(shape, dtype=dtype))


def step(batch=3, ntok=2, **kw):
    a = dict(ssm_pool=dev(4, H, P, N), slot_ids=dev(batch, dtype=I32), xbc=dev(batch, ntok, SHAPE.conv_dim), log_decay=dev(H, dtype=F32),
             y=dev(batch, ntok, H * P), positions=dev(batch, ntok, dtype=I32), inv_freq=dev(32, dtype=F32), stream=Stream)
    a.update(kw)
    bd.la_state_update(DESC, a.pop("ssm_pool"), a.pop("slot_ids"), a.pop("xbc"), a.pop("log_decay"), a.pop("y"), **a)


def prep(T=5, **kw):
    a = dict(k=dev(T, G, N), q=dev(T, G, N), k_out=dev(T, G, N), q_out=dev(T, G, N), positions=dev(T, dtype=I32), inv_freq=dev(64, dtype=F32),
             stream=Stream)
    a.update(kw)
    bd.la_qk_norm_rope(DESC, a.pop("k"), a.pop("q"), a.pop("k_out"), a.pop("q_out"), **a)


def scan(T=100, nseq=3, **kw):
    a = dict(ssm_pool=dev(4, H, P, N), cu=dev(nseq + 1, dtype=I32), ids=dev(nseq, dtype=I32), v=dev(T, H, P), k=dev(T, G, N), q=dev(T, G, N),
             log_decay=dev(H, dtype=F32), y=dev(T, H, P), ws=dev(1 << 12, dtype=U8), stream=Stream)
    a.update(kw)
    bd.la_chunk_scan(DESC, *[a.pop(n) for n in ("ssm_pool", "cu", "ids", "v", "k", "q", "log_decay", "y", "ws")], **a)


def plan(rows=3, **kw):
    a = dict(new=dev(rows, dtype=I32), past=dev(rows, dtype=I32), table=dev(rows, 2, dtype=I32), block=8, num_slots=6, cu_seqlens=dev(rows + 1, dtype=I32),
             slot_ids=dev(rows, dtype=I32), stream=Stream)
    a.update(kw)
    bd.mamba_batch_plan(a.pop("new"), a.pop("past"), a.pop("table"), a.pop("block"), a.pop("num_slots"), **a)


SHORT = [
    (step, dict(positions=dev(3, 1, dtype=I32))), (step, dict(positions=dev(3, 2, dtype=torch.int64))), (step, dict(xbc=dev(3, 2, SHAPE.conv_dim - 8))),
    (step, dict(xbc=dev(3, 2, SHAPE.conv_dim, dtype=F32))), (step, dict(k_weight=dev(N - 1, dtype=F32))), (step, dict(q_weight=dev(N))),
    (step, dict(log_decay=dev(1, dtype=F32))), (step, dict(scratch_slots=dev(3, 1, dtype=I32))), (step, dict(y=dev(3, 1, H * P))),
    (step, dict(ssm_pool=OnDevice(torch.zeros(4, H, N, P, dtype=torch.bfloat16).transpose(2, 3)))), (step, dict(inv_freq=dev(32))),
    (prep, dict(q=dev(4, G, N))), (prep, dict(k=dev(5, N, G))), (prep, dict(k=OnDevice(torch.zeros(5, N, 2, dtype=torch.bfloat16)[..., 0]))),
    (prep, dict(positions=dev(4, dtype=I32))), (prep, dict(q_out=dev(5, G, N, dtype=F32))), (prep, dict(k_out=dev(6, G, N))),
    (prep, dict(k=OnDevice(torch.zeros(1, G, N, dtype=torch.bfloat16).expand(5, G, N)))),
    (scan, dict(k=dev(99, G, N))), (scan, dict(v=OnDevice(torch.zeros(100, P, H, dtype=torch.bfloat16).transpose(1, 2)))),
    (scan, dict(y=dev(99, H, P))), (scan, dict(y=OnDevice(torch.zeros(100, H, 2 * P, dtype=torch.bfloat16)[..., :P]))),
    (scan, dict(ids=dev(2, dtype=I32))), (scan, dict(has_initial_state=dev(2, dtype=U8))), (scan, dict(has_initial_state=dev(3, dtype=I32))),
    (scan, dict(ckpt_slots=dev(2, 4, dtype=I32), ckpt_interval=128)), (scan, dict(ckpt_slots=dev(12, dtype=I32), ckpt_interval=128)),
    (plan, dict(past=dev(2, dtype=I32))), (plan, dict(table=dev(2, 2, dtype=I32))), (plan, dict(table=dev(6, dtype=I32))),
    (plan, dict(table=OnDevice(torch.zeros(2, 3, dtype=I32).t()))), (plan, dict(cu_seqlens=dev(3, dtype=I32))), (plan, dict(slot_ids=dev(2, dtype=I32))),
    (plan, dict(positions=dev(4, dtype=I32), token_rows=dev(5, dtype=I32))), (plan, dict(ckpt_slots=dev(2, 2, dtype=I32))),
    (plan, dict(has_initial_state=dev(3, dtype=I32))), (plan, dict(new=dev(3, dtype=torch.int64))),
]


@pytest.mark.parametrize("call,change", SHORT, ids=lambda x: getattr(x, "__name__", None) or "-".join(x))
def test_what_the_library_would_read_or_write_past_is_refused(library, call, change):
    with pytest.raises(ValueError):
        call(**change)
    assert not library.calls


def test_good_calls_are_passed_on_with_the_tensors_strides(library):
    step()
    prep()
    rows = torch.zeros(100, SHAPE.conv_dim, dtype=torch.bfloat16)
    v, k, q = rows[:, :H * P].view(100, H, P), rows[:, H * P:H * P + N].view(100, G, N), rows[:, H * P + N:]
    scan(v=OnDevice(v), k=OnDevice(k), q=OnDevice(q))
    plan(table=OnDevice(torch.zeros(3, 7, dtype=I32)[:, 2:4]), positions=dev(9, dtype=I32))
    assert [n for n, _ in library.calls] == ["la_state_update", "la_qk_norm_rope", "la_chunk_scan", "mamba_batch_plan"]
    args = library.calls[2][1]
    assert [args[i] for i in (13, 15, 17)] == [SHAPE.conv_dim] * 3
    args = library.calls[3][1]
    assert args[4] == 7 and args[5] == 2 and args[8] == 9


def test_a_single_token_may_have_any_stride(library):
    one = torch.zeros(1, SHAPE.conv_dim, dtype=torch.bfloat16)
    prep(T=1, k=OnDevice(one[:, :N].as_strided((1, G, N), (0, N, 1))))
    assert library.calls[0][1][2] == G * N
