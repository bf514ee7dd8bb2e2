"""The binding's checks of the gated delta rule's calls (no GPU): what is refused before the library is called.

Tensors are CPU tensors that say they are on a device, and the library is a stand-in that notes its calls."""
import pytest
import torch

from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import workloads as wl

SHAPE = wl.LayerShape(nheads=2, head_dim=64, d_state=128, n_groups=1)
H, P, N, G = SHAPE.nheads, SHAPE.head_dim, SHAPE.d_state, SHAPE.n_groups


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
        return lambda *a: self.calls.append(name) or 0


class Stream:
    cuda_stream = 0


@pytest.fixture
def library(monkeypatch):
    fake = Library()
    monkeypatch.setattr(bd, "_lib", fake)
    return fake


def dev(*shape, dtype=torch.bfloat16):
    return OnDevice(torch.zeros(shape, dtype=dtype))


def pool(t=None):
    return dev(4, H, P, N) if t is None else OnDevice(t)


def scan(ssm, nseq=3, tokens=100, **kw):
    f32, i32 = torch.float32, torch.int32
    bd.gdn_chunk_scan(bd.layer_desc(SHAPE), ssm, dev(nseq + 1, dtype=i32), dev(nseq, dtype=i32), dev(tokens, H, P),
                      dev(tokens, G, N), dev(tokens, G, N), dev(tokens, H, dtype=f32), dev(tokens, H, dtype=f32), dev(H, dtype=f32),
                      dev(tokens, H, P), dev(1 << 20, dtype=torch.uint8), stream=Stream, **kw)


@pytest.mark.parametrize("rows,given", [(2, (2, 4)), (0, (0, 4)), (3, (12,)), (3, (3, 2, 2))])
def test_a_checkpoint_table_that_is_not_a_row_a_sequence_is_refused(library, rows, given):
    """The device reads ckpt_slots[sequence * max_ckpt + m] of every sequence."""
    with pytest.raises(ValueError, match="ckpt_slots"):
        scan(pool(), ckpt_slots=dev(*given, dtype=torch.int32), ckpt_interval=64)
    assert not library.calls


@pytest.mark.parametrize("rows", [3, 5])
def test_a_checkpoint_table_of_enough_rows_is_taken(library, rows):
    scan(pool(), ckpt_slots=dev(rows, 4, dtype=torch.int32), ckpt_interval=64)
    assert library.calls == ["gdn_chunk_scan"]


def step(ssm, **kw):
    f32, i32 = torch.float32, torch.int32
    bd.gdn_state_update(bd.layer_desc(SHAPE), ssm, dev(2, dtype=i32), dev(2, 1, SHAPE.conv_dim), dev(2, 1, H, dtype=f32),
                        dev(2, 1, H, dtype=f32), dev(H, dtype=f32), dev(2, 1, H * P), stream=Stream, **kw)


POOL = torch.zeros(4, H, P, N, dtype=torch.bfloat16)
WIDE = torch.zeros(4, 2, H, P, N, dtype=torch.bfloat16)
WRONG = {
    "keys before values": POOL.transpose(2, 3),
    "its memory transposed": torch.zeros(4, H, N, P, dtype=torch.bfloat16).transpose(2, 3),
    "every second key": torch.zeros(4, H, P, 2 * N, dtype=torch.bfloat16)[..., ::2],
    "a head too few": torch.zeros(4, H + 1, P, N, dtype=torch.bfloat16)[:, 1:, :, :64],
    "a slot too small": torch.zeros(4, H * P * N - 8, dtype=torch.bfloat16),
    "one number": torch.zeros(4 * H * P * N, dtype=torch.bfloat16),
}
RIGHT = {"dense": POOL, "slots apart": WIDE[:, 0], "flat": POOL.view(4, -1), "one slot": POOL[:1], "room behind": WIDE.view(4, -1),
         "empty": POOL[:0]}


@pytest.mark.parametrize("call", [step, scan])
@pytest.mark.parametrize("layout", WRONG)
def test_a_pool_whose_slots_are_not_dense_states_is_refused(library, call, layout):
    """The device reads a slot as (nheads, head_dim, d_state) without gaps."""
    with pytest.raises(ValueError, match="ssm_pool"):
        call(pool(WRONG[layout]))
    assert not library.calls


@pytest.mark.parametrize("call", [step, scan])
@pytest.mark.parametrize("layout", RIGHT)
def test_a_pool_of_dense_slots_is_taken(library, call, layout):
    call(pool(RIGHT[layout]))
    assert len(library.calls) == 1
