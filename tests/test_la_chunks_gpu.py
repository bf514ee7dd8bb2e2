"""Linear attention's scan over many chunks: heads that forget slowly, whose state takes hundreds of chunks' decays, cut into
segments and not.

Tolerance, as the error of a head's state over its length (a root of a sum of squares).  Each chunk rounds a value once to 24
bits, up or down as it comes: 2^-24 / sqrt(3) rms of it at most, sqrt(chunks) times that together.  What a chunk adds is off by its
tokens' weights (2^-24), its keys' parts (2^-24) and the sum's own bits, 2^-22 in all.  For 512 chunks 1.02e-6.  A decay that is one
number rounded to 24 bits is off by up to 2^-25 the same way in every chunk: 1.5e-5, and e^(-2.56e-8) rounds to 1."""
import numpy as np
import pytest

from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

from gpu_util import to_dev, to_i32

pytestmark = pytest.mark.gpu

SLOW = [-1e-4, -1e-5, -1e-6, -1e-7, -1e-8, -1e-9, -2e-10, 0.0]  # a head each


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    bld.build()
    bd.lib()
    torch.cuda.set_device(0)


def run(P, N, lens, decay, seed, initial):
    """(error of each head's state over its length by sequence, error word) of one seeded scan into an fp32 pool."""
    import torch
    H, T, n = len(decay), sum(lens), len(lens)
    shape = wl.LayerShape(nheads=H, head_dim=P, d_state=N, n_groups=1)
    desc = bd.layer_desc(shape, state=wl.F32)
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn(T, H, P, device="cuda", generator=g).bfloat16()
    k, q = (torch.randn(T, 1, N, device="cuda", generator=g).bfloat16() for _ in range(2))
    pool = initial * torch.randn(n, H, P, N, device="cuda", generator=g)
    start, y = pool.double(), torch.empty_like(v)
    work = torch.empty(bd.la_chunk_scan_workspace_bytes(desc, T, n), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.la_chunk_scan(desc, pool, to_i32(wl.cu_seqlens(np.asarray(lens, np.int32))), to_i32(range(n)), v, k, q,
                     to_dev(np.asarray(decay, np.float32), wl.F32), y, work, has_initial_state=torch.ones(n, dtype=torch.uint8, device="cuda"),
                     err_word=err)
    l, out, at = torch.tensor(np.asarray(decay, np.float32).astype(np.float64), device="cuda"), [], 0
    for i, m in enumerate(lens):
        if m:
            back = torch.exp(l[:, None] * torch.arange(m - 1, -1, -1, device="cuda", dtype=torch.float64))  # (head, token)
            add = torch.einsum("ht,thp,tn->hpn", back, v[at:at + m].double(), k[at:at + m, 0].double())
            want = torch.exp(l * m)[:, None, None] * start[i] + add
            out.append(((pool[i].double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)).tolist())
        at += m
    return out, int(err.item())


@pytest.mark.parametrize("lens", [[65536], [0] * 9 + [65536], [64, 40000, 0, 1]], ids=["cut", "whole", "ragged"])
@pytest.mark.parametrize("P,N", [(128, 128), (64, 128), (64, 64)])
def test_slow_heads_keep_their_decay_over_many_chunks(P, N, lens):
    errors, word = run(P, N, lens, SLOW, 90, 500.0)  # (what 65536 tokens add is about 256 a value)
    chunks = (max(lens) + 127) // 128
    assert word == 0
    for e in errors:
        assert max(e) <= chunks ** 0.5 * 2.0 ** -24 / 3 ** 0.5 + 2.0 ** -22, errors
