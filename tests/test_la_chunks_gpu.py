"""Linear attention's scan over many chunks: heads that forget slowly, whose state takes hundreds of chunks' decays, cut into
segments and not; what an fp32 pool holds of heads of 128 values, whose keys' parts two groups of warps ready; blocks that work on
more sequences than their ring of units holds; a captured prefill whose lengths change.

Tolerance, as the error of a head's state over its length (a root of a sum of squares).  Each chunk rounds a value once to 24
bits, up or down as it comes: 2^-24 / sqrt(3) rms of it at most, sqrt(chunks) times that together.  What a chunk adds is off by its
tokens' weights (2^-24), its keys' parts (2^-24) and the sum's own bits, 2^-22 in all.  For 512 chunks 1.02e-6.  A decay that is one
number rounded to 24 bits is off by up to 2^-25 the same way in every chunk: 1.5e-5, and e^(-2.56e-8) rounds to 1."""
import numpy as np
import pytest

import la_ref as ref
from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

from gpu_util import to_dev, to_i32
from test_la_gpu import run_scan
from test_la_layer_gpu import example  # noqa: F401  (a fixture)

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


@pytest.mark.parametrize("lens", [[129, 128, 1, 77, 300], [3000], [5] * 40, [0] * 9 + [3000]], ids=["ragged", "cut", "short", "whole"])
@pytest.mark.parametrize("P,N", [(128, 128), (64, 128)])
def test_an_fp32_pool_holds_24_bits_of_any_head(P, N, lens):
    """A part of the keys (or values) lost for some rows leaves 16 bits, 1e-5."""
    errors, word = run(P, N, lens, ref.decays(80, 8), 91, 0.1)
    chunks = (max(lens) + 127) // 128
    assert word == 0
    for e in errors:
        assert max(e) <= chunks ** 0.5 * 2.0 ** -24 / 3 ** 0.5 + 2.0 ** -22, errors


@pytest.mark.parametrize("heads,head_dim,d_state,nseq", [(1, 64, 64, 3000), (2, 128, 128, 1450)])
@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
def test_blocks_take_more_sequences_than_their_ring_holds(heads, head_dim, d_state, nseq, st):
    """19 units a block, of 152, through a ring of 8: slots are used for the third time.  One in twenty has a second chunk."""
    g = wl.rng(92, 0)
    lens = np.where(g.random(nseq) < 0.05, g.integers(129, 135, nseq), g.integers(1, 5, nseq))
    assert heads * nseq > 2 * 8 * 152 + 152
    shape = wl.LayerShape(nheads=heads, head_dim=head_dim, d_state=d_state, n_groups=heads)
    assert run_scan(92, shape, st, wl.BF16, lens.tolist()) == 0


@pytest.mark.parametrize("heads,head_dim", [(2, 128), (8, 64), (40, 64)])  # the first is cut into segments at most lengths
def test_a_captured_prefill_serves_other_lengths(example, heads, head_dim):  # noqa: F811
    """Plan, copies, norm and rotation and scan captured once for 1500 tokens; what runs is what its buffers hold then."""
    import torch
    shape, n, most, B = wl.LayerShape(heads, head_dim, 128, heads), 3, 1500, 128
    i32 = dict(dtype=torch.int32, device="cuda")
    cols = 1 + 2 * most // B
    batches = [([700, 1, 799], [0, 0, 0]), ([0, 5, 1400], [700, 1, 799]), ([1, 0, 0], [700, 6, 2199]), ([128, 300, 77], [701, 6, 2199]),
               ([1500, 0, 0], [829, 306, 2276]), ([0, 0, 0], [2329, 306, 2276])]
    g = torch.Generator(device="cuda").manual_seed(9)
    rows = [torch.randn(most, shape.conv_dim, device="cuda", generator=g).bfloat16() for _ in batches]
    outs = []
    for captured in (False, True):
        layer = example.LinearAttentionLayer(shape, n * cols + 1, B, wl.F32, wl.BF16, seed=4)
        new, past, table = torch.zeros(n, **i32), torch.zeros(n, **i32), torch.randperm(n * cols, generator=torch.Generator().manual_seed(1)).to(**i32).view(n, cols)
        fill, x, y = layer.plan(new, past, table, most), torch.zeros_like(rows[0]), torch.zeros(most, heads, head_dim, dtype=torch.bfloat16, device="cuda")
        work = torch.empty(bd.la_chunk_scan_workspace_bytes(layer.desc, most, n), dtype=torch.uint8, device="cuda")
        layer.prefill(fill, x, y, work)  # (kernels are loaded with their first launch)
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                layer.prefill(fill, x, y, work)
        kept = []
        for (lens, before), r in zip(batches, rows):
            new.copy_(torch.tensor(lens, **i32))
            past.copy_(torch.tensor(before, **i32))
            x.copy_(r)
            y.fill_(7.0)
            graph.replay() if captured else layer.prefill(fill, x, y, work)
            kept += [y.clone(), layer.pool.clone()]
            assert (y[sum(lens):] == 7.0).all()
        layer.check()
        outs.append(kept)
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert not (outs[0][0] == 7.0).all() and outs[0][-1].abs().max() > 0
