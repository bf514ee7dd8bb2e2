"""A linear attention layer served the way an engine would: prompts prefilled in ragged batches with a state kept at
every block's end, a request that starts from another's kept state, tokens decoded one at a time from a captured
graph, drafts checked and committed.

    python examples/la_layer.py [--nheads H --head-dim P --d-state N --groups G --block B]

The projections around the mixer are left out: the layer starts from the channels [v | k | q] and ends at the heads'
outputs.  Weights and inputs are random.  The run prints how far the outputs of each way of serving lie from one pass
over the same tokens.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from recurrent_state_update_gb300 import binding as bd  # noqa: E402
from recurrent_state_update_gb300 import workloads as wl  # noqa: E402


class LinearAttentionLayer:
    """One layer's weights and its pool of pages, each a state.  A request's row of the block table names the page of the
    state after each block of its tokens.  Every call runs on the current stream."""

    def __init__(self, shape: wl.LayerShape, pages: int, block: int = 128, state: str = wl.F32, act: str = wl.BF16, seed: int = 0,
                 device="cuda"):
        self.shape, self.block, self.desc = shape, block, bd.layer_desc(shape, state=state, act=act)
        self.act = torch.bfloat16 if act == wl.BF16 else torch.float32
        H, N = shape.nheads, shape.d_state
        g = torch.Generator().manual_seed(seed)
        self.log_decay = -torch.exp(-torch.rand(H, generator=g) * math.log(500.0)).to(device)
        self.prep = dict(qk_norm=True, eps=1e-6, k_weight=(1 + 0.1 * torch.randn(N, generator=g)).to(device),
                         q_weight=(1 + 0.1 * torch.randn(N, generator=g)).to(device),
                         inv_freq=(10000.0 ** (-torch.arange(0, N, 2) / N)).float().to(device))
        self.pool = torch.zeros(pages, H, shape.head_dim, N, dtype=torch.bfloat16 if state == wl.BF16 else torch.float32, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)

    def plan(self, new, past, table, tokens):
        """Device buffers of a batch of at most `tokens` tokens; `fill` makes them anew from what new and past hold then."""
        rows, i32 = new.shape[0], dict(dtype=torch.int32, device=new.device)
        out = dict(cu_seqlens=torch.zeros(rows + 1, **i32), slot_ids=torch.zeros(rows, **i32), copy_src=torch.zeros(rows, **i32),
                   copy_dst=torch.zeros(rows, **i32), ckpt_slots=torch.zeros(rows, table.shape[1], **i32),
                   positions=torch.zeros(tokens, **i32), has_initial_state=torch.zeros(rows, dtype=torch.uint8, device=new.device))

        def fill():
            bd.mamba_batch_plan(new, past, table, self.block, self.pool.shape[0], err_word=self.err, **out)
            bd.mamba_slot_copy(self.desc, self.pool, out["copy_src"], out["copy_dst"], err_word=self.err)
            return out
        return fill

    def prefill(self, fill, rows, y=None, work=None):
        """Channels (tokens, conv_dim) of a planned batch; rows behind its last token are left alone.  Returns (tokens, H, P)."""
        s, T, b = self.shape, rows.shape[0], fill()
        HP, GN = s.nheads * s.head_dim, s.n_groups * s.d_state
        v, k, q = rows[:, :HP].view(T, s.nheads, s.head_dim), rows[:, HP:HP + GN], rows[:, HP + GN:]
        k2, q2 = (torch.empty(T, s.n_groups, s.d_state, dtype=self.act, device=rows.device) for _ in range(2))
        bd.la_qk_norm_rope(self.desc, k, q, k2, q2, positions=b["positions"], **self.prep)
        y = torch.empty(T, s.nheads, s.head_dim, dtype=self.act, device=rows.device) if y is None else y
        n = b["slot_ids"].shape[0]
        if work is None:
            work = torch.empty(bd.la_chunk_scan_workspace_bytes(self.desc, T, n), dtype=torch.uint8, device=rows.device)
        bd.la_chunk_scan(self.desc, self.pool, b["cu_seqlens"], b["slot_ids"], v, k2, q2, self.log_decay, y, work,
                         has_initial_state=b["has_initial_state"], ckpt_slots=b["ckpt_slots"], ckpt_interval=self.block, err_word=self.err)
        return y

    def step(self, fill, past, x, y, scratch=None):
        """Channels (rows, ntok, conv_dim) of a planned batch of ntok tokens a row, the states after each to `scratch`
        (rows, ntok) if it is given; outputs to y."""
        b = fill()
        positions = (past[:, None] + torch.arange(x.shape[1], dtype=torch.int32, device=x.device)).contiguous()
        bd.la_state_update(self.desc, self.pool, b["slot_ids"], x, self.log_decay, y, scratch_slots=scratch, positions=positions,
                           err_word=self.err, **self.prep)
        return b

    def check(self):
        """Raises what the kernels flagged (synchronises)."""
        word = int(self.err.item())
        if word:
            raise RuntimeError(f"the layer's calls flagged {word:#x}")


def serve(layer, x, prompt, chunk, decode, drafts, accept):
    """Each request's channels x[i] (tokens, conv_dim) through the layer: a prompt of prompt[i] tokens, `chunk` at most
    (a multiple of the block) a request and batch, `decode` single tokens, `drafts` drafts of which accept[i] are kept.
    One more request takes the first request's first block from its kept state and goes on with the same tokens.
    Returns (outputs of each request (tokens, H * P), outputs of the one more behind its first block)."""
    n, dev, s, B = len(prompt), layer.pool.device, layer.shape, layer.block
    i32 = dict(dtype=torch.int32, device=dev)
    cols = max(p + decode + drafts for p in prompt) // B + 1
    table = torch.arange((n + 1) * cols, **i32).view(n + 1, cols)
    scratch = torch.arange(n * drafts, **i32).view(n, drafts) + (n + 1) * cols
    past, new, out = torch.zeros(n, **i32), torch.zeros(n, **i32), [[] for _ in prompt]
    most = sum(min(p, chunk) for p in prompt)
    fill = layer.plan(new, past, table[:n], most)
    at = [0] * n
    while any(a < p for a, p in zip(at, prompt)):
        take = [min(chunk, p - a) for a, p in zip(at, prompt)]
        new.copy_(torch.tensor(take, **i32))
        rows = torch.zeros(most, s.conv_dim, dtype=layer.act, device=dev)
        rows[:sum(take)] = torch.cat([x[i][at[i]:at[i] + t] for i, t in enumerate(take)])
        y = layer.prefill(fill, rows)[:sum(take)]
        for i, o in enumerate(y.split(take)):
            out[i].append(o.flatten(1))
            at[i] += take[i]
        past.add_(new)
    # another request whose first block of tokens is the first's: its state is there already
    shared = None
    if prompt[0] > B:
        row = table[n:].clone()
        row[0, 0] = table[0, 0]
        tail = x[0][B:prompt[0]].contiguous()
        one = layer.plan(torch.tensor([tail.shape[0]], **i32), torch.tensor([B], **i32), row, tail.shape[0])
        shared = layer.prefill(one, tail).flatten(1)
    # single tokens, each the same graph: what changes is in its buffers
    new.fill_(1)
    fill = layer.plan(new, past, table[:n], n)
    token, y = torch.zeros(n, 1, s.conv_dim, dtype=layer.act, device=dev), torch.zeros(n, 1, s.nheads * s.head_dim, dtype=layer.act, device=dev)

    def one_token():
        layer.step(fill, past, token, y)
        past.add_(1)

    graph = None
    for t in range(decode):
        token.copy_(torch.stack([x[i][at[i]:at[i] + 1] for i in range(n)]))
        if t == 0:
            one_token()  # (before the capture: kernels are loaded with their first launch)
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    one_token()
            graph.replay()
        for i in range(n):
            out[i].append(y[i].clone())
            at[i] += 1
    if drafts:  # (they end in the block they begin in: a commit leaves the state in the page that they were planned to)
        new.fill_(drafts)
        fill = layer.plan(new, past, table[:n], n * drafts)
        yd = torch.zeros(n, drafts, s.nheads * s.head_dim, dtype=layer.act, device=dev)
        b = layer.step(fill, past, torch.stack([x[i][at[i]:at[i] + drafts] for i in range(n)]), yd, scratch)
        bd.mamba_spec_commit(layer.desc, layer.pool, b["slot_ids"], scratch, torch.tensor(accept, **i32), err_word=layer.err)
        for i in range(n):
            out[i].append(yd[i, :accept[i]])
    return [torch.cat(o) for o in out], shared, table


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--nheads", type=int, default=32)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--d-state", type=int, default=128)
    ap.add_argument("--groups", type=int, default=32)
    ap.add_argument("--block", type=int, default=256)
    a = ap.parse_args()
    shape = wl.LayerShape(a.nheads, a.head_dim, a.d_state, a.groups)
    prompt, decode, drafts, accept = [1500, 300, 1], 6, 4, [3, 4, 0]
    n, most = len(prompt), [p + decode + drafts for p in prompt]
    pages = (n + 1) * (max(most) // a.block + 1) + n * drafts
    layer = LinearAttentionLayer(shape, pages, a.block)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = [torch.randn(t, shape.conv_dim, device="cuda", generator=g).to(layer.act) for t in most]
    out, shared, _ = serve(layer, x, prompt, 2 * a.block, decode, drafts, accept)
    layer.check()

    whole = LinearAttentionLayer(shape, n, 1 << 20)  # the same weights, all tokens in one pass
    lens = [int(o.shape[0]) for o in out]
    i32 = dict(dtype=torch.int32, device="cuda")
    fill = whole.plan(torch.tensor(lens, **i32), torch.zeros(n, **i32), torch.arange(n, **i32).view(n, 1), sum(lens))
    y = whole.prefill(fill, torch.cat([t[:m] for t, m in zip(x, lens)])).flatten(1).split(lens)
    whole.check()
    for i, (o, w) in enumerate(zip(out, y)):
        ends = [0, prompt[i], prompt[i] + decode, lens[i]]
        rms = ["%s %.2e" % (name, (o[lo:hi].float() - w[lo:hi].float()).norm() / w[lo:hi].float().norm())
               for name, lo, hi in zip(("prompt", "single tokens", "drafts"), ends, ends[1:]) if hi > lo]
        print("request %d (%d tokens): rms difference from one pass: %s" % (i, lens[i], ", ".join(rms)))
    w = y[0][a.block:prompt[0]].float()
    print("from a kept state: rms difference from one pass: %.2e" % ((shared.float() - w).norm() / w.norm()))


if __name__ == "__main__":
    main()
