"""A gated delta rule layer served the way an engine would: prompts prefilled in one ragged batch, tokens
decoded one at a time, drafts checked and committed, and a sequence whose cache is kept in 8 bits.

    python examples/gdn_layer.py [--nheads H --head-dim P --d-state N --groups G]

The projections around the mixer are left out: the layer starts from the channels [v | k | q] before their
convolution, one step and one write gate a head, and ends at the heads' outputs.  Weights and inputs are
random.  The run prints how far the outputs of each way of serving lie from one pass over the same tokens.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from recurrent_state_update_gb300 import binding as bd  # noqa: E402
from recurrent_state_update_gb300 import workloads as wl  # noqa: E402


def _aligned(n: int) -> int:
    return (n + 255) // 256 * 256


class GatedDeltaLayer:
    """One layer's weights, its slot pools (states and convolution windows) and its 8-bit entries.

    Slot ids and entries are int32 device tensors; -1 pads.  Every call runs on the current stream and
    allocates only its outputs (and the scan's workspace, which it keeps)."""

    def __init__(self, shape: wl.LayerShape, slots: int, entries: int = 0, state: str = wl.BF16, act: str = wl.BF16,
                 seed: int = 0, device="cuda"):
        self.shape, self.desc = shape, bd.layer_desc(shape, state=state, act=act)
        self.act = torch.bfloat16 if act == wl.BF16 else torch.float32
        prm = wl.layer_params(wl.rng(seed, 0), shape)
        self.A, self.dt_bias, self.conv_w = (torch.from_numpy(prm[n]).to(device) for n in ("A", "dt_bias", "conv_w"))
        st = torch.bfloat16 if state == wl.BF16 else torch.float32
        H, P, N = shape.nheads, shape.head_dim, shape.d_state
        self.ssm = torch.zeros(slots, H, P, N, dtype=st, device=device)
        self.conv = torch.zeros(slots, shape.conv_dim, shape.conv_cols, dtype=self.act, device=device)
        self.store = torch.zeros(entries, bd.mamba_int8_entry_bytes(self.desc), dtype=torch.uint8, device=device)
        # an entry holds codes, scales and the convolution window, each on a 256-byte boundary
        at = _aligned(H * P * N) + _aligned(4 * H * N)
        size = shape.conv_dim * shape.conv_cols * self.conv.element_size()
        self.windows = self.store[:, at:at + size].view(self.act).view(entries, shape.conv_dim, shape.conv_cols)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.work = torch.empty(0, dtype=torch.uint8, device=device)

    def _new(self, *size):
        return torch.empty(*size, dtype=self.act, device=self.ssm.device)

    def prefill(self, cu_seqlens, slots, xbc, dt, beta, continues=None):
        """Channels (tokens, conv_dim) of the sequences bounded by cu_seqlens, from their slots' states where
        `continues` says so (uint8) and from nothing otherwise.  Returns (tokens, H, P)."""
        s, T = self.shape, xbc.shape[0]
        v, k, q = (self._new(T, n, d) for n, d in ((s.nheads, s.head_dim), (s.n_groups, s.d_state), (s.n_groups, s.d_state)))
        bd.mamba_conv_varlen(self.desc, cu_seqlens, xbc, self.conv_w, v, k, q, conv_pool=self.conv, slot_ids=slots,
                             has_initial_state=continues, err_word=self.err)
        need = bd.gdn_chunk_scan_workspace_bytes(self.desc, T, cu_seqlens.shape[0] - 1)
        if self.work.numel() < need:
            self.work = torch.empty(need, dtype=torch.uint8, device=self.ssm.device)
        y = self._new(T, s.nheads, s.head_dim)
        bd.gdn_chunk_scan(self.desc, self.ssm, cu_seqlens, slots, v, k, q, dt, beta, self.A, y, self.work,
                          dt_bias=self.dt_bias, has_initial_state=continues, err_word=self.err)
        return y

    def step(self, slots, xbc, dt, beta, scratch=None):
        """Channels (batch, ntok, conv_dim): one token a request, or several drafts whose states go to
        `scratch` (batch, ntok).  Returns (batch, ntok, H * P)."""
        u = self._new(*xbc.shape)
        bd.mamba_conv_update(self.desc, self.conv, slots, xbc, self.conv_w, u, err_word=self.err)
        y = self._new(xbc.shape[0], xbc.shape[1], self.shape.nheads * self.shape.head_dim)
        bd.gdn_state_update(self.desc, self.ssm, slots, u, dt, beta, self.A, y, dt_bias=self.dt_bias,
                            scratch_slots=scratch, err_word=self.err)
        return y

    def commit(self, slots, scratch, accepted):
        """Keeps the first accepted[i] drafts of request i."""
        bd.mamba_spec_commit(self.desc, self.ssm, slots, scratch, accepted, conv_pool=self.conv, err_word=self.err)

    def to_entries(self, slots, entries):
        bd.mamba_ckpt_store_int8(self.desc, self.ssm, slots, entries, self.store, conv_pool=self.conv, err_word=self.err)

    def from_entries(self, entries, slots):
        bd.mamba_ckpt_load_int8(self.desc, self.ssm, entries, slots, self.store, conv_pool=self.conv, err_word=self.err)

    def step_int8(self, entries, xbc, dt, beta):
        """One token a request (batch, 1, conv_dim) on caches held in 8 bits.  Returns (batch, H * P)."""
        u = self._new(*xbc.shape)
        bd.mamba_conv_update(self.desc, self.windows, entries, xbc, self.conv_w, u, err_word=self.err)
        y = self._new(xbc.shape[0], self.shape.nheads * self.shape.head_dim)
        bd.gdn_state_update_int8(self.desc, self.store, entries, u[:, 0], dt[:, 0], beta[:, 0], self.A, y,
                                 dt_bias=self.dt_bias, err_word=self.err)
        return y

    def check(self):
        """Raises what the kernels flagged (synchronises)."""
        word = int(self.err.item())
        if word:
            raise RuntimeError(f"the layer's calls flagged {word:#x}")


def serve(layer, xbc, dt, beta, prompt, decode, accept, tail):
    """Each request's tokens through the layer: a prompt of prompt[i], `decode` single tokens, as many drafts
    as the layer's windows hold, of which accept[i] are kept, and `tail` tokens on an 8-bit cache.

    xbc, dt and beta are lists of one (tokens, ..) tensor a request.  Returns a list of outputs a request,
    (tokens, H * P): prompt, single tokens, kept drafts, tail."""
    n, dev, ns = len(prompt), layer.ssm.device, layer.shape.num_spec

    def i32(a):
        return torch.tensor(a, dtype=torch.int32, device=dev)

    slots = i32(list(range(n)))
    scratch = i32([[n + i * ns + j for j in range(ns)] for i in range(n)])
    at = [0] * n

    def take(count):
        got = [torch.stack([t[i][at[i]:at[i] + count] for i in range(n)]).contiguous() for t in (xbc, dt, beta)]
        return got

    cu = i32([0] + torch.tensor(prompt).cumsum(0).tolist())
    y = layer.prefill(cu, slots, *(torch.cat([t[i][:prompt[i]] for i in range(n)]) for t in (xbc, dt, beta)))
    out = [[p.flatten(1)] for p in y.split(list(prompt))]
    at = list(prompt)
    for _ in range(decode):
        y = layer.step(slots, *take(1))
        for i in range(n):
            out[i].append(y[i])
            at[i] += 1
    if ns:
        y = layer.step(slots, *take(ns), scratch=scratch)
        layer.commit(slots, scratch, i32(accept))
        for i in range(n):
            out[i].append(y[i, :accept[i]])
            at[i] += accept[i]
    if tail:
        layer.to_entries(slots, slots)
        for _ in range(tail):
            y = layer.step_int8(slots, *take(1))
            for i in range(n):
                out[i].append(y[i:i + 1])
                at[i] += 1
        layer.from_entries(slots, slots)
    return [torch.cat(o) for o in out]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--nheads", type=int, default=32)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--d-state", type=int, default=128)
    ap.add_argument("--groups", type=int, default=16)
    a = ap.parse_args()
    shape = wl.LayerShape(a.nheads, a.head_dim, a.d_state, a.groups, conv_kernel=4, num_spec=4)
    prompt, decode, accept, tail = [700, 64, 1], 6, [3, 4, 0], 6
    n = len(prompt)
    layer = GatedDeltaLayer(shape, slots=n * (1 + shape.num_spec), entries=n)
    g = torch.Generator(device="cuda").manual_seed(1)
    most = [p + decode + shape.num_spec + tail for p in prompt]
    xbc = [torch.randn(t, shape.conv_dim, device="cuda", generator=g).to(layer.act) for t in most]
    dt = [torch.randn(t, shape.nheads, device="cuda", generator=g) for t in most]
    beta = [torch.randn(t, shape.nheads, device="cuda", generator=g) for t in most]
    out = serve(layer, xbc, dt, beta, prompt, decode, accept, tail)
    layer.check()

    whole = GatedDeltaLayer(shape, slots=n)  # the same weights, all tokens in one pass
    cu = torch.tensor([0] + [int(o.shape[0]) for o in out], dtype=torch.int32, device="cuda").cumsum(0).int()
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    y = whole.prefill(cu, slots, *(torch.cat([x[:o.shape[0]] for x, o in zip(t, out)]) for t in (xbc, dt, beta)))
    whole.check()
    for i, (o, w) in enumerate(zip(out, y.split([int(o.shape[0]) for o in out]))):
        d, w = o.float() - w.flatten(1).float(), w.flatten(1).float()
        ends = [0, prompt[i], prompt[i] + decode, prompt[i] + decode + accept[i], o.shape[0]]
        rms = ["%s %.2e" % (name, d[lo:hi].norm() / w[lo:hi].norm())
               for name, lo, hi in zip(("prompt", "single tokens", "drafts", "8-bit cache"), ends, ends[1:]) if hi > lo]
        print("request %d (%d tokens): rms difference from one pass: %s" % (i, o.shape[0], ", ".join(rms)))


if __name__ == "__main__":
    main()
