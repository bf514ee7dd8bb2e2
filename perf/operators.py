"""Cases of the gated delta rule operators: the recurrent step over a slot pool (gdn_state_update), the
chunked scan of a varlen prefill batch (gdn_chunk_scan), and the recurrent step on int8 cache entries
(gdn_state_update_int8) with the entries read back into a pool.

Per head h of a layer with nheads = H, head_dim = P (values), d_state = N (keys), n_groups = G and group
g = h / (H / G), with the state S of shape (P, N):

    a = exp(softplus(dt + dt_bias) * A),  b = sigmoid(beta),  k, q scaled to unit length
    u = b * (v - a * S k),   S <- a * S + u k^T,   y = N**-0.5 * S q

run() with ``own`` false is the plain form of each, in 32 bits with elementary torch operations; with ``own``
true it makes the calls a user of the package makes.  exact() evaluates the recurrence in 64 bits.
"""
import math
import random

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-6          # under the root of the unit-length scaling
CHUNK = 64          # tokens a chunk of the plain scan
CONV = 4            # conv kernel of the layer, whose window an int8 entry holds too


def listed():
    layer = dict(heads=32, groups=16, p=128, n=128, state="bf16", act="bf16")  # generic gated delta layer
    wide = dict(layer, heads=128, groups=8, p=64)  # heads and groups of the package's own Mamba2 configuration
    return [
        # one request being answered: the shortest call there is, where latency counts
        dict(layer, name="step one request", op="step", batch=1, pad=0, ntok=1, draft=False),
        # a full decode batch of a busy server, half of the pool's slots in use
        dict(layer, name="step full batch", op="step", batch=256, pad=0, ntok=1, draft=False),
        # an odd batch with padding rows, states kept in 32 bits
        dict(layer, name="step odd padded f32", op="step", batch=37, pad=4, ntok=1, draft=False, state="f32"),
        # speculative decoding: four drafted tokens, the state after each kept in a scratch slot
        dict(layer, name="step four drafts", op="step", batch=48, pad=0, ntok=4, draft=True),
        # many narrow heads over few key groups
        dict(wide, name="step narrow heads", op="step", batch=61, pad=3, ntok=1, draft=False),
        # one long prompt: few rows, a long chain
        dict(layer, name="scan one prompt", op="scan", nseq=1, tokens=8192, seeded=False, interval=0),
        # a prefill batch of ragged prompts with a prefix-cache checkpoint every 1024 tokens
        dict(layer, name="scan ragged batch", op="scan", nseq=8, tokens=32768, seeded=False, interval=1024),
        # short continuations of stored states: chunks mostly partial
        dict(layer, name="scan short seeded", op="scan", nseq=29, tokens=4001, seeded=True, interval=0),
        # states in 32 bits: the precise form
        dict(layer, name="scan f32 state", op="scan", nseq=3, tokens=2003, seeded=True, interval=0, state="f32"),
        # many narrow heads over few key groups
        dict(wide, name="scan narrow heads", op="scan", nseq=4, tokens=8192, seeded=False, interval=0),
        # one request decoding on the int8 cache, then restored into a pool slot
        dict(layer, name="int8 one request", op="int8", batch=1, steps=8),
        # a batch doing the same
        dict(layer, name="int8 batch", op="int8", batch=192, steps=8),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    heads, groups, p, n = rng.choice([(32, 16, 128, 128), (16, 16, 128, 128), (48, 8, 128, 128), (128, 8, 64, 128),
                                      (24, 4, 64, 128), (8, 4, 64, 64), (12, 2, 32, 64)])
    c = dict(heads=heads, groups=groups, p=p, n=n, state="bf16", act="bf16")
    op = rng.choice(["step", "scan", "int8"])
    work = heads * p * n / (32 * 128 * 128)  # of a token, against the listed layer's
    if op == "step":
        c["state"], c["act"] = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        batch = spread(1, 200 / max(1.0, work))
        draft = rng.random() < 0.3
        return dict(c, op=op, batch=batch, pad=rng.randint(0, batch // 8), ntok=rng.randint(2, 6) if draft else 1, draft=draft)
    if op == "scan":
        if rng.random() < 0.25:
            c["state"], c["act"] = rng.choice([("f32", "bf16"), ("f32", "f32")])
            tokens = spread(1, 2000 / max(1.0, work))
        else:
            tokens = spread(1, 16000 / max(1.0, work))
        return dict(c, op=op, nseq=min(spread(1, 24), tokens), tokens=tokens, seeded=rng.random() < 0.5,
                    interval=rng.choice([0, 64, 512, 1024]) if tokens > 600 else 0)
    return dict(c, op=op, batch=spread(1, 190 / max(1.0, work)), steps=rng.randint(1, 12))


def lengths_of(case):
    """The sequences' lengths: from a third of the mean to as much as closes the sum, the same for a case always."""
    r = random.Random(case["nseq"] * 1000003 + case["tokens"])
    left, out = case["tokens"], []
    for i in range(case["nseq"], 0, -1):
        mean = left // i
        out.append(left if i == 1 else min(max(1, r.randint((mean + 2) // 3, max(1, 5 * mean // 3))), left - (i - 1)))
        left -= out[-1]
    return out


def conv_dim(case):
    return case["heads"] * case["p"] + 2 * case["groups"] * case["n"]


def entry_layout(case):
    """(offset of the scales, bytes of an int8 entry): codes, scales and conv window, each on 256 bytes."""
    up = lambda b: (b + 255) // 256 * 256  # noqa: E731
    codes = up(case["heads"] * case["p"] * case["n"])
    scales = up(case["heads"] * case["n"] * 4)
    return codes, codes + scales + up(conv_dim(case) * (CONV - 1) * BYTES[case["act"]])


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    H, G, P, N = case["heads"], case["groups"], case["p"], case["n"]
    act, st = DTYPE[case["act"]], DTYPE[case["state"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    def silu(x):
        return x / (1 + torch.exp(-x))

    # the layer: decay rates from 1 to 16 and steps around 0.01, so that a head forgets over 10 to 1000 tokens
    A = -torch.exp(torch.rand(H, generator=gen, device=dev) * math.log(16.0))
    step = torch.exp(math.log(0.005) + torch.rand(H, generator=gen, device=dev) * math.log(4.0))
    s = dict(case=case, A=A, dt_bias=torch.log(torch.expm1(step)))

    def pool(slots):
        return (0.1 * normal(slots, H, P, N)).to(st)

    if case["op"] == "scan":
        lens = lengths_of(case)
        T, nseq = case["tokens"], case["nseq"]
        # what the causal conv and its SiLU leave: values, keys and queries
        s.update(v=silu(normal(T, H, P)).to(act), k=silu(normal(T, G, N)).to(act), q=silu(normal(T, G, N)).to(act),
                 dt=normal(T, H), beta=normal(T, H), y=torch.zeros(T, H, P, dtype=act, device=dev))
        at = [0]
        for x in lens:
            at.append(at[-1] + x)
        kept = [x // case["interval"] if case["interval"] else 0 for x in lens]
        S = nseq + sum(kept) + 1
        ids = torch.randperm(S, generator=cpu)
        slots, rest = ids[:nseq], ids[nseq:].tolist()
        ckpt = torch.full((nseq, max(1, max(kept))), -1, dtype=torch.int32)
        for i, n in enumerate(kept):
            for j in range(n):
                ckpt[i, j] = rest.pop()
        s.update(pool=pool(S), cu=torch.tensor(at, dtype=torch.int32, device=dev),
                 slots=slots.to(torch.int32).to(dev), ckpt=ckpt.to(dev) if case["interval"] else None,
                 seeded=torch.full((nseq,), int(case["seeded"]), dtype=torch.uint8, device=dev))
        # the plain form's plan: the token at each place of the padded chunks (T: none) and where states go
        nc = (max(lens) + CHUNK - 1) // CHUNK
        place = torch.full((nseq, nc * CHUNK), T, dtype=torch.int64)
        for i, x in enumerate(lens):
            place[i, :x] = torch.arange(at[i], at[i + 1])
        s.update(place=place.view(nseq, nc, CHUNK).to(dev), slots64=slots.to(dev), nc=nc,
                 token=torch.cat([i * nc * CHUNK + torch.arange(x) for i, x in enumerate(lens)]).to(dev))
        s["saves"] = {}
        for i, n in enumerate(kept):
            for j in range(n):
                s["saves"].setdefault((j + 1) * case["interval"] // CHUNK - 1, []).append((i, int(ckpt[i, j])))
        s["saves"] = {c: tuple(torch.tensor(x, device=dev) for x in zip(*w)) for c, w in s["saves"].items()}
        if own:
            from recurrent_state_update_gb300 import binding as bd
            s["desc"] = layer(bd, case)
            s["work"] = torch.empty(max(16, bd.gdn_chunk_scan_workspace_bytes(s["desc"], T, nseq)), dtype=torch.uint8, device=dev)
        return s

    batch = case["batch"]
    ntok = case["steps"] if case["op"] == "int8" else case["ntok"]
    lead = (ntok, batch, 1) if case["op"] == "int8" else (batch, ntok)
    s.update(xbc=silu(normal(*lead, conv_dim(case))).to(act), dt=normal(*lead, H), beta=normal(*lead, H),
             y=torch.zeros(*lead, H * P, dtype=act, device=dev))
    if case["op"] == "int8":
        E = batch + batch // 4 + 1
        at, size = entry_layout(case)
        ids = torch.randperm(E, generator=cpu)[:batch]
        store = torch.zeros(E, size, dtype=torch.uint8, device=dev)
        codes = store[:, : H * P * N].view(torch.int8).view(E, H, P, N)
        scales = store[:, at:at + 4 * H * N].view(torch.float32).view(E, H, N)
        state = 0.1 * normal(E, H, P, N)
        scales.copy_(state.abs().amax(dim=2) / 127)
        codes.copy_(torch.round(state / scales[:, :, None]).clamp(-127, 127))
        s.update(store=store, codes=codes, scales=scales, entries=ids.to(torch.int32).to(dev), ids=ids.to(dev),
                 pool=torch.zeros(batch + 1, H, P, N, dtype=st, device=dev),
                 back=torch.randperm(batch + 1, generator=cpu)[:batch].to(torch.int32).to(dev))
        s["back64"] = s["back"].long()
    else:
        S = 2 * batch + (batch * ntok if case["draft"] else 0)
        ids = torch.randperm(S, generator=cpu)
        slots = ids[:batch].clone()
        slots[torch.randperm(batch, generator=cpu)[: case["pad"]]] = -1
        live = (slots >= 0).nonzero()[:, 0]
        s.update(pool=pool(S), slots=slots.to(torch.int32).to(dev), live=live.to(dev), live_slots=slots[live].to(dev))
        if case["draft"]:
            s["scratch"] = ids[batch:batch + batch * ntok].view(batch, ntok).to(torch.int32).to(dev)
            s["live_scratch"] = s["scratch"].long()[s["live"]]
    if own:
        from recurrent_state_update_gb300 import binding as bd
        s["desc"] = layer(bd, case)
    return s


def layer(bd, case):
    from recurrent_state_update_gb300 import workloads as wl
    shape = wl.LayerShape(nheads=case["heads"], head_dim=case["p"], d_state=case["n"], n_groups=case["groups"], conv_kernel=CONV)
    return bd.layer_desc(shape, state=case["state"], act=case["act"], dt="f32")


def run(s):
    op = s["case"]["op"]
    if op == "scan":
        return run_scan(s) if own else plain_scan(s)
    if op == "int8":
        return run_int8(s) if own else plain_int8(s)
    return run_step(s) if own else plain_step(s)


def run_step(s):
    from recurrent_state_update_gb300 import binding as bd
    bd.gdn_state_update(s["desc"], s["pool"], s["slots"], s["xbc"], s["dt"], s["beta"], s["A"], s["y"],
                        dt_bias=s["dt_bias"], scratch_slots=s.get("scratch"))
    return {"y": s["y"], "pool": s["pool"]}


def run_scan(s):
    from recurrent_state_update_gb300 import binding as bd
    bd.gdn_chunk_scan(s["desc"], s["pool"], s["cu"], s["slots"], s["v"], s["k"], s["q"], s["dt"], s["beta"], s["A"],
                      s["y"], s["work"], dt_bias=s["dt_bias"], has_initial_state=s["seeded"], ckpt_slots=s["ckpt"],
                      ckpt_interval=s["case"]["interval"])
    return {"y": s["y"], "pool": s["pool"]}


def run_int8(s):
    from recurrent_state_update_gb300 import binding as bd
    for t in range(s["case"]["steps"]):
        bd.gdn_state_update_int8(s["desc"], s["store"], s["entries"], s["xbc"][t], s["dt"][t], s["beta"][t], s["A"],
                                 s["y"][t], dt_bias=s["dt_bias"])
    bd.mamba_ckpt_load_int8(s["desc"], s["pool"], s["entries"], s["back"], s["store"])
    return {"y": s["y"], "pool": s["pool"]}


# ---- the plain forms ----

def unit(x):
    return x / torch.sqrt((x * x).sum(dim=-1, keepdim=True) + EPS)


def gates(s, dt, beta):
    x = dt.float() + s["dt_bias"]
    return torch.where(x > 20, x, torch.log1p(torch.exp(x))) * s["A"], 1 / (1 + torch.exp(-beta.float()))


def split(case, xbc):
    """v, k, q of the conv's channels (..., conv_dim), in 32 bits, k and q of unit length and one a head."""
    H, G, P, N = case["heads"], case["groups"], case["p"], case["n"]
    x = xbc.float()
    v, k, q = x[..., : H * P], x[..., H * P: H * P + G * N], x[..., H * P + G * N:]
    k, q = (unit(t.reshape(*t.shape[:-1], G, N)).repeat_interleave(H // G, dim=-2) for t in (k, q))
    return v.reshape(*v.shape[:-1], H, P), k, q


def token(S, v, k, q, g, b):
    """One token of the recurrence on states S (..., P, N): the new states and the outputs."""
    S = S * torch.exp(g)[..., None, None]
    u = b[..., None] * (v - (S * k[..., None, :]).sum(dim=-1))
    S = S + u[..., None] * k[..., None, :]
    return S, (S * q[..., None, :]).sum(dim=-1) * k.shape[-1] ** -0.5


def plain_step(s):
    case, live = s["case"], s["live"]
    v, k, q = split(case, s["xbc"][live])
    g, b = gates(s, s["dt"][live], s["beta"][live])
    S, ys = s["pool"][s["live_slots"]].float(), []
    for t in range(case["ntok"]):
        S, y = token(S, v[:, t], k[:, t], q[:, t], g[:, t], b[:, t])
        ys.append(y)
        if case["draft"]:
            s["pool"][s["live_scratch"][:, t]] = S.to(s["pool"].dtype)
    if not case["draft"]:
        s["pool"][s["live_slots"]] = S.to(s["pool"].dtype)
    s["y"][live] = torch.stack(ys, dim=1).flatten(2).to(s["y"].dtype)
    return {"y": s["y"], "pool": s["pool"]}


def plain_int8(s):
    case, ids = s["case"], s["ids"]
    for t in range(case["steps"]):
        v, k, q = split(case, s["xbc"][t, :, 0])
        g, b = gates(s, s["dt"][t, :, 0], s["beta"][t, :, 0])
        S, y = token(s["codes"][ids].float() * s["scales"][ids][:, :, None], v, k, q, g, b)
        s["y"][t, :, 0] = y.flatten(1).to(s["y"].dtype)
        top = S.abs().amax(dim=2)
        s["scales"][ids] = top / 127
        s["codes"][ids] = torch.round(S * torch.where(top > 0, 127 / top, 0)[:, :, None]).clamp(-127, 127).to(torch.int8)
    s["pool"][s["back64"]] = (s["codes"][ids].float() * s["scales"][ids][:, :, None]).to(s["pool"].dtype)
    return {"y": s["y"], "pool": s["pool"]}


def plain_scan(s):
    """Chunks of 64 tokens: with c the running sum of the log decays within a chunk and U the values u,
    (I + L) U = b (V - e^c K S^T), L_ij = b_i (k_i . k_j) e^(c_i - c_j) below the diagonal."""
    case, place, nc = s["case"], s["place"], s["nc"]
    H, G, N, nseq = case["heads"], case["groups"], case["n"], case["nseq"]

    def chunks(x):  # (T, heads, ...) -> (sequence, head, chunk, token, ...), zeros past a sequence's end
        x = torch.cat([x, torch.zeros_like(x[:1])])[place]
        return x.movedim(3, 1)

    v = chunks(s["v"].float())
    k, q = (chunks(unit(s[n].float())).repeat_interleave(H // G, dim=1) for n in ("k", "q"))
    g, b = (chunks(t) for t in gates(s, s["dt"], s["beta"]))
    c = torch.cumsum(g, dim=-1)
    i = torch.arange(CHUNK, device=c.device)
    below = i[:, None] >= i
    decay = torch.exp(torch.where(below, c[..., :, None] - c[..., None, :], -math.inf))
    L = b[..., None] * (k @ k.transpose(-1, -2)) * torch.where(i[:, None] > i, decay, 0)
    inv = torch.eye(CHUNK, device=c.device).expand_as(L).contiguous()
    for r in range(1, CHUNK):
        inv[..., r, :] -= (L[..., r, None, :r] @ inv[..., :r, :])[..., 0, :]
    w = inv @ ((b * torch.exp(c))[..., None] * k)
    u0 = inv @ (b[..., None] * v)
    pairs = (q @ k.transpose(-1, -2)) * decay
    qc = q * torch.exp(c)[..., None]
    last = c[..., -1:]
    kc = (k * torch.exp(last - c)[..., None]).transpose(-1, -2)
    S = s["pool"][s["slots64"]].float().transpose(-1, -2)
    S = S if case["seeded"] else torch.zeros_like(S)
    ys = []
    for j in range(nc):
        u = u0[:, :, j] - w[:, :, j] @ S
        ys.append(qc[:, :, j] @ S + pairs[:, :, j] @ u)
        S = torch.exp(last[:, :, j])[..., None] * S + kc[:, :, j] @ u
        if j in s["saves"]:
            rows, slots = s["saves"][j]
            s["pool"][slots] = S[rows].transpose(-1, -2).to(s["pool"].dtype)
    s["pool"][s["slots64"]] = S.transpose(-1, -2).to(s["pool"].dtype)
    y = torch.stack(ys, dim=2).permute(0, 2, 3, 1, 4).flatten(0, 2)  # by sequence, chunk and token
    s["y"].copy_(y[s["token"]] * N ** -0.5)
    return {"y": s["y"], "pool": s["pool"]}


# ---- what a pass cannot do without ----

def work(case):
    H, G, P, N = case["heads"], case["groups"], case["p"], case["n"]
    ab, state = BYTES[case["act"]], H * P * N
    token_bytes = ab * (2 * H * P + 2 * G * N) + 8 * H  # v, y, k, q; dt and beta in 32 bits
    if case["op"] == "scan":
        lens = lengths_of(case)
        kept = sum(x // case["interval"] for x in lens) if case["interval"] else 0
        states = case["nseq"] * (2 if case["seeded"] else 1) + kept
        return {"bytes": case["tokens"] * token_bytes + states * state * BYTES[case["state"]], "flops": 6 * state * case["tokens"]}
    if case["op"] == "int8":
        rows = case["batch"]
        entry = state + 4 * H * N
        return {"bytes": rows * (case["steps"] * (token_bytes + 2 * entry) + entry + state * BYTES[case["state"]]),
                "flops": 6 * state * rows * case["steps"]}
    rows = case["batch"] - case["pad"]
    moved = 1 + (case["ntok"] if case["draft"] else 1)
    return {"bytes": rows * (case["ntok"] * token_bytes + moved * state * BYTES[case["state"]]), "flops": 6 * state * rows * case["ntok"]}


# ---- the recurrence in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    H, G, P, N = case["heads"], case["groups"], case["p"], case["n"]
    rep = H // G

    def norm64(x):
        x = x.to(d)
        return (x / torch.linalg.vector_norm(torch.cat([x, torch.full_like(x[..., :1], math.sqrt(EPS))], -1), dim=-1, keepdim=True)
                ).repeat_interleave(rep, dim=-2)

    def update(S, v, k, q, dt, beta):
        a = torch.exp(torch.nn.functional.softplus(dt.to(d) + s["dt_bias"].to(d), threshold=50.0) * s["A"].to(d))
        S = S * a[..., None, None]
        u = torch.sigmoid(beta.to(d))[..., None] * (v.to(d) - torch.matmul(S, k[..., None])[..., 0])
        S = torch.addcmul(S, u[..., :, None], k[..., None, :])
        return S, torch.matmul(S, q[..., None])[..., 0] / math.sqrt(N)

    if case["op"] == "scan":
        lens = lengths_of(case)
        pool, y = s["pool"].to(d), torch.zeros(case["tokens"], H, P, dtype=d, device="cuda")
        order = sorted(range(case["nseq"]), key=lambda i: -lens[i])  # longest first: those alive are the first rows
        start = s["cu"].cpu().tolist()
        first = torch.tensor([start[i] for i in order], device="cuda")
        slot = s["slots"].cpu().tolist()
        S = pool[[slot[i] for i in order]] * (1.0 if case["seeded"] else 0.0)
        ckpt = s["ckpt"].cpu().tolist() if case["interval"] else None
        k, q = norm64(s["k"]), norm64(s["q"])
        for t in range(max(lens)):
            m = sum(x > t for x in lens)
            at = first[:m] + t
            S[:m], o = update(S[:m], s["v"][at], k[at], q[at], s["dt"][at], s["beta"][at])
            y[at] = o
            if ckpt and (t + 1) % case["interval"] == 0:
                for r in range(m):
                    pool[ckpt[order[r]][(t + 1) // case["interval"] - 1]] = S[r]
        for r, i in enumerate(order):
            pool[slot[i]] = S[r]
        return {"y": y, "pool": pool}
    H_P = H * P
    x, y = s["xbc"], torch.zeros(s["y"].shape, dtype=d, device="cuda")
    if case["op"] == "int8":
        codes, scales = s["codes"][s["ids"]].to(d), s["scales"][s["ids"]].to(d)
        for t in range(case["steps"]):
            row = x[t, :, 0]
            kq = [norm64(z.reshape(-1, G, N)) for z in (row[:, H_P: H_P + G * N], row[:, H_P + G * N:])]
            S, o = update(codes * scales[:, :, None, :], row[:, :H_P].reshape(-1, H, P), *kq, s["dt"][t, :, 0], s["beta"][t, :, 0])
            y[t, :, 0] = o.reshape(-1, H_P)
            scales = S.abs().max(dim=2).values / 127
            codes = torch.round(S / scales[:, :, None, :])
        pool = s["pool"].to(d)
        pool[s["back"].long()] = codes * scales[:, :, None, :]
        return {"y": y, "pool": pool}
    pool, slots = s["pool"].to(d), s["slots"].cpu().tolist()
    for i in range(case["batch"]):
        if slots[i] < 0:
            continue
        S = pool[slots[i]]
        for t in range(case["ntok"]):
            row = x[i, t]
            kq = [norm64(z.reshape(G, N)) for z in (row[H_P: H_P + G * N], row[H_P + G * N:])]
            S, o = update(S, row[:H_P].reshape(H, P), *kq, s["dt"][i, t], s["beta"][i, t])
            y[i, t] = o.reshape(H_P)
            if case["draft"]:
                pool[int(s["scratch"][i, t])] = S
        if not case["draft"]:
            pool[slots[i]] = S
    return {"y": y, "pool": pool}
