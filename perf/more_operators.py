"""Cases of linear attention with a fixed decay for each head, served from a slot pool: the recurrent step with
the norm and rotation of its keys and queries (la_state_update), the chunked scan of a varlen prefill batch
(la_chunk_scan), norm and rotation on their own (la_qk_norm_rope), and the plan of a batch from its requests'
lengths and block table (mamba_batch_plan).

Per head h of a layer with nheads = H, head_dim = P (values), d_state = N (keys), n_groups = G and group
g = h / (H / G), with the state S of shape (P, N):

    k = rotate(k / sqrt(mean(k^2) + eps) * k_weight, position), q the same with q_weight
    S <- exp(log_decay) * S + v k^T,   y = N**-0.5 * S q

run() with ``own`` false is the plain form of each, in 32 bits with elementary torch operations; with ``own``
true it makes the calls a user of the package makes.  exact() evaluates the formulas in 64 bits.
"""
import math
import random

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-6          # of the norms
BASE = 10000.0      # of the rotation's frequencies
CHUNK = 128         # tokens a chunk of the plain scan
FAR = 131072        # positions that decoding reaches


def listed():
    layer = dict(heads=32, groups=32, p=128, n=128, rot=128, inter=False, state="f32", act="bf16")  # generic layer
    wide = dict(layer, heads=128, groups=8, p=64, rot=64, state="bf16")  # heads and groups of the package's Mamba2 layer
    plan = dict(op="plan", block=1024)
    return [
        # one request being answered: the shortest call there is, where latency counts
        dict(layer, name="step one request", op="step", batch=1, pad=0, ntok=1, draft=False),
        # a full decode batch of a busy server, half of the pool's slots in use, states kept in 32 bits
        dict(layer, name="step full batch", op="step", batch=256, pad=0, ntok=1, draft=False),
        # an odd batch with padding rows: many narrow heads over few key groups, half of each key rotated
        dict(wide, name="step odd padded narrow", op="step", batch=61, pad=3, ntok=1, draft=False),
        # speculative decoding: four drafted tokens, the state after each kept in a scratch slot
        dict(layer, name="step four drafts", op="step", batch=48, pad=0, ntok=4, draft=True, state="bf16"),
        # one long prompt: few heads' chains
        dict(layer, name="scan one prompt", op="scan", nseq=1, tokens=8192, seeded=False, interval=0),
        # a prefill batch of ragged prompts with a prefix-cache checkpoint every 1024 tokens
        dict(layer, name="scan ragged batch", op="scan", nseq=8, tokens=32768, seeded=False, interval=1024, state="bf16"),
        # short continuations of stored states: chunks mostly partial
        dict(layer, name="scan short seeded", op="scan", nseq=29, tokens=4001, seeded=True, interval=0),
        # many narrow heads over few key groups
        dict(wide, name="scan narrow heads", op="scan", nseq=4, tokens=8192, seeded=True, interval=0),
        # keys and queries of a small batch
        dict(layer, name="norm and rotation small", op="rope", tokens=61),
        # keys and queries of a prefill batch
        dict(layer, name="norm and rotation prefill", op="rope", tokens=16384),
        # a decode batch: a token a request, some of them passing into a new block
        dict(plan, name="plan decode batch", rows=256, pad=7, tokens=249, long=False),
        # a prefill batch of long prompts, with a column of the block table for each 1024 tokens
        dict(plan, name="plan prefill batch", rows=96, pad=5, tokens=131072, long=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    heads, groups, p, n = rng.choice([(32, 32, 128, 128), (16, 16, 128, 128), (48, 8, 128, 128), (128, 8, 64, 128),
                                      (24, 4, 64, 128), (40, 40, 64, 64), (12, 2, 32, 64)])
    c = dict(heads=heads, groups=groups, p=p, n=n, rot=rng.choice([n, n // 2]), inter=rng.random() < 0.25)
    c["state"], c["act"] = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "bf16"), ("f32", "f32")])
    op = rng.choice(["step", "step", "scan", "scan", "scan", "rope", "plan"])
    work = heads * p * n / (32 * 128 * 128)  # of a token, against the listed layer's
    if op == "step":
        batch = spread(1, 160 / max(1.0, work))
        draft = rng.random() < 0.3
        return dict(c, op=op, batch=batch, pad=rng.randint(0, batch // 8), ntok=rng.randint(2, 6) if draft else 1, draft=draft)
    if op == "scan":
        tokens = spread(1, (2000 if c["act"] == "f32" else 16000) / max(1.0, work))
        return dict(c, op=op, nseq=min(spread(1, 24), tokens), tokens=tokens, seeded=rng.random() < 0.5,
                    interval=rng.choice([0, 128, 512, 1024]) if tokens > 600 else 0)
    if op == "rope":
        return dict(c, op=op, tokens=spread(1, 16000 / max(1.0, work)))
    rows = spread(1, 512)
    pad = rng.randint(0, rows // 8)
    long = rng.random() < 0.5
    return dict(op="plan", rows=rows, pad=pad, tokens=(rows - pad) * (spread(8, 256) if long else 1), long=long,
                block=rng.choice([0, 128, 256, 1024]))


def lengths_of(case):
    """The sequences' lengths: from a third of the mean to as much as closes the sum, the same for a case always."""
    n = case["nseq"] if case["op"] == "scan" else case["rows"] - case["pad"]
    r = random.Random(n * 1000003 + case["tokens"])
    left, out = case["tokens"], []
    for i in range(n, 0, -1):
        mean = left // i
        out.append(left if i == 1 else min(max(1, r.randint((mean + 2) // 3, max(1, 5 * mean // 3))), left - (i - 1)))
        left -= out[-1]
    return out


def sizes(case):
    """(values, keys) of one token's channels v | k | q."""
    return case["heads"] * case["p"], case["groups"] * case["n"]


def prepare(case, seed):
    dev = "cuda"
    if case["op"] == "plan":
        return prepare_plan(case, seed)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    H, G, P, N = case["heads"], case["groups"], case["p"], case["n"]
    HP, GN = sizes(case)
    act, st = DTYPE[case["act"]], DTYPE[case["state"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    # the layer: heads that forget over 1 to 500 tokens, weights of the norms around 1
    s = dict(case=case, log_decay=-torch.exp(-torch.rand(H, generator=gen, device=dev) * math.log(500.0)),
             k_weight=1 + 0.1 * normal(N), q_weight=1 + 0.1 * normal(N),
             inv_freq=(BASE ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])).float().to(dev))
    if own:
        from recurrent_state_update_gb300 import binding as bd
        s["desc"] = layer(bd, case)

    def pool(slots):
        return (0.1 * normal(slots, H, P, N)).to(st)

    if case["op"] == "rope":
        T = case["tokens"]
        row = normal(T, HP + 2 * GN).to(act)  # what the projection leaves: v | k | q
        start = int(torch.randint(0, FAR, (1,), generator=cpu))
        s.update(k=row[:, HP:HP + GN].view(T, G, N), q=row[:, HP + GN:].view(T, G, N),
                 positions=torch.arange(start, start + T, dtype=torch.int32, device=dev),
                 k_out=torch.zeros(T, G, N, dtype=act, device=dev), q_out=torch.zeros(T, G, N, dtype=act, device=dev))
        return s

    if case["op"] == "scan":
        lens = lengths_of(case)
        T, nseq = case["tokens"], case["nseq"]
        # values as the projection leaves them, among its other channels; keys and queries after norm and rotation
        s.update(v=normal(T, HP + 2 * GN).to(act)[:, :HP].view(T, H, P), k=normal(T, G, N).to(act), q=normal(T, G, N).to(act),
                 y=torch.zeros(T, H, P, dtype=act, device=dev))
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
        # the plain form's plan: the token at each place of the padded chunks (T: none), the weights that a chunk's
        # tokens have in its last state, and where states go
        nc = (max(lens) + CHUNK - 1) // CHUNK
        place = torch.full((nseq, nc * CHUNK), T, dtype=torch.int64)
        held = torch.zeros(nseq, nc, dtype=torch.int64)
        for i, x in enumerate(lens):
            place[i, :x] = torch.arange(at[i], at[i + 1])
            held[i] = (x - torch.arange(nc) * CHUNK).clamp(0, CHUNK)
        s.update(place=place.view(nseq, nc, CHUNK).to(dev), held=held.to(dev), slots64=slots.to(dev), nc=nc,
                 token=torch.cat([i * nc * CHUNK + torch.arange(x) for i, x in enumerate(lens)]).to(dev))
        s["saves"] = {}
        for i, n in enumerate(kept):
            for j in range(n):
                s["saves"].setdefault((j + 1) * case["interval"] // CHUNK - 1, []).append((i, int(ckpt[i, j])))
        s["saves"] = {c: tuple(torch.tensor(x, device=dev) for x in zip(*w)) for c, w in s["saves"].items()}
        if own:
            s["work"] = torch.empty(max(16, bd.la_chunk_scan_workspace_bytes(s["desc"], T, nseq)), dtype=torch.uint8, device=dev)
        return s

    batch, ntok = case["batch"], case["ntok"]
    S = 2 * batch + (batch * ntok if case["draft"] else 0)
    ids = torch.randperm(S, generator=cpu)
    slots = ids[:batch].clone()
    slots[torch.randperm(batch, generator=cpu)[: case["pad"]]] = -1
    live = (slots >= 0).nonzero()[:, 0]
    pos = torch.randint(0, FAR, (batch, 1), generator=cpu) + torch.arange(ntok)
    s.update(xbc=normal(batch, ntok, HP + 2 * GN).to(act), y=torch.zeros(batch, ntok, HP, dtype=act, device=dev),
             positions=pos.to(torch.int32).to(dev), pool=pool(S), slots=slots.to(torch.int32).to(dev), live=live.to(dev),
             live_slots=slots[live].to(dev))
    if case["draft"]:
        s["scratch"] = ids[batch:batch + batch * ntok].view(batch, ntok).to(torch.int32).to(dev)
        s["live_scratch"] = s["scratch"].long()[s["live"]]
    return s


def prepare_plan(case, seed):
    r = random.Random(seed)
    rows, block = case["rows"], case["block"]
    lens = lengths_of(case)
    # prompts are new or go on from a block's border; decoding requests are anywhere
    computed = [block * r.randint(0, 8) if case["long"] else r.randint(0, 8 * (block or 1024)) for _ in lens]
    order = r.sample(range(rows), rows - case["pad"])
    new, past = [0] * rows, [0] * rows
    for i, n, c in zip(order, lens, computed):
        new[i], past[i] = n, c
    cols = 1 + (8 * block + max(lens)) // block if block else 1
    slots = rows * cols + 1
    ids = list(range(slots))
    r.shuffle(ids)

    def dev(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def out(*shape):
        return torch.zeros(*shape, dtype=torch.int32, device="cuda")

    total = case["tokens"]
    return dict(case=case, new=dev(new), past=dev(past), table=dev(ids[:rows * cols]).view(rows, cols), slots_total=slots,
                cu=out(rows + 1), positions=out(total), token_rows=out(total), slots=out(rows), copy_src=out(rows),
                copy_dst=out(rows), ckpt=out(rows, max(1, cols - 1)),
                seeded=torch.zeros(rows, dtype=torch.uint8, device="cuda"))


def layer(bd, case):
    from recurrent_state_update_gb300 import workloads as wl
    shape = wl.LayerShape(nheads=case["heads"], head_dim=case["p"], d_state=case["n"], n_groups=case["groups"])
    return bd.layer_desc(shape, state=case["state"], act=case["act"], dt="f32")


def run(s):
    op = s["case"]["op"]
    if own:
        return {"step": run_step, "scan": run_scan, "rope": run_rope, "plan": run_plan}[op](s)
    return {"step": plain_step, "scan": plain_scan, "rope": plain_rope, "plan": plain_plan}[op](s)


def run_step(s):
    from recurrent_state_update_gb300 import binding as bd
    bd.la_state_update(s["desc"], s["pool"], s["slots"], s["xbc"], s["log_decay"], s["y"], scratch_slots=s.get("scratch"),
                       qk_norm=True, k_weight=s["k_weight"], q_weight=s["q_weight"], eps=EPS, positions=s["positions"],
                       inv_freq=s["inv_freq"], interleaved=s["case"]["inter"])
    return {"y": s["y"], "pool": s["pool"]}


def run_scan(s):
    from recurrent_state_update_gb300 import binding as bd
    bd.la_chunk_scan(s["desc"], s["pool"], s["cu"], s["slots"], s["v"], s["k"], s["q"], s["log_decay"], s["y"], s["work"],
                     has_initial_state=s["seeded"], ckpt_slots=s["ckpt"], ckpt_interval=s["case"]["interval"])
    return {"y": s["y"], "pool": s["pool"]}


def run_rope(s):
    from recurrent_state_update_gb300 import binding as bd
    bd.la_qk_norm_rope(s["desc"], s["k"], s["q"], s["k_out"], s["q_out"], qk_norm=True, k_weight=s["k_weight"],
                       q_weight=s["q_weight"], eps=EPS, positions=s["positions"], inv_freq=s["inv_freq"],
                       interleaved=s["case"]["inter"])
    return {"k": s["k_out"], "q": s["q_out"]}


PLAN_OUT = ("cu", "positions", "token_rows", "slots", "seeded", "copy_src", "copy_dst", "ckpt")


def run_plan(s):
    from recurrent_state_update_gb300 import binding as bd
    bd.mamba_batch_plan(s["new"], s["past"], s["table"], s["case"]["block"], s["slots_total"], cu_seqlens=s["cu"],
                        slot_ids=s["slots"], has_initial_state=s["seeded"], copy_src=s["copy_src"], copy_dst=s["copy_dst"],
                        ckpt_slots=s["ckpt"], positions=s["positions"], token_rows=s["token_rows"])
    return {n: s[n] for n in PLAN_OUT}


# ---- the plain forms ----

def norm_rotate(s, x, weight, positions):
    """Keys or queries (..., heads, N) at positions (...), in 32 bits; the angles in 64."""
    case = s["case"]
    x = x.float()
    x = x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight
    R = case["rot"]
    angle = positions.double()[..., None] * s["inv_freq"].double()
    cos, sin = (f(angle).float()[..., None, :] for f in (torch.cos, torch.sin))
    turned = x[..., :R]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if case["inter"] else (turned[..., :R // 2], turned[..., R // 2:])
    pair = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(pair, dim=-1).flatten(-2) if case["inter"] else torch.cat(pair, dim=-1)
    return torch.cat([turned, x[..., R:]], dim=-1)


def plain_rope(s):
    s["k_out"].copy_(norm_rotate(s, s["k"], s["k_weight"], s["positions"]))
    s["q_out"].copy_(norm_rotate(s, s["q"], s["q_weight"], s["positions"]))
    return {"k": s["k_out"], "q": s["q_out"]}


def plain_step(s):
    case, live = s["case"], s["live"]
    H, G, P, N = case["heads"], case["groups"], case["p"], case["n"]
    HP, GN = sizes(case)
    x, pos = s["xbc"][live], s["positions"][live]
    lead = x.shape[:2]
    v = x[..., :HP].float().reshape(*lead, H, P)
    k = norm_rotate(s, x[..., HP:HP + GN].reshape(*lead, G, N), s["k_weight"], pos).repeat_interleave(H // G, dim=2)
    q = norm_rotate(s, x[..., HP + GN:].reshape(*lead, G, N), s["q_weight"], pos).repeat_interleave(H // G, dim=2)
    decay = torch.exp(s["log_decay"])[:, None, None]
    S, ys = s["pool"][s["live_slots"]].float(), []
    for t in range(case["ntok"]):
        S = S * decay + v[:, t, :, :, None] * k[:, t, :, None, :]
        ys.append((S * q[:, t, :, None, :]).sum(dim=-1) * N ** -0.5)
        if case["draft"]:
            s["pool"][s["live_scratch"][:, t]] = S.to(s["pool"].dtype)
    if not case["draft"]:
        s["pool"][s["live_slots"]] = S.to(s["pool"].dtype)
    s["y"][live] = torch.stack(ys, dim=1).flatten(2).to(s["y"].dtype)
    return {"y": s["y"], "pool": s["pool"]}


def plain_scan(s):
    """Chunks of 128 tokens: y_i = d^(i+1) S q_i + sum_(j <= i) d^(i-j) (q_i . k_j) v_j, and S takes d^(L-1-j) v_j k_j^T
    of each of a chunk's L tokens, d = exp(log_decay)."""
    case, place, nc, g = s["case"], s["place"], s["nc"], s["log_decay"]
    H, G, N = case["heads"], case["groups"], case["n"]

    def chunks(x):  # (T, heads, ...) -> (sequence, head, chunk, token, ...), zeros past a sequence's end
        x = torch.cat([x, torch.zeros_like(x[:1])])[place]
        return x.movedim(3, 1)

    v = chunks(s["v"].float())
    k, q = (chunks(s[n].float()).repeat_interleave(H // G, dim=1) for n in ("k", "q"))
    i = torch.arange(CHUNK, device=g.device)
    gap = torch.where(i[:, None] >= i, (i[:, None] - i).float(), math.inf)
    decay = torch.where(gap < math.inf, torch.exp(torch.where(gap < math.inf, gap, 0.0) * g[:, None, None]), 0.0)
    intra = ((q @ k.transpose(-1, -2)) * decay[:, None]) @ v
    left = (s["held"][:, None, :, None] - 1 - i).float()  # (sequence, 1, chunk, token): tokens after this one in its chunk
    kc = k * torch.where(left >= 0, torch.exp(left.clamp(min=0) * g[:, None, None]), 0.0)[..., None]
    add = v.transpose(-1, -2) @ kc
    over = torch.exp(s["held"].float()[:, None] * g[:, None])[..., None, None]  # (sequence, head, chunk, 1, 1)
    qc = q * torch.exp((i + 1).float() * g[:, None])[:, None, :, None]
    S = s["pool"][s["slots64"]].float()
    S = S if case["seeded"] else torch.zeros_like(S)
    ys = []
    for j in range(nc):
        ys.append(intra[:, :, j] + qc[:, :, j] @ S.transpose(-1, -2))
        S = over[:, :, j] * S + add[:, :, j]
        if j in s["saves"]:
            rows, slots = s["saves"][j]
            s["pool"][slots] = S[rows].to(s["pool"].dtype)
    s["pool"][s["slots64"]] = S.to(s["pool"].dtype)
    y = torch.stack(ys, dim=2).permute(0, 2, 3, 1, 4).flatten(0, 2)  # by sequence, chunk and token
    s["y"].copy_(y[s["token"]] * N ** -0.5)
    return {"y": s["y"], "pool": s["pool"]}


def plain_plan(s):
    case, new, past = s["case"], s["new"].long(), s["past"].long()
    rows, block, total = case["rows"], case["block"], case["tokens"]
    dev = new.device
    s["cu"][0] = 0
    s["cu"][1:] = torch.cumsum(new, 0)
    t = torch.arange(total, device=dev)
    row = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    s["token_rows"].copy_(row)
    s["positions"].copy_(past[row] + t - s["cu"].long()[row])
    live, seeded = new > 0, (new > 0) & (past > 0)
    size = block if block else 1 << 62
    first, last = (past - 1).clamp(min=0) // size, (past + new - 1).clamp(min=0) // size
    src, dst = (s["table"].gather(1, c[:, None])[:, 0] for c in (first, last))
    s["slots"].copy_(torch.where(live, dst, -1))
    s["seeded"].copy_(seeded)
    moves = seeded & (src != dst)
    s["copy_src"].copy_(torch.where(moves, src, -1))
    s["copy_dst"].copy_(torch.where(moves, dst, -1))
    if block:
        n = torch.arange(1, s["ckpt"].shape[1] + 1, device=dev)
        column = past[:, None] // block + n - 1
        due = live[:, None] & (past % block == 0)[:, None] & (n * block < new[:, None])
        page = s["table"].gather(1, column.clamp(max=s["table"].shape[1] - 1))
        s["ckpt"].copy_(torch.where(due, page, -1))
    else:
        s["ckpt"].fill_(-1)
    return {n: s[n] for n in PLAN_OUT}


# ---- what a pass cannot do without ----

def work(case):
    if case["op"] == "plan":
        rows, block = case["rows"], case["block"]
        kept = case["tokens"] // block if block else 0
        cols = max(1, (8 * block + max(lengths_of(case))) // block) if block else 1
        return {"bytes": 4 * (2 * rows + 2 * rows + kept) + 4 * (rows + 1 + 2 * case["tokens"] + 3 * rows + rows * cols) + rows,
                "flops": 2 * case["tokens"] + 8 * rows}
    H, P, N = case["heads"], case["p"], case["n"]
    HP, GN = sizes(case)
    ab, sb, state = BYTES[case["act"]], BYTES[case["state"]], H * P * N
    if case["op"] == "rope":
        return {"bytes": case["tokens"] * (4 * GN * ab + 4) + 8 * N + 2 * case["rot"], "flops": 20 * GN * case["tokens"]}
    token_bytes = ab * (2 * HP + 2 * GN)
    if case["op"] == "scan":
        lens = lengths_of(case)
        kept = sum(x // case["interval"] for x in lens) if case["interval"] else 0
        states = case["nseq"] * (2 if case["seeded"] else 1) + kept
        return {"bytes": case["tokens"] * token_bytes + states * state * sb, "flops": 4 * state * case["tokens"]}
    rows = case["batch"] - case["pad"]
    moved = 1 + (case["ntok"] if case["draft"] else 1)
    return {"bytes": rows * (case["ntok"] * token_bytes + moved * state * sb), "flops": 5 * state * rows * case["ntok"]}


# ---- the formulas in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return exact_plan(s)
    d = torch.float64
    H, G, P, N = case["heads"], case["groups"], case["p"], case["n"]
    HP, GN = sizes(case)
    R = case["rot"]

    def turn(x, weight, pos):
        """Each pair as one complex number, turned by its angle."""
        x = x.to(d)
        x = x * torch.rsqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True).square() / N + EPS) * weight.to(d)
        head = x[..., :R].unflatten(-1, (R // 2, 2) if case["inter"] else (2, R // 2))
        z = torch.complex(head[..., 0], head[..., 1]) if case["inter"] else torch.complex(head[..., 0, :], head[..., 1, :])
        phase = torch.outer(pos.reshape(-1).to(d), s["inv_freq"].to(d)).reshape(*pos.shape, 1, R // 2)
        z = z * torch.polar(torch.ones_like(phase), phase)
        out = x.clone()
        if case["inter"]:
            out[..., 0:R:2], out[..., 1:R:2] = z.real, z.imag
        else:
            out[..., :R // 2], out[..., R // 2:R] = z.real, z.imag
        return out

    if case["op"] == "rope":
        return {"k": turn(s["k"], s["k_weight"], s["positions"]), "q": turn(s["q"], s["q_weight"], s["positions"])}
    decay = torch.exp(s["log_decay"].to(d))[:, None, None]
    rep = H // G

    def token(S, v, k, q):
        S = torch.addcmul(S * decay, v.to(d)[..., :, None], k.repeat_interleave(rep, dim=-2)[..., None, :])
        return S, torch.matmul(S, q.repeat_interleave(rep, dim=-2)[..., None])[..., 0] / math.sqrt(N)

    pool = s["pool"].to(d)
    if case["op"] == "scan":
        lens = lengths_of(case)
        y = torch.zeros(case["tokens"], H, P, dtype=d, device="cuda")
        order = sorted(range(case["nseq"]), key=lambda i: -lens[i])  # longest first: those alive are the first rows
        start = s["cu"].cpu().tolist()
        first = torch.tensor([start[i] for i in order], device="cuda")
        slot = s["slots"].cpu().tolist()
        S = pool[[slot[i] for i in order]] * (1.0 if case["seeded"] else 0.0)
        ckpt = s["ckpt"].cpu().tolist() if case["interval"] else None
        k, q = s["k"].to(d), s["q"].to(d)
        for t in range(max(lens)):
            m = sum(x > t for x in lens)
            at = first[:m] + t
            S[:m], y[at] = token(S[:m], s["v"][at], k[at], q[at])
            if ckpt and (t + 1) % case["interval"] == 0:
                for r in range(m):
                    pool[ckpt[order[r]][(t + 1) // case["interval"] - 1]] = S[r]
        for r, i in enumerate(order):
            pool[slot[i]] = S[r]
        return {"y": y, "pool": pool}
    slots, y = s["slots"].cpu().tolist(), torch.zeros(s["y"].shape, dtype=d, device="cuda")
    for i in range(case["batch"]):
        if slots[i] < 0:
            continue
        S, x, pos = pool[slots[i]], s["xbc"][i], s["positions"][i]
        k = turn(x[:, HP:HP + GN].reshape(-1, G, N), s["k_weight"], pos)
        q = turn(x[:, HP + GN:].reshape(-1, G, N), s["q_weight"], pos)
        for t in range(case["ntok"]):
            S, o = token(S, x[t, :HP].reshape(H, P), k[t], q[t])
            y[i, t] = o.reshape(HP)
            if case["draft"]:
                pool[int(s["scratch"][i, t])] = S
        if not case["draft"]:
            pool[slots[i]] = S
    return {"y": y, "pool": pool}


def exact_plan(s):
    case = s["case"]
    block, new, past, table = case["block"], s["new"].tolist(), s["past"].tolist(), s["table"].tolist()
    o = dict(cu=[0], positions=[], token_rows=[], slots=[], seeded=[], copy_src=[], copy_dst=[], ckpt=[])
    for i, (n, c) in enumerate(zip(new, past)):
        o["cu"].append(o["cu"][-1] + n)
        o["positions"] += range(c, c + n)
        o["token_rows"] += [i] * n
        page = [table[i][(t - 1) // block if block else 0] if t else -1 for t in (c, c + n)]
        o["slots"].append(page[1] if n else -1)
        o["seeded"].append(int(n > 0 and c > 0))
        moved = n > 0 and c > 0 and page[0] != page[1]
        o["copy_src"].append(page[0] if moved else -1)
        o["copy_dst"].append(page[1] if moved else -1)
        row = [-1] * s["ckpt"].shape[1]
        if block and n and c % block == 0:
            for j in range(1, (n - 1) // block + 1):
                row[j - 1] = table[i][c // block + j - 1]
        o["ckpt"].append(row)
    return {n: torch.tensor(o[n], dtype=s[n].dtype, device="cuda") for n in PLAN_OUT}
