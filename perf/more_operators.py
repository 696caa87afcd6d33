"""Cases, plain forms and exact values of the recurrent layers' gated delta
rule and of the slots that a step's new tokens take in the paged cache.

    decode   the gated delta rule for one to a few rows a sequence, the state
             after each row kept: bf16 outputs and fp32 states
    prefill  the same rule over ragged prompts, from the sequences' states to
             their new ones
    assign   pages from the free stack for each request's new tokens: block
             table, lengths, first rows, positions and cache slots
    append   the new tokens' latents and index keys into those slots (8 bits)

The rule, for a state S [128 values][128 keys] of one head and row t:
    S~ = S diag(exp(gate_t)),  u = beta_t (v_t - S~ k_t)
    S  = S~ + u k_t^T,         out_t = scale S q_t

`run` computes them in elementary torch operations where `own` is false and
through the package's entry points where it is true.
"""
import math

import torch

own = False

DIM, BLOCK, LATENT, KEY = 128, 64, 576, 128
SCALE = 1.0 / math.sqrt(DIM)
CHUNK = 16   # rows that the plain form takes at once


def listed():
    return [
        # one conversation's next token in a layer of 32 heads: latency
        {"name": "decode_one", "op": "decode", "batch": 1, "nq": 1, "heads": 32, "qk_heads": 32, "gate": "channel"},
        # a decode batch: a layer's states read and written once
        {"name": "decode_batch", "op": "decode", "batch": 32, "nq": 1, "heads": 96, "qk_heads": 96, "gate": "channel"},
        # speculative verify: the state after each of four draft rows is kept, the accepted one goes on
        {"name": "decode_drafts", "op": "decode", "batch": 8, "nq": 4, "heads": 96, "qk_heads": 96, "gate": "channel"},
        # shared query and key heads, one decay a head, an odd batch
        {"name": "decode_shared", "op": "decode", "batch": 101, "nq": 2, "heads": 33, "qk_heads": 11, "gate": "head"},
        # three short prompts; shared query and key heads, one decay a head
        {"name": "prefill_short", "op": "prefill", "lens": "3:5:71", "heads": 33, "qk_heads": 11, "gate": "head"},
        # ragged prompts that share a step
        {"name": "prefill_ragged", "op": "prefill", "lens": "7:1:1501", "heads": 96, "qk_heads": 96, "gate": "channel"},
        # one chunk of a long prompt, behind the state of those before it
        {"name": "prefill_chunk", "op": "prefill", "lens": "2048", "heads": 96, "qk_heads": 96, "gate": "channel"},
        # a long prompt in one call
        {"name": "prefill_long", "op": "prefill", "lens": "16385", "heads": 96, "qk_heads": 96, "gate": "channel"},
        # a decode step's slots: a new token for each of 64 contexts
        {"name": "assign_step", "op": "assign", "batch": 64, "cached": 160000, "new": 1},
        # a step that mixes prompts, chunks and single tokens of many requests
        {"name": "assign_mixed", "op": "assign", "batch": 2048, "cached": 8192, "new": 257},
        # the new tokens of a decode step into their slots
        {"name": "append_step", "op": "append", "rows": 64},
        # the new tokens of a prefill step into their slots
        {"name": "append_prefill", "op": "append", "rows": 16385},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["decode", "decode", "prefill", "prefill", "assign", "append"])
    if op == "assign":
        return {"op": op, "batch": log_int(1, 4096), "cached": log_int(1, 100000), "new": log_int(1, 300)}
    if op == "append":
        return {"op": op, "rows": log_int(1, 16000)}
    qk = log_int(1, 96)
    heads = qk * rng.choice([r for r in (1, 1, 1, 2, 3, 4) if qk * r <= 96])
    case = {"op": op, "heads": heads, "qk_heads": qk, "gate": rng.choice(["channel", "channel", "head"])}
    if op == "decode":
        nq = rng.choice([1, 1, 2, 3, 4, 7])
        case.update(batch=log_int(1, min(256, 12000 // (heads * nq))), nq=nq)
    else:
        top = log_int(1, 8192)
        n = log_int(1, max(1, min(24, 700000 // (top * heads))))
        case["lens"] = f"{n}:{rng.randint(0, top)}:{top}"
    return case


# ---------------------------------------------------------------- inputs
def lengths(case, seed):
    """"n:lo:hi": n lengths in [lo, hi], spread evenly and shuffled by the seed; "a" alone: one sequence."""
    p = [int(x) for x in case["lens"].split(":")]
    if len(p) == 1:
        return p
    n, lo, hi = p
    if n == 1:
        return [hi]
    g = torch.Generator().manual_seed(seed + 17)
    return [lo + (hi - lo) * i // (n - 1) for i in torch.randperm(n, generator=g).tolist()]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "assign":
        st = prepare_assign(case, g)
    elif case["op"] == "append":
        st = prepare_append(case, g)
    else:
        st = prepare_delta(case, seed, g)
    st["op"] = case["op"]
    if own:
        from dsa_sparse_attention_index_gb300 import binding

        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] in ("decode", "prefill"):
            st["pool"] = binding.StatePool(st["states"])
            st["x"] = binding.DeltaRows(st["q"], st["k"], st["v"], st["gate"], st["beta"], SCALE)
        if case["op"] == "prefill":
            st["ws"] = binding.workspace(binding.gated_delta_prefill_workspace_size(
                st["q"].shape[0], len(st["lens"]), case["heads"]))
        if case["op"] == "append":
            st["cache"] = binding.PagedCache(st["kv"], st["kv"].shape[1], 0, BLOCK * LATENT, binding.KEY_FP8_E4M3,
                                             st["latent_scale"])
    return st


def prepare_delta(case, seed, g):
    dev, heads, qk = "cuda", case["heads"], case["qk_heads"]
    if case["op"] == "decode":
        lens, kept = [case["nq"]] * case["batch"], case["nq"]
    else:
        lens, kept = lengths(case, seed), 1
    batch, rows = len(lens), sum(lens)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # queries and keys of length one beside the values in the projections' buffer, so rows lie apart
    width = (2 * qk + heads) * DIM
    qkv = torch.empty((rows, width), dtype=torch.bfloat16, device=dev)
    step = max(1, (1 << 27) // width)
    for i in range(0, rows, step):
        x = randn(min(step, rows - i), 2 * qk + heads, DIM)
        x[:, :2 * qk] /= x[:, :2 * qk].norm(dim=2, keepdim=True)
        qkv[i:i + step] = x.view(-1, width).to(torch.bfloat16)
    q, k, v = (t.unflatten(1, (-1, DIM)) for t in qkv.split((qk * DIM, qk * DIM, heads * DIM), 1))
    # decays from slow (0.999 a row) to fast (0.2 a row), by head and channel; softplus of the token's own part
    rate = torch.exp(torch.empty((heads, DIM), device=dev).uniform_(math.log(1e-3), math.log(1.5), generator=g))
    if case["gate"] == "head":
        gate = -rate[:, 0] * torch.nn.functional.softplus(randn(rows, heads))
    else:
        gate = torch.empty((rows, heads, DIM), device=dev)
        for i in range(0, rows, step):
            n = min(step, rows - i)
            gate[i:i + n] = -rate * torch.nn.functional.softplus(randn(n, heads, DIM))
    beta = torch.sigmoid(randn(rows, heads))
    # slots 0..batch-1 hold the sequences' states, the kept ones go behind them, either in shuffled order
    states = torch.zeros((batch * (1 + kept), heads, DIM, DIM), device=dev)
    states[:batch] = randn(batch, heads, DIM, DIM) * 0.3
    slots_in = torch.randperm(batch, generator=g, device=dev).to(torch.int32)
    if case["op"] == "prefill" and batch > 1:
        slots_in[::2] = -1   # new requests start from nothing
    slots_out = batch + torch.randperm(batch * kept, generator=g, device=dev).to(torch.int32)
    if case["op"] == "decode":
        slots_out = slots_out.view(batch, kept)
    starts = torch.tensor([sum(lens[:b]) for b in range(batch + 1)], dtype=torch.int32, device=dev)
    return {"lens": lens, "q": q, "k": k, "v": v, "gate": gate, "beta": beta, "states": states, "slots_in": slots_in,
            "slots_out": slots_out, "starts": starts, "batch": batch, "nq": case.get("nq"),
            "out": torch.zeros((rows, heads, DIM), dtype=torch.bfloat16, device=dev)}


def new_lengths(case):
    if case["new"] == 1:
        return torch.ones(case["batch"], dtype=torch.int64)
    return (case["new"] + 1) * torch.arange(case["batch"]) // case["batch"]


def prepare_assign(case, g):
    dev, batch = "cuda", case["batch"]
    # every length from none to the largest as often, in another order for each seed
    spread = torch.arange(batch, device=dev)
    cached = (case["cached"] * (spread + 1) // batch)[torch.randperm(batch, generator=g, device=dev)]
    new = new_lengths(case).to(dev)[torch.randperm(batch, generator=g, device=dev)]
    have, need = -(-cached // BLOCK), -(-(cached + new) // BLOCK)
    used, taken, rows = int(have.sum()), int((need - have).sum()), int(new.sum())
    blocks = used + taken + 1000   # a free stack with more pages than the step takes
    perm = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    table = torch.full((batch, -(-(case["cached"] + case["new"]) // BLOCK)), -1, dtype=torch.int32, device=dev)
    at = torch.arange(table.shape[1], device=dev)
    table[at[None] < have[:, None]] = perm[:used]
    free = torch.zeros(blocks, dtype=torch.int32, device=dev)
    free[:blocks - used] = perm[used:]

    def ints(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=dev)

    most = rows + 37   # rows of a buffer that every step uses
    return {"cached": cached.to(torch.int32), "new": new.to(torch.int32), "free": free, "num_blocks": blocks,
            "free_count": torch.tensor([blocks - used], dtype=torch.int32, device=dev), "free_left": ints(1), "table": table,
            "seq_lens": ints(batch), "starts": ints(batch + 1), "positions": ints(most), "slots": ints(most)}


def prepare_append(case, g):
    dev, rows = "cuda", case["rows"]
    blocks = rows // BLOCK + 9
    slots = torch.randperm(blocks * BLOCK, generator=g, device=dev)[:rows].to(torch.int32)
    slots[torch.rand(rows, generator=g, device=dev) < 0.02] = -1   # padding rows
    latent = torch.randn((rows, LATENT), generator=g, device=dev) * torch.rand((rows, 1), generator=g, device=dev).add(0.5)
    key = torch.randn((rows, KEY), generator=g, device=dev)
    scale = 0.01 + 0.02 * float(torch.rand((), generator=g, device=dev))
    return {"slots": slots, "latent": latent.to(torch.bfloat16), "key": key.to(torch.bfloat16), "latent_scale": scale,
            "kv": torch.zeros((blocks, BLOCK * (LATENT + KEY + 4)), dtype=torch.uint8, device=dev)}


# ---------------------------------------------------------------- plain forms
def padded(st, t):
    """Rows [rows, heads, ...] as fp32 [batch, heads, longest, ...], zeros behind a sequence's last row."""
    at = torch.arange(-(-max(st["lens"]) // CHUNK) * CHUNK, device=t.device)
    row = st["starts"][:-1, None] + at
    there = row < st["starts"][1:, None]
    x = t[torch.where(there, row, 0).long()] * there.reshape(there.shape + (1,) * (t.dim() - 1))
    return x.float().transpose(1, 2)


def plain_delta(st):
    heads, batch = st["v"].shape[1], st["batch"]
    out, states = st["out"], st["states"]
    S = states[st["slots_in"].clamp(min=0).long()] * (st["slots_in"] >= 0)[:, None, None, None]
    share = heads // st["q"].shape[1]
    gate = st["gate"] if st["gate"].dim() == 3 else st["gate"][:, :, None].expand(-1, -1, DIM)
    if st["op"] == "decode":
        nq = st["nq"]
        q, k = (st[n].float().repeat_interleave(share, 1).unflatten(0, (batch, nq)) for n in "qk")
        v, decay, beta = (t.unflatten(0, (batch, nq)) for t in (st["v"].float(), torch.exp(gate), st["beta"]))
        for j in range(nq):
            S = S * decay[:, j, :, None, :]
            u = beta[:, j, :, None] * (v[:, j] - (S * k[:, j, :, None, :]).sum(3))
            S = S + u[..., None] * k[:, j, :, None, :]
            out.unflatten(0, (batch, nq))[:, j] = ((S * q[:, j, :, None, :]).sum(3) * SCALE).to(torch.bfloat16)
            states[st["slots_out"][:, j].long()] = S
        return {"out": out, "states": states[batch:]}
    rows = out.shape[0]
    if rows:
        seq = torch.arange(batch, device=out.device).repeat_interleave(torch.diff(st["starts"]), output_size=rows)
        place = torch.arange(rows, device=out.device) - st["starts"].long()[seq]
        q, k = (padded(st, st[n]).repeat_interleave(share, 1) for n in "qk")
        v, gate, beta = padded(st, st["v"]), padded(st, gate), padded(st, st["beta"])
        y = torch.empty_like(v)
        keep = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=out.device).tril()
        eye = torch.eye(CHUNK, device=out.device)
        # a chunk of rows at once: the rows' effect on each other by one small triangular system
        for t in range(0, q.shape[2], CHUNK):
            at = slice(t, t + CHUNK)
            Q, K, V, b = q[:, :, at], k[:, :, at], v[:, :, at], beta[:, :, at, None]
            G = gate[:, :, at].double().cumsum(2)
            # decay from row j (behind it) to row i (with it), by channel
            D = (G[:, :, :, None] - G[:, :, None]).masked_fill(~keep[..., None], -math.inf).exp().float()
            kd = K[:, :, None] * D
            A = b * (K[:, :, :, None] * kd).sum(4).tril(-1)
            B = (Q[:, :, :, None] * kd).sum(4)
            P = G.exp().float()
            R = b * (V - (K * P) @ S.transpose(2, 3))
            # (I + A)^-1 R: A^16 = 0, so the inverse is (I - A)(I + A^2)(I + A^4)(I + A^8)
            A2 = A @ A
            A4 = A2 @ A2
            U = (eye - A) @ ((eye + A2) @ ((eye + A4) @ (R + (A4 @ A4) @ R)))
            y[:, :, at] = (Q * P) @ S.transpose(2, 3) + B @ U
            S = S * P[:, :, -1, None, :] + U.transpose(2, 3) @ (K * D[:, :, -1])
        out[:] = (y[seq, :, place] * SCALE).to(torch.bfloat16)
    states[st["slots_out"].long()] = S
    return {"out": out, "states": states[batch:]}


def plain_assign(st):
    new, table = st["new"].long(), st["table"]
    total = st["cached"].long() + new
    have, need = -(-st["cached"].long() // BLOCK), -(-total // BLOCK)
    st["seq_lens"][:] = total
    st["starts"][1:] = new.cumsum(0)
    before = (need - have).cumsum(0) - (need - have)   # pages taken by the requests before
    at = torch.arange(table.shape[1], device=table.device)
    page = before[:, None] + at - have[:, None]
    fresh = (at >= have[:, None]) & (at < need[:, None])
    count = st["free_count"].long()
    table[:] = torch.where(fresh, st["free"][(count - 1 - page).clamp(min=0)], table)
    st["free_left"][:] = count - (need - have).sum()
    row = torch.arange(st["slots"].shape[0], device=table.device)
    seq = torch.searchsorted(st["starts"].long(), row, right=True) - 1
    there = seq < new.shape[0]
    seq = seq.clamp(max=new.shape[0] - 1)
    pos = st["cached"].long()[seq] + row - st["starts"].long()[seq]
    pos = torch.where(there, pos, 0)
    st["positions"][:] = torch.where(there, pos, -1)
    st["slots"][:] = torch.where(there, table[seq, pos // BLOCK].long() * BLOCK + pos % BLOCK, -1)
    return {n: st[n] for n in ("table", "seq_lens", "starts", "positions", "slots", "free_left")}


def cache_parts(st):
    """The pool's latents and keys as the 8-bit values that they are, and the keys' scales."""
    kv = st["kv"]
    f8 = kv[:, :BLOCK * (LATENT + KEY)].view(torch.float8_e4m3fn)
    return {"latent": f8[:, :BLOCK * LATENT], "key": f8[:, BLOCK * LATENT:],
            "scale": kv[:, BLOCK * (LATENT + KEY):].view(torch.float32)}


def plain_append(st):
    there = st["slots"] >= 0
    slot = st["slots"][there].long()
    block, at = slot // BLOCK, slot % BLOCK
    x, key = st["latent"][there].float() / st["latent_scale"], st["key"][there].float()
    s = key.abs().amax(1, keepdim=True) / 448
    s = torch.where(s == 0, 1.0, s)
    kv = st["kv"]
    to = kv[:, :BLOCK * LATENT].unflatten(1, (BLOCK, LATENT))
    to[block, at] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    to = kv[:, BLOCK * LATENT:BLOCK * (LATENT + KEY)].unflatten(1, (BLOCK, KEY))
    to[block, at] = (key / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    kv[:, BLOCK * (LATENT + KEY):].view(torch.float32)[block, at] = s[:, 0]
    return cache_parts(st)


def run(st):
    if not own:
        return {"decode": plain_delta, "prefill": plain_delta, "assign": plain_assign, "append": plain_append}[st["op"]](st)
    from dsa_sparse_attention_index_gb300 import binding

    if st["op"] == "decode":
        binding.gated_delta_decode(st["pool"], st["x"], st["nq"], st["slots_in"], st["slots_out"], st["out"], st["status"])
        return {"out": st["out"], "states": st["states"][st["batch"]:]}
    if st["op"] == "prefill":
        binding.gated_delta_prefill(st["pool"], st["x"], st["starts"], st["slots_in"], st["slots_out"], st["out"], st["ws"],
                                    st["status"])
        return {"out": st["out"], "states": st["states"][st["batch"]:]}
    if st["op"] == "assign":
        binding.assign_slots(st["cached"], st["new"], st["free"], st["free_count"], st["num_blocks"], st["table"],
                             st["seq_lens"], st["starts"], st["positions"], st["slots"], st["free_left"], st["status"])
        return {n: st[n] for n in ("table", "seq_lens", "starts", "positions", "slots", "free_left")}
    binding.cache_append_slots(st["cache"], st["slots"], st["latent"], st["key"], st["status"])
    return cache_parts(st)


# ---------------------------------------------------------------- work and exact values
def work(case):
    if case["op"] == "append":
        return {"bytes": case["rows"] * (4 + 3 * (LATENT + KEY) + 4), "flops": 0}
    if case["op"] == "assign":
        # lengths read, lengths and first rows written, a page off the stack and into the table, two numbers a row
        rows = int(new_lengths(case).sum())
        return {"bytes": 16 * case["batch"] + 8 * rows / BLOCK + 8 * rows, "flops": 0}
    heads, qk = case["heads"], case["qk_heads"]
    lens = [case["nq"]] * case["batch"] if case["op"] == "decode" else lengths(case, 0)
    rows, batch = sum(lens), len(lens)
    gate = 4 * (DIM if case["gate"] == "channel" else 1)
    row = 2 * 2 * qk * DIM + heads * (2 * 2 * DIM + gate + 4)
    if case["op"] == "decode":
        states = batch * (1 + case["nq"])
    else:
        states = batch + (batch // 2 if batch > 1 else 1)
    # the decay, two products with the state and its update
    return {"bytes": rows * row + states * heads * 4 * DIM * DIM, "flops": 7 * rows * heads * DIM * DIM}


def exact(case, seed):
    if case["op"] == "assign":
        return None   # whole numbers only
    st = prepare(case, seed)
    if case["op"] == "append":
        blocks = st["kv"].shape[0]
        latent, key, scale = (torch.zeros((blocks, BLOCK, n), dtype=torch.float64) for n in (LATENT, KEY, 1))
        x, y = st["latent"].double().cpu() / st["latent_scale"], st["key"].double().cpu()
        for r, s in enumerate(st["slots"].tolist()):
            if s >= 0:
                top = float(y[r].abs().max()) / 448 or 1.0
                latent[s // 64, s % 64], key[s // 64, s % 64], scale[s // 64, s % 64] = x[r].clamp(-448, 448), y[r] / top, top
        return {"latent": latent.flatten(1), "key": key.flatten(1), "scale": scale.flatten(1)}
    # row by row, as the rule is written; sequences that have ended keep their state
    heads = st["v"].shape[1]
    of = torch.arange(heads, device="cuda") * st["q"].shape[1] // heads
    lens = torch.tensor(st["lens"], device="cuda")
    S = torch.zeros((len(lens), heads, DIM, DIM), dtype=torch.float64, device="cuda")
    for b, s in enumerate(st["slots_in"].tolist()):
        if s >= 0:
            S[b] = st["states"][s].double()
    out, states = torch.zeros_like(st["out"], dtype=torch.float64), torch.zeros_like(st["states"], dtype=torch.float64)
    first = st["starts"][:-1].long()
    for t in range(max(st["lens"])):
        live = None if t < min(st["lens"]) else torch.nonzero(t < lens)[:, 0]
        r = first + t if live is None else first[live] + t
        old = S if live is None else S[live]
        g = st["gate"][r].double()
        old = old * torch.exp(g)[:, :, None, :] if g.dim() == 3 else old * torch.exp(g)[:, :, None, None]
        kt, qt = st["k"][r].double()[:, of], st["q"][r].double()[:, of]
        u = st["beta"][r].double()[..., None] * (st["v"][r].double() - torch.einsum("bhvk,bhk->bhv", old, kt))
        old.addcmul_(u[..., None], kt[:, :, None, :])
        out[r] = torch.einsum("bhvk,bhk->bhv", old, qt) * SCALE
        if live is None:
            S = old
        else:
            S[live] = old
        if case["op"] == "decode":
            states[st["slots_out"][:, t].long()] = S
    if case["op"] == "prefill":
        states[st["slots_out"].long()] = S
    return {"out": out, "states": states[len(lens):]}
