"""Cases, plain forms and exact values of the cache's dense attention, its
attention weights and its eviction.

    attend  attention of every query row over every token it sees in the paged
            cache (latents of 4 or 8 bits), without a selection: bf16 outputs
            and fp32 log-sum-exps
    mass    the attention weight that each cached token received, summed over
            heads and query rows and added to a running total: over all the
            tokens a row sees, or over the tokens its top-k selected
    evict   the tokens to keep (the first, the latest, and those of the largest
            total in between) and their records moved into fresh pages

`run` computes them in elementary torch operations where `own` is false and
through the package's entry points where it is true.
"""
import math

import torch

own = False

BLOCK, HEADS, LATENT, VALUE = 64, 96, 576, 512
RECORD = {"fp8": 576, "nvfp4": 352}               # latent bytes a token
KEY_BYTES = {"fp8": (128, 4), "mxfp4": (64, 4)}   # index-key codes and scales a token
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
SM_SCALE = 1.0 / math.sqrt(LATENT)


def listed():
    return [
        # one short conversation: a layer without an indexer, or a context too short for a selection
        {"name": "attend_one_row", "op": "attend", "latents": "nvfp4", "lens": "997", "nq": 1},
        # speculative verify: four draft rows a sequence over ragged contexts
        {"name": "attend_drafts", "op": "attend", "latents": "nvfp4", "lens": "8:1000:6001", "nq": 4},
        # a decode batch whose caches are held at a budget by eviction
        {"name": "attend_batch", "op": "attend", "latents": "nvfp4", "lens": "32:8192:65537", "nq": 1},
        # one long context in 8 bits: all the work lies along the tokens
        {"name": "attend_long_fp8", "op": "attend", "latents": "fp8", "lens": "1000001", "nq": 1},
        # a prefill chunk behind a prefix: 512 causal rows of one sequence
        {"name": "attend_chunk", "op": "attend", "latents": "nvfp4", "lens": "16388", "nq": 512},
        # a short context's weights
        {"name": "mass_short_fp8", "op": "mass", "latents": "fp8", "lens": "2:1500:2100", "nq": 2, "k": 0},
        # the weights of a decode batch
        {"name": "mass_batch", "op": "mass", "latents": "nvfp4", "lens": "16:16384:65537", "nq": 1, "k": 0},
        # a prompt's last rows as the window that judges its tokens
        {"name": "mass_window", "op": "mass", "latents": "nvfp4", "lens": "32770", "nq": 64, "k": 0},
        # the weights of the tokens that the top-k selected, long contexts
        {"name": "mass_selected_fp8", "op": "mass", "latents": "fp8", "lens": "32:16384:65536", "nq": 1, "k": 2048},
        # one sequence a little over its budget
        {"name": "evict_one", "op": "evict", "latents": "nvfp4", "keys": "mxfp4", "lens": "5001", "keep": 2048,
         "sink": 4, "recent": 512},
        # a batch at 420 bytes a token, down to a budget of 8,192
        {"name": "evict_batch", "op": "evict", "latents": "nvfp4", "keys": "mxfp4", "lens": "32:16384:49152",
         "keep": 8192, "sink": 64, "recent": 1024},
        # long contexts at 708 bytes a token, about halved
        {"name": "evict_long_fp8", "op": "evict", "latents": "fp8", "keys": "fp8", "lens": "4:131072:163840",
         "keep": 65536, "sink": 4, "recent": 4096},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attend", "mass", "evict"])
    case = {"op": op, "latents": rng.choice(["nvfp4", "nvfp4", "fp8"])}
    if op == "evict":
        top = log_int(200, 163840)
        n = log_int(1, max(1, min(32, 600000 // top)))
        keep = log_int(32, max(33, top))
        case.update(keys=rng.choice(["fp8", "mxfp4"]), lens=f"{n}:{max(1, top // 3)}:{top}", keep=keep,
                    sink=rng.choice([0, 4, min(64, keep // 4)]), recent=rng.randint(0, keep // 2))
    else:
        nq = rng.choice([1, 1, 2, 3, 4, 64])
        k = 0 if op == "attend" else rng.choice([0, rng.randint(1, 2048)])
        top = log_int(64, 262144 if nq < 64 else 32768)
        n = log_int(1, max(1, min(32 if nq < 64 else 4, 1000000 // top)))
        case.update(lens=f"{n}:{max(1, top // 4)}:{top}", nq=nq)
        if op == "mass":
            case["k"] = k
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
    spread = [lo + (hi - lo) * i // (n - 1) for i in range(n)]
    g = torch.Generator().manual_seed(seed + 17)
    return [spread[i] for i in torch.randperm(n, generator=g).tolist()]


def rand_latents(n, fmt, scale, g, dev):
    """n latent records (uint8) of N(0, 1) values, encoded for the given latent scale."""
    x = torch.randn((n, LATENT), generator=g, device=dev) / scale
    tail = x[:, VALUE:].clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    if fmt == "fp8":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    blk = x[:, :VALUE].reshape(n, VALUE // 16, 16)
    sc = (blk.abs().amax(2) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    step = sc.float().clamp(min=2.0 ** -9)[..., None]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
    code = torch.bucketize((blk / step).abs().contiguous(), mids) + 8 * (blk < 0)
    code = code.reshape(n, VALUE).to(torch.uint8)
    return torch.cat([code[:, 0::2] | (code[:, 1::2] << 4), sc.view(torch.uint8), tail], 1)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens = lengths(case, seed)
    batch, nq = len(lens), case.get("nq", 1)
    rows = batch * nq
    fmt, keys = case["latents"], case.get("keys", "mxfp4")
    rec, (kb, ks) = RECORD[fmt], KEY_BYTES[keys]
    nblk = [-(-L // BLOCK) for L in lens]
    used, most = sum(nblk), max(nblk)
    row_stride = BLOCK * (rec + kb + ks)
    scale = 0.5 + 1.5 * float(torch.rand((), generator=g, device=dev))

    pool = torch.empty((used, row_stride), dtype=torch.uint8, device=dev)
    pool[:, BLOCK * rec:] = torch.randint(0, 256, (used, BLOCK * (kb + ks)), generator=g, device=dev, dtype=torch.uint8)
    for i in range(0, used, 1024):
        n = min(1024, used - i)
        pool[i:i + n, :BLOCK * rec] = rand_latents(n * BLOCK, fmt, scale, g, dev).view(n, BLOCK * rec)
    perm = torch.randperm(used, generator=g, device=dev).to(torch.int32)
    table = torch.full((batch, most), -1, dtype=torch.int32, device=dev)
    at = 0
    for b in range(batch):
        table[b, :nblk[b]] = perm[at:at + nblk[b]]
        at += nblk[b]
    st = {"op": case["op"], "fmt": fmt, "keys": keys, "scale": scale, "lens": lens, "nq": nq, "pool": pool, "table": table,
          "seq_lens": torch.tensor(lens, dtype=torch.int32, device=dev)}
    if own:
        from dsa_sparse_attention_index_gb300 import binding

        st["cache"] = binding.PagedCache(pool, row_stride, 0, BLOCK * rec,
                                         binding.KEY_FP8_E4M3 if keys == "fp8" else binding.KEY_MXFP4, scale,
                                         binding.LATENT_FP8_E4M3 if fmt == "fp8" else binding.LATENT_NVFP4)
        st["batch"] = binding.Batch(table, st["seq_lens"], nq, max(lens))
        st["status"] = torch.zeros(1, dtype=torch.int32, device=dev)

    if case["op"] in ("attend", "mass"):
        # heads of every sharpness, from nearly uniform to a few tokens that take most of the weight
        sharp = torch.linspace(0.5, 3.0, HEADS, device=dev)[None, :, None]
        st["q"] = (torch.randn((rows, HEADS, LATENT), generator=g, device=dev) * sharp).to(torch.bfloat16)
    if case["op"] == "attend":
        st["out"] = torch.empty((rows, HEADS, VALUE), dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.empty((rows, HEADS), dtype=torch.float32, device=dev)
        if own:
            st["ws"] = binding.workspace(binding.dense_mla_workspace_size(rows, max(lens)))
    elif case["op"] == "mass":
        k = case["k"]
        st["idx"] = None
        if k:
            st["idx"] = torch.full((rows, k), -1, dtype=torch.int32, device=dev)
            for r in range(rows):
                vis = max(0, lens[r // nq] - (nq - 1) + r % nq)
                n = min(k, vis)
                pick = torch.rand(vis, generator=g, device=dev).topk(n).indices
                st["idx"][r, :n] = pick.sort().values.to(torch.int32)
        ld = -(-max(lens) // 4) * 4
        st["before"] = torch.empty((batch, ld), device=dev).exponential_(1.0, generator=g)
        st["mass"] = torch.zeros((batch, ld), dtype=torch.float32, device=dev)
        st["lse"] = torch.stack([plain_logits(st, r)[0].logsumexp(1) for r in range(rows)])
        if own:
            st["ws"] = binding.workspace(binding.attention_mass_workspace_size(rows, max(lens), k))
    else:
        keep = case["keep"]
        st.update(keep=keep, sink=case["sink"], recent=case["recent"])
        mass = torch.exp(2.5 * torch.randn((batch, max(lens)), generator=g, device=dev))
        # tokens that no row ever selected, and totals that tie
        mass = torch.where(torch.rand(mass.shape, generator=g, device=dev) < 0.2, torch.zeros_like(mass), mass)
        st["mass"] = torch.where(torch.rand(mass.shape, generator=g, device=dev) < 0.1, mass.round(), mass)
        dblk = -(-keep // BLOCK)
        st["dst"] = torch.zeros((batch * dblk, row_stride), dtype=torch.uint8, device=dev)
        st["dst_table"] = torch.randperm(batch * dblk, generator=g, device=dev).to(torch.int32).view(batch, dblk)
        st["kept"] = torch.empty((batch, keep), dtype=torch.int32, device=dev)
        st["new_mass"] = torch.empty((batch, keep), dtype=torch.float32, device=dev)
        st["new_lens"] = torch.empty(batch, dtype=torch.int32, device=dev)
        if own:
            st["dst_cache"] = binding.PagedCache(st["dst"], row_stride, 0, BLOCK * rec, st["cache"].key_format, scale,
                                                 st["cache"].latent_format)
            st["ws"] = binding.workspace(binding.cache_evict_workspace_size(batch, max(lens), keep))
    return st


# ---------------------------------------------------------------- plain forms
def plain_latents(st, b, tokens=None):
    """Latents of sequence b without the layer's scale, fp32 [n, 576]; all its tokens, or those listed."""
    rec = RECORD[st["fmt"]]
    if tokens is None:
        n = -(-st["lens"][b] // BLOCK)
        r = st["pool"][st["table"][b, :n].long(), :BLOCK * rec].reshape(n * BLOCK, rec)[:st["lens"][b]]
    else:
        row = st["table"][b][tokens // BLOCK].long()
        slots = st["pool"][:, :BLOCK * rec].unflatten(1, (BLOCK, rec))
        r = slots[row, tokens % BLOCK]
    if st["fmt"] == "fp8":
        return r.contiguous().view(torch.float8_e4m3fn).float()
    grid = torch.tensor(E2M1, device=r.device)
    codes = torch.stack([r[:, :256] & 15, r[:, :256] >> 4], 2).reshape(-1, VALUE // 16, 16)
    scales = r[:, 256:288].contiguous().view(torch.float8_e4m3fn).float()
    head = grid[codes.long()] * scales[..., None]
    return torch.cat([head.reshape(-1, VALUE), r[:, 288:].contiguous().view(torch.float8_e4m3fn).float()], 1)


def plain_logits(st, row, latents=None):
    """Row's scaled logits fp32 [96, n], its latents and its tokens (None: the first n)."""
    b, j = row // st["nq"], row % st["nq"]
    tokens = None
    if st.get("idx") is not None:
        tokens = st["idx"][row]
        tokens = tokens[tokens >= 0].long()
        latents = plain_latents(st, b, tokens)
    else:
        if latents is None:
            latents = plain_latents(st, b)
        latents = latents[:max(0, st["lens"][b] - (st["nq"] - 1) + j)]
    return st["q"][row].float() @ latents.T * (SM_SCALE * st["scale"]), latents, tokens


def plain_attend(st):
    out, lse = torch.empty_like(st["out"]), torch.empty_like(st["lse"])
    for b in range(len(st["lens"])):
        latents = plain_latents(st, b)
        for row in range(b * st["nq"], (b + 1) * st["nq"]):
            logits, lat, _ = plain_logits(st, row, latents)
            if lat.shape[0] == 0:
                out[row], lse[row] = 0.0, -math.inf
                continue
            top = logits.amax(1, keepdim=True)
            p = torch.exp(logits - top)
            s = p.sum(1, keepdim=True)
            out[row] = ((p @ lat[:, :VALUE]) * (st["scale"] / s)).to(torch.bfloat16)
            lse[row] = (top + torch.log(s))[:, 0]
    return {"out": out, "lse": lse}


def plain_mass(st):
    mass = torch.zeros_like(st["before"])
    for b, L in enumerate(st["lens"]):
        total = st["before"][b, :L].clone()
        latents = plain_latents(st, b) if st["idx"] is None else None
        for row in range(b * st["nq"], (b + 1) * st["nq"]):
            logits, lat, tokens = plain_logits(st, row, latents)
            if lat.shape[0] == 0:
                continue
            w = torch.exp(logits - st["lse"][row][:, None]).sum(0)
            if tokens is None:
                total[:w.shape[0]] += w
            else:
                total[tokens] += w
        mass[b, :L] = total
    return {"mass": mass}


def plain_evict(st):
    keep, sink, recent = st["keep"], st["sink"], st["recent"]
    rec, (kb, ks) = RECORD[st["fmt"]], KEY_BYTES[st["keys"]]
    parts = ((0, rec), (BLOCK * rec, kb), (BLOCK * (rec + kb), ks))   # offset in a row, bytes a token
    kept, new_mass = torch.full_like(st["kept"], -1), torch.zeros_like(st["new_mass"])
    new_lens, dst = torch.empty_like(st["new_lens"]), torch.zeros_like(st["dst"])
    for b, L in enumerate(st["lens"]):
        if L <= keep:
            tok = torch.arange(L, device=kept.device)
        else:
            middle = st["mass"][b, sink:L - recent]
            best = torch.sort(middle, descending=True, stable=True).indices[:keep - sink - recent] + sink
            tok = torch.cat([torch.arange(sink, device=kept.device), best.sort().values,
                             torch.arange(L - recent, L, device=kept.device)])
        n = tok.shape[0]
        kept[b, :n] = tok.to(torch.int32)
        new_mass[b, :n] = st["mass"][b, tok]
        new_lens[b] = n
        to = torch.arange(n, device=kept.device)
        src_row, dst_row = st["table"][b][tok // BLOCK].long(), st["dst_table"][b][to // BLOCK].long()
        for off, size in parts:
            s = st["pool"][:, off:off + BLOCK * size].unflatten(1, (BLOCK, size))
            d = dst[:, off:off + BLOCK * size].unflatten(1, (BLOCK, size))
            d[dst_row, to % BLOCK] = s[src_row, tok % BLOCK]
    return {"kept": kept, "mass": new_mass, "lens": new_lens, "pool": dst}


def run(st):
    if not own:
        return {"attend": plain_attend, "mass": plain_mass, "evict": plain_evict}[st["op"]](st)
    from dsa_sparse_attention_index_gb300 import binding

    if st["op"] == "attend":
        binding.dense_mla_decode(st["cache"], st["batch"], st["q"], SM_SCALE, st["out"], st["lse"], st["ws"], st["status"])
        return {"out": st["out"], "lse": st["lse"]}
    if st["op"] == "mass":
        binding.attention_mass(st["cache"], st["batch"], st["q"], st["lse"], SM_SCALE, st["before"], st["mass"], st["ws"],
                               st["status"], idx=st["idx"])
        return {"mass": st["mass"]}
    binding.cache_evict(st["cache"], st["batch"], st["mass"], st["keep"], st["sink"], st["recent"], st["dst_cache"],
                        st["dst_table"], st["kept"], st["new_mass"], st["new_lens"], st["ws"], st["status"])
    return {"kept": st["kept"], "mass": st["new_mass"], "lens": st["new_lens"], "pool": st["dst"]}


# ---------------------------------------------------------------- work and exact values
def work(case):
    lens = lengths(case, 0)
    nq, rec = case.get("nq", 1), RECORD[case["latents"]]
    if case["op"] == "evict":
        # every total once; a kept token's record and total read and written, its index written
        kept = sum(min(L, case["keep"]) for L in lens)
        token = rec + sum(KEY_BYTES[case["keys"]])
        return {"bytes": 4 * sum(lens) + kept * (2 * token + 8), "flops": 0}
    vis = [max(0, L - (nq - 1) + j) for L in lens for j in range(nq)]
    rows = len(vis)
    if case["op"] == "attend":
        return {"bytes": sum(lens) * rec + rows * HEADS * (2 * (LATENT + VALUE) + 4),
                "flops": 2 * HEADS * (LATENT + VALUE) * sum(vis)}
    # the queries and log-sum-exps, the totals read and written, and the latents seen
    k = case["k"]
    seen = sum(min(k, v) for v in vis) if k else sum(vis)
    latents = sum(min(L, nq * k) for L in lens) if k else sum(lens)
    return {"bytes": latents * rec + (4 * seen if k else 0) + 8 * sum(lens) + rows * HEADS * (2 * LATENT + 4),
            "flops": 2 * HEADS * LATENT * seen}


def exact(case, seed):
    w = work(case)
    if w["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    lens, nq, rec = st["lens"], st["nq"], RECORD[st["fmt"]]
    if st["op"] == "evict":
        kept, mass = torch.full_like(st["kept"], -1).cpu(), torch.zeros(st["new_mass"].shape, dtype=torch.float64)
        lens_out, dst = torch.zeros(len(lens), dtype=torch.int32), torch.zeros_like(st["dst"])
        kb, ks = KEY_BYTES[st["keys"]]
        for b, L in enumerate(lens):
            m = st["mass"][b, :L].double().cpu()
            rank = m.clone()
            rank[:st["sink"]] = math.inf
            rank[L - st["recent"]:] = math.inf
            # an order by (total descending, index ascending): the stable sort of the negated totals
            order = torch.argsort(-rank, stable=True)[:min(L, st["keep"])]
            tok = torch.sort(order).values
            n = len(tok)
            kept[b, :n], mass[b, :n], lens_out[b] = tok.int(), m[tok], n
            tok = tok.to(dst.device)
            to = torch.arange(n, device=dst.device)
            src, out = st["table"][b].long()[tok // 64], st["dst_table"][b].long()[to // 64]
            for off, size in ((0, rec), (64 * rec, kb), (64 * (rec + kb), ks)):
                at = off + (tok % 64) * size
                to_at = off + (to % 64) * size
                for c in range(size):
                    dst[out, to_at + c] = st["pool"][src, at + c]
        return {"kept": kept, "mass": mass, "lens": lens_out, "pool": dst}

    f8 = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    f4 = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    out = torch.zeros((len(lens) * nq, HEADS, VALUE), dtype=torch.float64, device="cuda")
    lse = torch.full((len(lens) * nq, HEADS), -math.inf, dtype=torch.float64, device="cuda")
    mass = torch.zeros_like(st["before"], dtype=torch.float64) if st["op"] == "mass" else None
    for b, L in enumerate(lens):
        t = torch.arange(L, device="cuda")
        raw = st["pool"][st["table"][b].long()[t // 64]].view(L, -1) if L else st["pool"][:0]
        raw = torch.gather(raw, 1, (t % 64 * rec)[:, None] + torch.arange(rec, device="cuda")[None, :]).long()
        if st["fmt"] == "fp8":
            c = f8[raw]
        else:
            c = torch.empty((L, LATENT), dtype=torch.float64, device="cuda")
            c[:, 0:VALUE:2], c[:, 1:VALUE:2] = f4[raw[:, :256] % 16], f4[raw[:, :256] // 16]
            c[:, :VALUE] *= f8[raw[:, 256:288]].repeat_interleave(16, 1)
            c[:, VALUE:] = f8[raw[:, 288:]]
        c = c * st["scale"]
        if mass is not None:
            mass[b, :L] = st["before"][b, :L].double()
        for row in range(b * nq, (b + 1) * nq):
            see = torch.arange(max(0, L - (nq - 1) + row % nq), device="cuda")
            if st.get("idx") is not None:
                see = st["idx"][row].long()
                see = see[see >= 0]
            x = st["q"][row].double() @ c[see].T * SM_SCALE
            if mass is not None:
                mass[b].index_add_(0, see, torch.exp(x - st["lse"][row].double()[:, None]).sum(0))
            elif len(see):
                out[row], lse[row] = torch.softmax(x, 1) @ c[see][:, :VALUE], torch.logsumexp(x, 1)
    return {"mass": mass} if mass is not None else {"out": out, "lse": lse}
