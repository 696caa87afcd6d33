"""gated_delta_decode and gated_delta_prefill against the rule in 64 bits: row
and head mixes, decays, strides, slots, empty and one-row sequences, special
values, streams and graphs, and errors found on the device."""
import math

import pytest
import torch

from dsa_sparse_attention_index_gb300 import binding as B
from plain_delta import DIM, inputs, out_tolerance, rule, state_tolerance

pytestmark = pytest.mark.gpu
SCALE = DIM ** -0.5


def pool_of(slots, heads, seed=1, apart=0):
    """States 0.3 N(0, 1) in slots that lie `apart` floats apart; the gaps hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = heads * DIM * DIM
    wide = torch.full((slots, n + apart), math.nan, device="cuda")
    wide[:, :n] = 0.3 * torch.randn((slots, n), generator=g, device="cuda")
    return wide[:, :n].unflatten(1, (heads, DIM, DIM))


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prefill(pool, x, starts, slots_in, slots_out, out, st, stream=None):
    ws = B.workspace(B.gated_delta_prefill_workspace_size(x[2].shape[0], len(slots_in), pool.shape[1]))
    B.gated_delta_prefill(B.StatePool(pool), B.DeltaRows(*x, SCALE), starts, slots_in, slots_out, out, ws, st, stream)
    return ws


def check_state(got, want, rows, size):
    off = (got.double() - want).flatten(1).norm(dim=1)
    assert (off <= state_tolerance(rows, size)).all(), (off / size).max()


def check_out(got, want, rows, size, mass, q, chunked=True):
    off, tol = (got.double() - want).abs(), out_tolerance(want, rows, size, mass, q, SCALE, chunked)
    assert (off <= tol).all(), (off / tol).max()


@pytest.mark.parametrize("batch,nq,heads,qk,gate,apart", [
    (1, 1, 1, 1, "channel", 0), (1, 1, 96, 96, "channel", 0), (3, 2, 6, 2, "head", 8), (70, 1, 5, 5, "channel", 8),
    (2, 4, 96, 32, "head", 0), (5, 7, 7, 7, "channel", 1000), (33, 3, 33, 11, "channel", 64)])
def test_decode(batch, nq, heads, qk, gate, apart):
    x = inputs(batch * nq, heads, qk, gate, seed=batch + nq, apart=apart)
    q, k, v, g, beta = x
    slots = batch * (nq + 1) + 2
    pool = pool_of(slots, heads, apart=32 * (apart > 0))
    before = pool.clone()
    order = torch.randperm(slots, generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    slots_in, slots_out = order[:batch].clone(), order[batch:batch * (nq + 1)].clone().view(batch, nq)
    slots_in[0] = -1 if batch > 1 else slots_in[0]
    slots_out[-1, 0] = -1 if nq > 1 else slots_out[-1, 0]
    if nq > 1 and batch > 2:
        slots_out[1, 1] = slots_in[1]                    # in place
    out, st = torch.full((batch * nq, heads, DIM), math.nan, dtype=torch.bfloat16, device="cuda"), status()
    B.gated_delta_decode(B.StatePool(pool), B.DeltaRows(*x, SCALE), nq, slots_in, slots_out, out, st)
    assert st.item() == 0
    written = set()
    for b in range(batch):
        r = slice(b * nq, (b + 1) * nq)
        s0 = before[slots_in[b]] if slots_in[b] >= 0 else torch.zeros_like(before[0])
        want, states, size, mass = rule(q[r], k[r], v[r], g[r], beta[r], SCALE, s0)
        check_out(out[r], want, nq, size, mass, q[r], chunked=False)
        for j in range(nq):
            if slots_out[b, j] >= 0:
                check_state(pool[slots_out[b, j]], states[j], j + 1, size)
                written.add(int(slots_out[b, j]))
    for s in set(range(slots)) - written:
        assert torch.equal(pool[s], before[s])


LENS = [[1], [0], [64], [0, 0, 1], [63, 65, 0, 1, 2], [130, 17, 200], [16, 15, 33, 128, 127, 129]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("heads,qk,gate", [(1, 1, "channel"), (6, 2, "channel"), (4, 4, "head"), (40, 8, "head")])
def test_prefill(lens, heads, qk, gate):
    batch, lead, tail = len(lens), 3, 5                # rows before the first sequence and behind the last
    rows = lead + sum(lens) + tail
    x = inputs(rows, heads, qk, gate, seed=sum(lens), apart=8 * (heads == 6))
    q, k, v, g, beta = x
    for t in x:                                        # never read
        t[:lead] = math.nan
        t[rows - tail:] = math.nan
    pool = pool_of(2 * batch + 1, heads)
    before = pool.clone()
    slots_in = torch.arange(batch, dtype=torch.int32, device="cuda")
    slots_out = slots_in + batch
    slots_in[1::3] = -1
    slots_out[2::3] = slots_in[2::3]                   # in place
    if batch > 3:
        slots_out[3] = -1
    first = [lead + sum(lens[:b]) for b in range(batch + 1)]
    out, st = torch.full((rows, heads, DIM), 7.0, dtype=torch.bfloat16, device="cuda"), status()
    prefill(pool, x, ints(*first), slots_in, slots_out, out, st)
    assert st.item() == 0
    assert (out[:lead] == 7).all() and (out[rows - tail:] == 7).all()
    written = set()
    for b, n in enumerate(lens):
        r = slice(first[b], first[b + 1])
        s0 = before[slots_in[b]] if slots_in[b] >= 0 else torch.zeros_like(before[0])
        want, states, size, mass = rule(q[r], k[r], v[r], g[r], beta[r], SCALE, s0)
        check_out(out[r], want, n, size, mass, q[r])
        if slots_out[b] >= 0:
            check_state(pool[slots_out[b]], states[-1] if n else s0.double(), n, size)
            written.add(int(slots_out[b]))
    for s in set(range(2 * batch + 1)) - written:
        assert torch.equal(pool[s], before[s])


@pytest.mark.parametrize("batch", [33, 200])
def test_prefill_of_many_sequences(batch):
    """A mixed step: most sequences bring a row or two, some a prompt, some nothing."""
    g = torch.Generator().manual_seed(batch)
    lens = torch.where(torch.rand(batch, generator=g) < 0.8, torch.randint(0, 3, (batch,), generator=g),
                       torch.randint(15, 140, (batch,), generator=g)).tolist()
    lens[5], lens[6], lens[7] = 20, 21, 0
    rows, heads = sum(lens), 2
    x = inputs(rows, heads, heads, seed=batch)
    pool = pool_of(2 * batch, heads)
    before = pool.clone()
    slots_in = torch.randperm(batch, generator=g).to(torch.int32).cuda()
    slots_out = (batch + torch.randperm(batch, generator=g)).to(torch.int32).cuda()
    first = [sum(lens[:b]) for b in range(batch + 1)]
    out, st = torch.zeros((rows, heads, DIM), dtype=torch.bfloat16, device="cuda"), status()
    prefill(pool, x, ints(*first), slots_in, slots_out, out, st)
    assert st.item() == 0
    for b, n in enumerate(lens):
        r = slice(first[b], first[b + 1])
        s0 = before[slots_in[b]]
        want, states, size, mass = rule(*(t[r] for t in x), SCALE, s0)
        check_out(out[r], want, n, size, mass, x[0][r])
        check_state(pool[slots_out[b]], states[-1] if n else s0.double(), n, size)


def one(n, heads=2, seed=0, gate="channel"):
    x = inputs(n, heads, heads, gate, seed=seed)
    pool = pool_of(2, heads, seed=seed + 1)
    out, st = torch.zeros((n, heads, DIM), dtype=torch.bfloat16, device="cuda"), status()
    return x, pool, out, st


def run_one(x, pool, out, st):
    before = pool[0].clone()
    prefill(pool, x, ints(0, out.shape[0]), ints(0), ints(1), out, st)
    assert st.item() == 0
    want, states, size, mass = rule(*x, SCALE, before)
    check_out(out, want, out.shape[0], size, mass, x[0])
    check_state(pool[1], states[-1], out.shape[0], size)
    return want


@pytest.mark.parametrize("what", ["none", "reset", "rare reset", "fast", "very fast", "mixed", "growing", "growing fast"])
def test_decays(what):
    n = 150
    x, pool, out, st = one(n, seed=5)
    g = x[3]
    if what == "none":
        g.zero_()
    elif what == "reset":
        g[::7] = -math.inf
    elif what == "rare reset":
        g[40, :, ::3] = -math.inf
        g[41, :, 1::3] = -200.0
        g[100] = -math.inf
    elif what == "fast":
        g.fill_(-8.0)
    elif what == "very fast":
        g.fill_(-40.0)
    elif what == "mixed":
        g[:] = torch.where(torch.rand(g.shape, device="cuda") < 0.3, -30 * torch.rand(g.shape, device="cuda"), g)
    elif what == "growing":
        g[:, :, ::2] = 0.01
    else:
        g[30:90] = 0.2
    run_one(x, pool, out, st)


@pytest.mark.parametrize("what", ["beta 0", "beta 1", "beta 2", "one key", "zero keys", "two keys", "large values", "tiny",
                                  "long keys"])
def test_extremes(what):
    n = 140
    x, pool, out, st = one(n, seed=9)
    q, k, v, g, beta = x
    if what.startswith("beta"):
        beta.fill_(float(what[-1]))
    elif what == "one key":        # the same key over and over: each row replaces the one before
        k[:] = k[:1]
        beta.fill_(1.0)
        g.zero_()
    elif what == "two keys":
        k[:] = k[:2].repeat(n // 2, 1, 1)
        beta.fill_(2.0)
        g.zero_()
    elif what == "zero keys":
        k[::3] = 0
    elif what == "large values":
        v.mul_(2.0 ** 100)
        pool.mul_(2.0 ** 100)
    elif what == "long keys":      # |k| = 8: beta |k|^2 is what counts
        k.mul_(8.0)
        beta.mul_(1.0 / 64)
    else:
        v.mul_(2.0 ** -60)
        pool.mul_(2.0 ** -60)
    run_one(x, pool, out, st)


@pytest.mark.parametrize("where", ["v", "k", "q", "gate", "beta"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_before_a_bad_one_keep_their_values(where, bad):
    n, at = 150, 77
    x, pool, out, st = one(n, seed=11)
    good = torch.empty_like(out)
    p2 = pool.clone()
    prefill(p2, x, ints(0, n), ints(0), ints(1), good, st)
    want, _, size, mass = rule(*x, SCALE, pool[0])
    t = x["q k v gate beta".split().index(where)]
    t.view(n, 2, -1)[at, 0, 0] = bad
    prefill(pool, x, ints(0, n), ints(0), ints(1), out, st)
    assert st.item() == 0
    check_out(out[:at], want[:at], n, size, mass[:at], x[0][:at])
    assert torch.isfinite(out[:, 1]).all() and torch.equal(out[:, 1], good[:, 1])   # the other head
    bad64, states, _, _ = rule(*x, SCALE, pool[0])
    assert torch.equal(torch.isnan(out[at:, 0]) | torch.isinf(out[at:, 0]), ~torch.isfinite(bad64[at:, 0]))
    assert torch.equal(torch.isfinite(pool[1]), torch.isfinite(states[-1]))


def test_prefill_in_pieces_is_prefill_at_once_and_decode_goes_on():
    """A prompt at once, in chunks of 100 rows, and its last rows as draft rows: the same states and outputs."""
    n, heads = 333, 8
    x, pool, out, st = one(n, heads, seed=21)
    want, states, size, mass = rule(*x, SCALE, pool[0])
    for lo in range(0, 330, 110):
        part = [t[lo:lo + 110] for t in x]
        o = out[lo:lo + 110]
        prefill(pool, part, ints(0, 110), ints(1 if lo else 0), ints(1), o, st)
    B.gated_delta_decode(B.StatePool(pool), B.DeltaRows(*(t[330:] for t in x), SCALE), 3, ints(1), ints(-1, -1, 1).view(1, 3),
                         out[330:], st)
    assert st.item() == 0
    check_out(out, want, n, size, mass, x[0])
    check_state(pool[1], states[-1], n, size)


def test_states_in_the_packed_pool():
    """Slots that are parts of the cache's block rows: nothing else of the rows changes."""
    heads, stride = 3, 45312 * 5
    raw = torch.randint(0, 256, (4, stride), dtype=torch.uint8, device="cuda")
    view = raw[:, 128:128 + heads * 65536].view(torch.float32).unflatten(1, (heads, DIM, DIM))
    view.copy_(pool_of(4, heads))
    before, s0 = raw.clone(), view.clone()
    x = inputs(2, heads, heads, seed=3)
    out, st = torch.zeros((2, heads, DIM), dtype=torch.bfloat16, device="cuda"), status()
    B.gated_delta_decode(B.StatePool(view), B.DeltaRows(*x, SCALE), 2, ints(2), ints(-1, 3).view(1, 2), out, st)
    assert st.item() == 0
    want, states, size, mass = rule(*x, SCALE, s0[2])
    check_state(view[3], states[1], 2, size)
    check_out(out, want, 2, size, mass, x[0], chunked=False)
    view[3] = s0[3]
    assert torch.equal(raw, before)


def test_bad_slots_and_starts_are_reported():
    heads = 2
    x = inputs(40, heads, heads, seed=4)
    for slots_in, slots_out, starts in (([5], [0], [0, 40]), ([-2], [0], [0, 40]), ([0], [5], [0, 40]),
                                        ([0], [-3], [0, 40]), ([0], [1], [0, 41]), ([0], [1], [-1, 4]),
                                        ([0], [1], [9, 8]), ([0], [1], [2 ** 31 - 1, 4])):
        pool = pool_of(5, heads)
        before = pool.clone()
        out, st = torch.zeros((40, heads, DIM), dtype=torch.bfloat16, device="cuda"), status()
        prefill(pool, x, ints(*starts), ints(*slots_in), ints(*slots_out), out, st)
        assert st.item() == B.ERR_BOUNDS
        keep = [s for s in range(5) if s not in slots_out]
        assert torch.equal(pool[keep], before[keep])
    pool, st = pool_of(5, heads), status()
    out = torch.zeros((40, heads, DIM), dtype=torch.bfloat16, device="cuda")
    B.gated_delta_decode(B.StatePool(pool), B.DeltaRows(*x, SCALE), 20, ints(7, 0), torch.full_like(ints(*range(40)), -1)
                         .view(2, 20), out, st)
    assert st.item() == B.ERR_BOUNDS


def test_overlapping_sequences_whose_chunks_exceed_32_bits_are_reported():
    rows, batch = 1_800_000, 154_000    # every other sequence has all rows: 77,000 x 28,125 chunks > 2^31
    x = [torch.zeros((rows, 1, DIM), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    x += [torch.zeros((rows, 1), device="cuda"), torch.zeros((rows, 1), device="cuda")]
    pool, st = pool_of(2, 1), status()
    before = pool.clone()
    starts = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    starts[1::2] = rows
    none = torch.full((batch,), -1, dtype=torch.int32, device="cuda")
    out = torch.ones((rows, 1, DIM), dtype=torch.bfloat16, device="cuda")
    prefill(pool, x, starts, none, none, out, st)
    assert st.item() == B.ERR_BOUNDS
    assert torch.equal(pool, before) and (out == 0).all()


def test_side_stream_and_graph():
    """A prompt and the next token of two sequences, eagerly on a side stream, then captured and replayed over other
    workspace contents: the same bits."""
    n, heads = 300, 4
    x, pool, out, st = one(n, heads, seed=31)
    before = pool.clone()
    want, states, size, mass = rule(*x, SCALE, pool[0])
    ws = B.workspace(B.gated_delta_prefill_workspace_size(n, 1, heads))
    starts, a, b, both = ints(0, n), ints(0), ints(1), ints(0, 1)
    step, next_out = B.DeltaRows(*(t[:2] for t in x), SCALE), torch.zeros_like(out[:2])

    def calls(stream=None):
        B.gated_delta_prefill(B.StatePool(pool), B.DeltaRows(*x, SCALE), starts, a, b, out, ws, st, stream)
        B.gated_delta_decode(B.StatePool(pool), step, 1, both, both.view(2, 1), next_out, st, stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls(side)
    side.synchronize()
    check_out(out, want, n, size, mass, x[0])
    eager = out.clone(), next_out.clone(), pool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(2):
        pool.copy_(before)
        out.zero_()
        next_out.zero_()
        ws.fill_(0xA5)
        graph.replay()
        torch.cuda.synchronize()
        assert st.item() == 0
        for got, kept in zip((out, next_out, pool), eager):
            assert torch.equal(got, kept)


def test_a_sequence_does_not_depend_on_its_batch():
    """Alone, among others and on two streams at once: the same bits."""
    lens, heads = [150, 7, 333, 64, 21], 3
    rows, first = sum(lens), [sum([150, 7, 333, 64, 21][:b]) for b in range(6)]
    x = inputs(rows, heads, heads, seed=77)
    pool = pool_of(2 * len(lens), heads)
    before = pool.clone()
    slots = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    out, st = torch.zeros((rows, heads, DIM), dtype=torch.bfloat16, device="cuda"), status()
    prefill(pool, x, ints(*first), slots, slots + len(lens), out, st)
    streams, alone = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        part = [t[first[b]:first[b + 1]].clone() for t in x]
        p, o = before[b:b + 1].repeat(2, 1, 1, 1), torch.zeros((n, heads, DIM), dtype=torch.bfloat16, device="cuda")
        args = part, p, o, ints(0, n), ints(0), ints(1)
        ws = B.workspace(B.gated_delta_prefill_workspace_size(n, 1, heads))
        alone.append((args, ws))
    torch.cuda.synchronize()
    for i, ((part, p, o, starts, a, b), ws) in enumerate(alone):
        B.gated_delta_prefill(B.StatePool(p), B.DeltaRows(*part, SCALE), starts, a, b, o, ws, st, streams[i % 2])
    torch.cuda.synchronize()
    assert st.item() == 0
    for b, ((_, p, o, *_), _) in enumerate(alone):
        assert torch.equal(o, out[first[b]:first[b + 1]]) and torch.equal(p[1], pool[len(lens) + b])


def test_slots_beyond_4_gib():
    heads, apart = 1, (5 << 30) // 4
    raw = torch.zeros(apart + heads * DIM * DIM, device="cuda")
    pool = raw.as_strided((2, heads, DIM, DIM), (apart, DIM * DIM, DIM, 1))
    pool.copy_(pool_of(2, heads))
    s0 = pool[1].clone()
    x, out, st = inputs(100, heads, heads, seed=8), torch.zeros((100, heads, DIM), dtype=torch.bfloat16, device="cuda"), status()
    want, states, size, mass = rule(*x, SCALE, s0)
    prefill(pool, [t[:97] for t in x], ints(0, 97), ints(1), ints(1), out[:97], st)
    B.gated_delta_decode(B.StatePool(pool), B.DeltaRows(*(t[97:] for t in x), SCALE), 3, ints(1), ints(-1, -1, 1).view(1, 3),
                         out[97:], st)
    assert st.item() == 0
    check_out(out, want, 100, size, mass, x[0])
    check_state(pool[1], states[-1], 100, size)
