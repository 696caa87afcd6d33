"""dsa_assign_slots and dsa_cache_append_slots: pages, lengths, rows and slots
against a plain loop over the requests, in place, over errors found on the
device, in a captured step; the write against dsa_cache_append, byte for byte;
and a whole step of the calls that take what they make."""
import numpy as np
import pytest
import torch

from dsa_sparse_attention_index_gb300 import binding as B
from dsa_sparse_attention_index_gb300 import synth
from plain_delta import DIM, inputs, out_tolerance, rule, state_tolerance

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def plain(cached, new, free, count, table):
    """One request after another: (table, seq_lens, row_starts, positions, slots, pages left)."""
    table, starts, positions, slots = [list(r) for r in table], [0], [], []
    for i, (c, n) in enumerate(zip(cached, new)):
        for p in range(c, c + n):
            if p % 64 == 0:
                count -= 1
                table[i][p // 64] = free[count]
            positions.append(p)
            slots.append(table[i][p // 64] * 64 + p % 64)
        starts.append(starts[-1] + n)
    return table, [c + n for c, n in zip(cached, new)], starts, positions, slots, count


class Step:
    """The arguments of one call over random pages."""

    def __init__(self, cached, new, spare=7, pad=5, seed=0, max_blocks=None):
        rng = np.random.default_rng(seed)
        have = [-(-c // 64) for c in cached]
        need = [-(-(c + n) // 64) for c, n in zip(cached, new)]
        self.blocks = sum(need) + spare
        perm = rng.permutation(self.blocks).tolist()
        width = max_blocks or max(need + [1]) + 1
        self.table0 = [[-7] * width for _ in cached]
        for i, h in enumerate(have):
            self.table0[i][:h] = [perm.pop() for _ in range(h)]
        self.free0 = perm
        self.cached, self.new, self.rows, self.pad = list(cached), list(new), sum(new), pad
        self.reset()

    def reset(self):
        self.c, self.n = ints(self.cached), ints(self.new)
        self.free = ints(self.free0 + [10 ** 9] * 3)          # behind the count
        self.count, self.left = ints([len(self.free0)]), ints([-5])
        self.table = ints(self.table0).view(len(self.cached), -1)
        self.lens, self.starts = ints([-9] * len(self.cached)), ints([-9] * (len(self.cached) + 1))
        self.pos, self.slots = ints([-9] * (self.rows + self.pad)), ints([-9] * (self.rows + self.pad))
        self.st = ints([0])

    def call(self, stream=None):
        B.assign_slots(self.c, self.n, self.free, self.count, self.blocks, self.table, self.lens, self.starts, self.pos,
                       self.slots, self.left, self.st, stream)

    def check(self):
        assert self.st.item() == 0
        table, lens, starts, pos, slots, left = plain(self.cached, self.new, self.free0, len(self.free0), self.table0)
        assert self.table.tolist() == table and self.lens.tolist() == lens and self.starts.tolist() == starts
        assert self.pos.tolist() == pos + [-1] * self.pad and self.slots.tolist() == slots + [-1] * self.pad
        assert self.left.item() == left


MIXES = {
    "one": ([0], [1]), "none new": ([5, 64], [0, 0]), "page ends": ([63, 64, 65, 128], [1, 1, 1, 64]),
    "empty requests": ([0, 0, 100, 0], [0, 70, 0, 0]), "decode": (list(range(0, 2000, 31)), [1] * 65),
    "prompts": ([0, 640, 3], [5000, 1, 2111]), "one long": ([1], [40000]),
    "2048": ([(7 * i) % 300 for i in range(2048)], [i % 5 for i in range(2048)]),
    "2049": ([(7 * i) % 300 for i in range(2049)], [(i + 1) % 3 for i in range(2049)]),
    "5000": ([(11 * i) % 90 for i in range(5000)], [(3 * i) % 31 for i in range(5000)]),
}


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("pad", [0, 5, 9000])
def test_assign(mix, pad):
    s = Step(*MIXES[mix], pad=pad, seed=len(mix))
    s.call()
    s.check()


@pytest.mark.parametrize("mix", ["page ends", "prompts", "2049"])
def test_assign_into_buffers_off_a_16_byte_boundary(mix):
    s = Step(*MIXES[mix])
    s.pos, s.slots = (torch.full((t.numel() + 3,), -9, dtype=torch.int32, device="cuda")[3:] for t in (s.pos, s.slots))
    s.call()
    s.check()


def test_assign_of_an_empty_batch():
    s = Step([3], [1], pad=6)
    none = s.c[:0]
    starts = ints([4])
    B.assign_slots(none, none, s.free, s.count, s.blocks, s.table[:0], s.lens[:0], starts, s.pos, s.slots, s.left, s.st)
    assert s.st.item() == 0 and starts.item() == 0 and s.left.item() == len(s.free0)
    assert (s.slots == -1).all() and (s.pos == -1).all()


@pytest.mark.parametrize("mix", ["page ends", "prompts", "5000"])
def test_assign_in_place_step_after_step(mix):
    """Lengths and the stack's count in place, as a captured step has them: replayed three times."""
    cached, new = MIXES[mix]
    s = Step(cached, new, spare=sum(-(-n // 64) + 1 for n in new) * 2 + 5, max_blocks=max(-(-(c + 3 * n) // 64)
                                                                                       for c, n in zip(cached, new)))
    B.assign_slots(s.c.clone(), s.n, s.free, s.count.clone(), s.blocks, s.table.clone(), s.lens, s.starts, s.pos, s.slots,
                   s.left, s.st)                               # a first launch outside of the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.assign_slots(s.c, s.n, s.free, s.count, s.blocks, s.table, s.c, s.starts, s.pos, s.slots, s.count, s.st)
    table, lens, left = s.table0, cached, len(s.free0)
    for _ in range(3):
        graph.replay()
        table, lens, starts, pos, slots, left = plain(lens, new, s.free0, left, table)
        assert s.st.item() == 0 and s.table.tolist() == table and s.c.tolist() == lens and s.count.item() == left
        assert s.slots.tolist() == slots + [-1] * s.pad and s.pos.tolist() == pos + [-1] * s.pad


def test_assign_errors_stay_in_bounds():
    """Lengths, pages and entries that cannot be: reported; what is around the buffers stays as it was."""
    def run(change, **kw):
        s = Step([10, 64, 100], [60, 3, 200], **kw)
        guard = {}
        for name in ("table", "lens", "starts", "pos", "slots"):
            t = getattr(s, name)
            wide = torch.full((t.numel() + 64,), 123456, dtype=torch.int32, device="cuda")
            wide[32:32 + t.numel()] = t.flatten()
            guard[name] = wide
            setattr(s, name, wide[32:32 + t.numel()].view(t.shape))
        change(s)
        before = {name: wide.clone() for name, wide in guard.items()}
        s.call()
        for name, wide in guard.items():
            n = getattr(s, name).numel()
            assert torch.equal(wide[:32], before[name][:32]) and torch.equal(wide[32 + n:], before[name][32 + n:]), name
        return s

    def put(name, at, value):
        def change(s):
            getattr(s, name).view(-1)[at] = value
        return change

    for change in (put("c", 1, -1), put("n", 0, -5), put("n", 2, 2 ** 31 - 1), put("c", 0, 2 ** 31 - 1),
                   put("count", 0, -1), put("count", 0, 1000), put("count", 0, 2)):
        assert run(change).st.item() == B.ERR_BOUNDS
    s = run(put("n", 1, -4))
    assert s.lens[1].item() == 0 and s.starts.tolist() == [0, 60, 60, 260]
    s = run(put("free", len(Step([10, 64, 100], [60, 3, 200]).free0) - 1, 10 ** 6))
    assert s.st.item() == B.ERR_BOUNDS and (s.slots[54:60] == -1).all() and (s.slots[:54] >= 0).all()
    s = run(put("table", 0, -3))
    assert s.st.item() == B.ERR_BOUNDS and (s.slots[:54] == -1).all()

    def short(s):
        s.pos, s.slots = s.pos[:100], s.slots[:100]
    s = run(short, pad=0)
    assert s.st.item() == B.ERR_BOUNDS and (s.slots >= 0).all() and s.starts.max().item() <= 100


FORMATS = [(synth.KEY_FP8, synth.LATENT_FP8), (synth.KEY_MXFP4, synth.LATENT_FP8), (synth.KEY_MXFP4, synth.LATENT_NVFP4),
           (synth.KEY_FP8, synth.LATENT_NVFP4)]


def new_rows(rows, seed):
    rng = np.random.default_rng(seed)
    lat = rng.standard_normal((rows, 576)) * np.exp(rng.uniform(-6, 6, (rows, 36, 1))).repeat(16, 2).reshape(rows, 576)
    key = rng.standard_normal((rows, 128)) * np.exp(rng.uniform(-2, 2, (rows, 1)))
    lat[0, :4], lat[-1, 32:48], key[-1], key[0, 32:64] = (1e30, -1e30, -0.0, 1e-38), 0.0, 0.0, 1e-35
    lat[rows // 2, 64:80] *= 1e-30
    return [torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda() for x in (lat, key)]


@pytest.mark.parametrize("kfmt,lfmt", FORMATS)
@pytest.mark.parametrize("lens,nq", [([1000, 64, 777], 1), ([5000, 130, 64, 65], 4), ([4000], 2048)])
def test_append_slots_writes_what_append_writes(kfmt, lfmt, lens, nq):
    case = synth.make_case("ap", seq_lens=lens, nq=nq, key_format=kfmt, seed=nq, spare_blocks=2, latent_format=lfmt)
    lat, key = new_rows(case.rows, nq)
    a, b = synth.device_case(case), synth.device_case(case)
    st = ints([0])
    B.cache_append(a.cache, a.batch, lat, key, st)
    t = np.array([L - nq + j for L in lens for j in range(nq)])
    table = np.asarray(case.block_table)
    slots = table[np.arange(case.rows) // nq, t // 64].astype(np.int64) * 64 + t % 64
    # padding rows between them, whose values are not read
    order = np.random.default_rng(1).permutation(case.rows + 3)
    rows, put = torch.full((case.rows + 3,), -1, dtype=torch.int32, device="cuda"), torch.from_numpy(order[:case.rows]).cuda()
    rows[put] = ints(slots.tolist())
    lat2, key2 = torch.full((case.rows + 3, 576), float("nan"), dtype=torch.bfloat16, device="cuda"), \
        torch.full((case.rows + 3, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lat2[put], key2[put] = lat, key
    B.cache_append_slots(b.cache, rows, lat2, key2, st)
    assert st.item() == 0 and torch.equal(a.cache.pool, b.cache.pool)


def test_append_slots_outside_the_pool_are_reported():
    case = synth.make_case("ap", seq_lens=[300], nq=1, seed=1, spare_blocks=2)
    dc, st = synth.device_case(case), ints([0])
    before = dc.cache.pool.clone()
    lat, key = new_rows(4, 3)
    n = dc.cache.pool.shape[0] * 64
    B.cache_append_slots(dc.cache, ints([-2, n, 2 ** 31 - 1, -1]), lat, key, st)
    assert st.item() == B.ERR_BOUNDS and torch.equal(dc.cache.pool, before)
    B.cache_append_slots(dc.cache, ints([]), lat[:0], key[:0], st)


def test_a_step_of_the_calls_together():
    """Two steps over three requests: pages and slots, the cache write, dense attention over the table that was built,
    and a recurrent layer over the same rows: prompts first, then a token each.  The cache is what dsa_cache_append
    writes into the same pages, the recurrent states are the rule's."""
    new = ([70, 0, 200], [1, 1, 1])
    blocks, heads, scale = 40, 4, DIM ** -0.5
    stride = 64 * (576 + 132)
    pool = torch.zeros((blocks, stride), dtype=torch.uint8, device="cuda")
    ref = pool.clone()
    cache, ref_cache = (B.PagedCache(p, stride, 0, 64 * 576, B.KEY_FP8_E4M3, 0.02) for p in (pool, ref))
    perm = np.random.default_rng(0).permutation(blocks).tolist()
    lens, table, free, count, st = ints([0, 0, 0]), ints([[-1] * 8] * 3), ints(perm), ints([blocks]), ints([0])
    starts = ints([0] * 4)
    states = torch.zeros((3, heads, DIM, DIM), device="cuda")
    want_state, slots_in, rng = [states[0].double()] * 3, ints([-1, -1, -1]), np.random.default_rng(5)
    total = [0, 0, 0]
    for step, n in enumerate(new):
        rows = sum(n)
        pos, slots = ints([0] * rows), ints([0] * rows)
        B.assign_slots(lens, ints(list(n)), free, count, blocks, table, lens, starts, pos, slots, count, st)
        lat, key = (torch.from_numpy(rng.standard_normal((rows, w)).astype(np.float32)).to(torch.bfloat16).cuda()
                    for w in (576, 128))
        B.cache_append_slots(cache, slots, lat, key, st)
        total = [t + k for t, k in zip(total, n)]
        assert lens.tolist() == total
        first = [sum(n[:i]) for i in range(4)]
        assert starts.tolist() == first
        for i in range(3):
            if n[i]:
                B.cache_append(ref_cache, B.Batch(table[i:i + 1].contiguous(), lens[i:i + 1].clone(), n[i], 512),
                               lat[first[i]:first[i + 1]].contiguous(), key[first[i]:first[i + 1]].contiguous(), st)
        assert torch.equal(pool, ref)
        x = inputs(rows, heads, 2, seed=step)
        out = torch.zeros((rows, heads, DIM), dtype=torch.bfloat16, device="cuda")
        spool, data = B.StatePool(states), B.DeltaRows(*x, scale)
        own = ints([0, 1, 2])
        if step == 0:
            ws = B.workspace(B.gated_delta_prefill_workspace_size(rows, 3, heads))
            B.gated_delta_prefill(spool, data, starts, slots_in, own, out, ws, st)
        else:
            B.gated_delta_decode(spool, data, 1, own, own.view(3, 1), out, st)
        for i in range(3):
            r = slice(first[i], first[i + 1])
            want, after, size, mass = rule(*(t[r] for t in x), scale, want_state[i])
            if n[i]:
                assert ((out[r].double() - want).abs() <= out_tolerance(want, 300, size, mass, x[0][r], scale, step == 0)).all()
                want_state[i] = after[-1]
            off = (states[i].double() - want_state[i]).flatten(1).norm(dim=1)
            assert (off <= state_tolerance(300, size)).all()
    # attention over the three requests' tokens, through the table
    q = torch.from_numpy(rng.standard_normal((3, 96, 576)).astype(np.float32)).to(torch.bfloat16).cuda()
    out, lse = torch.empty((3, 96, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((3, 96), device="cuda")
    ws = B.workspace(B.dense_mla_workspace_size(3, 512))
    B.dense_mla_decode(cache, B.Batch(table, lens, 1, 512), q, 0.04, out, lse, ws, st)
    assert st.item() == 0
    for i in range(3):
        at = torch.arange(total[i], device="cuda")
        codes = ref[:, :64 * 576].view(torch.float8_e4m3fn).unflatten(1, (64, 576))
        c = codes.view(torch.uint8)[table[i].long()[at // 64], at % 64].view(torch.float8_e4m3fn).double() * 0.02
        p = torch.softmax(q[i].double() @ c.T * 0.04, 1)
        # 2^-8 of the value and, for the kernel's own roundings of the weights to fp16, 2^-10 of the values' size
        assert ((out[i].double() - p @ c[:, :512]).abs() <= 2.0 ** -7 * (p @ c[:, :512].abs())).all()
