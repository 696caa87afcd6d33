"""dsa_attention_mass and dsa_cache_evict: the attention weight per cached
token against a plain 64-bit form, the eviction against a plain ranking and
copy (bit for bit), and the three calls together with the dense attention, as a
serving loop makes them: attend, add the weights, evict, go on with the smaller
cache.

Tolerance of a weight sum_h exp(l_h - lse_h), per head relative to exp(.):
  576 * 2^-24 * Sum |q c| sm_scale   the fp32 sum of 576 exact products
  2^-21 * (1 + |l| + |lse|)          the scaled argument's roundings and the exponential
then (96 + rows) * 2^-24 of the total for the fp32 sums over heads and rows.
"""
import dataclasses

import numpy as np
import pytest
import torch

import plain64
from dsa_sparse_attention_index_gb300 import binding, synth
from test_gpu_dense_mla import run_dense

pytestmark = pytest.mark.gpu

FP8, NV = synth.LATENT_FP8, synth.LATENT_NVFP4
BOUNDS = binding.ERR_BOUNDS


def plain_mass(case, before, lse, idx=None):
    """(mass, tolerance) float64 [batch, ld]; untouched entries keep `before`'s fill."""
    mass, tol = before.double().clone(), torch.zeros_like(before, dtype=torch.float64)
    for b in range(case.batch):
        L = int(case.seq_lens[b])
        c = plain64.latents(case, b)
        for j in range(case.nq):
            row = b * case.nq + j
            see = torch.arange(max(0, L - (case.nq - 1) + j))
            if idx is not None:
                see = idx[row][idx[row] >= 0].long()
            if len(see) == 0 or torch.isneginf(lse[row]).all():
                continue
            q, cs = plain64.queries(case, row), c[see]
            x = q @ cs.T * case.sm_scale
            bound = q.abs() @ cs.abs().T * case.sm_scale
            d = lse[row].double()[:, None]
            w = torch.exp(x - d)
            err = (w * (1.01 * 576 * 2.0 ** -24 * bound + 2.0 ** -21 * (1 + x.abs() + d.abs()))).sum(0)
            mass[b].index_add_(0, see, w.sum(0))
            tol[b].index_add_(0, see, err)
        tol[b, :L] += (96 + case.nq) * 2.0 ** -24 * mass[b, :L]
    return mass, tol


def run_mass(case, dc, lse, before, idx=None, in_place=False, stream=None):
    k = idx.shape[1] if idx is not None else 0
    ws = binding.workspace(binding.attention_mass_workspace_size(case.rows, dc.batch.max_seq_len, k))
    ws.fill_(255)
    mass_in = before.cuda() if before is not None else None
    out = mass_in if in_place else torch.full((case.batch, max(1, case.max_len + 3)), -7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.attention_mass(dc.cache, dc.batch, dc.q_mla, lse.cuda(), case.sm_scale, mass_in, out, ws, st,
                           idx=idx.cuda() if idx is not None else None, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), st.item()


def plain_lse(case, idx=None):
    out = []
    for row in range(case.rows):
        tokens = None if idx is None else idx[row][idx[row] >= 0].long()
        out.append(plain64.attend(case, row, tokens)[1])
    return torch.stack(out).float()


@pytest.mark.parametrize("fmt", [FP8, NV])
@pytest.mark.parametrize("lens,nq", [([1], 1), ([64], 1), ([127, 0, 129, 1], 1), ([1500], 1), ([3, 200, 700], 4),
                                     ([2, 66], 3), ([300], 64), ([20000, 5], 1)])
def test_mass_over_every_token(fmt, lens, nq):
    case = synth.make_case("mass", seq_lens=lens, nq=nq, seed=200 + len(lens) + nq, latent_format=fmt)
    lse = plain_lse(case)
    before = torch.rand((case.batch, case.max_len + 3), generator=torch.Generator().manual_seed(3))
    want, tol = plain_mass(case, before, lse)
    got, st = run_mass(case, synth.device_case(case), lse, before)
    assert st == 0
    for b, L in enumerate(lens):
        assert torch.all((got[b, :L].double() - want[b, :L]).abs() <= tol[b, :L]), (b, L)
        assert torch.all(got[b, L:] == -7.0)   # nothing behind the length


@pytest.mark.parametrize("fmt", [FP8, NV])
@pytest.mark.parametrize("lens,nq,k", [([5000, 100, 3000], 1, 2048), ([9000], 4, 300), ([64, 1, 0], 1, 1), ([700], 2, 129),
                                       ([200], 32, 17)])
def test_mass_over_selected_tokens(fmt, lens, nq, k):
    case = synth.make_case("mass_sel", seq_lens=lens, nq=nq, seed=300 + k, latent_format=fmt)
    g = torch.Generator().manual_seed(k)
    idx = torch.full((case.rows, k), -1, dtype=torch.int32)
    for r, vis in enumerate(case.row_lens()):
        n = min(k, int(vis))
        idx[r, :n] = torch.randperm(int(vis), generator=g)[:n].to(torch.int32)   # in no order
    if k > 20:
        idx[0, 3:9] = -1          # holes
        idx[0, 11] = idx[0, 10]   # a token listed twice counts twice
    lse = plain_lse(case, idx)
    before = torch.rand((case.batch, case.max_len + 3), generator=g)
    want, tol = plain_mass(case, before, lse, idx)
    dc = synth.device_case(case)
    got, st = run_mass(case, dc, lse, before, idx)
    assert st == 0
    again, _ = run_mass(case, dc, lse, before, idx, in_place=True)
    for b, L in enumerate(lens):
        assert torch.all((got[b, :L].double() - want[b, :L]).abs() <= tol[b, :L]), (b, L)
        assert torch.all(got[b, L:] == -7.0)
        assert torch.equal(again[b, :L], got[b, :L]) and torch.equal(again[b, L:], before[b, L:])


def test_mass_without_a_total_and_with_empty_rows():
    case = synth.make_case("mass_none", seq_lens=[300, 200], nq=2, seed=14)
    lse = plain_lse(case)
    lse[1] = -float("inf")   # a row that attended to nothing
    want, tol = plain_mass(case, torch.zeros((2, case.max_len + 3)), lse)
    got, st = run_mass(case, synth.device_case(case), lse, None)
    assert st == 0
    for b, L in enumerate([300, 200]):
        assert torch.all((got[b, :L].double() - want[b, :L]).abs() <= tol[b, :L])


@pytest.mark.parametrize("fmt", [FP8, NV])
def test_mass_keeps_masked_queries_out(fmt):
    """NaN and infinities in the query of a row, or of one head, whose LSE is -inf add nothing and disturb nothing."""
    case = synth.make_case("mass_masked", seq_lens=[300, 200], nq=2, seed=34, latent_format=fmt)
    lse = plain_lse(case)
    lse[1] = lse[2, 7] = lse[2, 95] = -float("inf")
    none = lse.masked_fill(torch.isneginf(lse), 1e30)   # whose weights vanish in the plain form
    want, tol = plain_mass(case, torch.zeros((2, case.max_len + 3)), none)
    q = case.q_mla.copy()
    q[1, ::2], q[1, 1::2], q[2, 7], q[2, 95, 575] = 0x7FC0, 0xFF80, 0x7F80, 0x7FC0
    masked = dataclasses.replace(case, q_mla=q)
    got, st = run_mass(masked, synth.device_case(masked), lse, None)
    assert st == 0
    for b, L in enumerate([300, 200]):
        assert torch.all((got[b, :L].double() - want[b, :L]).abs() <= tol[b, :L])


def test_mass_reports_bad_entries_and_pages():
    case = synth.make_case("mass_bad", seq_lens=[500], seed=15)
    lse = torch.zeros((1, 96))
    idx = torch.arange(100, dtype=torch.int32)[None].clone()
    idx[0, 7] = 500
    assert run_mass(case, synth.device_case(case), lse, None, idx)[1] == BOUNDS
    table = case.block_table.copy()
    table[0, 3] = case.num_blocks
    broken = dataclasses.replace(case, block_table=table)
    assert run_mass(broken, synth.device_case(broken), lse, None)[1] == BOUNDS


# ---------------------------------------------------------------- eviction
def order_value(x):
    """What totals are ranked by: NaN below -inf, -0 equal to +0."""
    return (-np.inf, 0) if np.isnan(x) else (float(x) + 0.0, 1)


def plain_kept(m, L, keep, sink, recent):
    if L <= keep:
        return list(range(L))
    middle = sorted(range(sink, L - recent), key=lambda t: (tuple(-v for v in order_value(m[t])), t))
    return sorted(list(range(sink)) + middle[:keep - sink - recent] + list(range(L - recent, L)))


def evict(case, dc, mass, keep, sink, recent, dst=None, dst_table=None, stream=None, with_mass=True):
    """dst: (cache, its pool on the host) or None: a fresh pool with other offsets and a padded stride."""
    rec, key = case.latent_bytes(), case.token_bytes()
    pages = -(-keep // 64)
    if dst is None:
        stride = 128 + 64 * key + 128 + 64 * rec + 256
        pool = torch.randint(0, 256, (case.batch * pages + 1, stride), dtype=torch.uint8,
                             generator=torch.Generator().manual_seed(4)).cuda()
        dst = binding.PagedCache(pool, stride, 128 + 64 * key + 128, 128, case.key_format, case.latent_scale,
                                 case.latent_format)
    if dst_table is None:
        perm = torch.randperm(case.batch * pages + 1, generator=torch.Generator().manual_seed(5))[:case.batch * pages]
        dst_table = perm.to(torch.int32).view(case.batch, pages).cuda()
    before = dst.pool.cpu().numpy().copy()
    kept = torch.full((case.batch, keep), -9, dtype=torch.int32, device="cuda")
    new_mass = torch.full((case.batch, keep + 5), -9.0, device="cuda") if with_mass else None
    lens = torch.full((case.batch,), -9, dtype=torch.int32, device="cuda")
    ws = binding.workspace(binding.cache_evict_workspace_size(case.batch, dc.batch.max_seq_len, keep))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.cache_evict(dc.cache, dc.batch, mass, keep, sink, recent, dst, dst_table, kept, new_mass, lens, ws, st,
                        stream=stream)
    torch.cuda.synchronize()
    return dict(dst=dst, table=dst_table, before=before, kept=kept.cpu().numpy(),
                mass=new_mass.cpu().numpy() if with_mass else None, lens=lens.cpu().numpy(), status=st.item())


def parts(case, cache):
    """(source offset, destination offset, bytes a token) of a row's record arrays."""
    code = case.token_bytes() - 4
    return [(case.latent_off, cache.latent_off, case.latent_bytes()), (case.index_off, cache.index_off, code),
            (case.index_off + 64 * code, cache.index_off + 64 * code, 4)]


def check_evict(case, mass, keep, sink, recent, r):
    m = mass.cpu().numpy()
    want = r["before"].copy()
    table = r["table"].cpu().numpy()
    for b in range(case.batch):
        L = int(case.seq_lens[b])
        tok = plain_kept(m[b], L, keep, sink, recent)
        n = len(tok)
        assert r["lens"][b] == n
        np.testing.assert_array_equal(r["kept"][b], tok + [-1] * (keep - n))
        if r["mass"] is not None:
            np.testing.assert_array_equal(r["mass"][b, :n], m[b][tok])
            assert np.all(r["mass"][b, n:] == 0)
        for i, t in enumerate(tok):
            src, dst = case.block_table[b, t // 64], table[b, i // 64]
            for so, do, size in parts(case, r["dst"]):
                want[dst, do + i % 64 * size:do + (i % 64 + 1) * size] = \
                    case.pool[src, so + t % 64 * size:so + (t % 64 + 1) * size]
    np.testing.assert_array_equal(r["dst"].pool.cpu().numpy(), want)   # the records, and nothing else


def totals(batch, n, kind, seed=0):
    rng = np.random.default_rng(seed)
    m = np.exp(2 * rng.standard_normal((batch, n))).astype(np.float32)
    if kind == "ties":
        m = np.floor(m).astype(np.float32)
    elif kind == "equal":
        m[:] = 0.25
    elif kind == "odd":
        pick = rng.integers(0, 8, m.shape)
        m = np.select([pick == 0, pick == 1, pick == 2, pick == 3, pick == 4],
                      [np.float32("nan"), np.float32("inf"), -np.float32("inf"), -np.float32(0), -m], m).astype(np.float32)
        m[rng.integers(0, 5, m.shape) == 0] = 0.0
    return torch.from_numpy(m).cuda()


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
@pytest.mark.parametrize("lens,keep,sink,recent", [([100, 37, 0, 64, 1], 40, 3, 10), ([65, 66, 64, 63], 64, 0, 0),
                                                   ([500, 129], 128, 64, 64), ([5001, 2100, 9000], 2000, 4, 100),
                                                   ([300, 2], 1, 0, 0), ([300, 2], 1, 1, 0), ([1000], 77, 0, 77)])
def test_evict_matches_plain(kind, lens, keep, sink, recent):
    case = synth.make_case("evict", seq_lens=lens, seed=400 + keep, key_format=synth.KEY_MXFP4, latent_format=NV)
    mass = totals(case.batch, case.max_len + 2, kind, keep)
    r = evict(case, synth.device_case(case), mass, keep, sink, recent)
    assert r["status"] == 0
    check_evict(case, mass, keep, sink, recent, r)


@pytest.mark.parametrize("key,fmt", [(synth.KEY_FP8, FP8), (synth.KEY_FP8, NV), (synth.KEY_MXFP4, FP8),
                                     (synth.KEY_MXFP4_NATIVE, NV)])
def test_evict_formats(key, fmt):
    case = synth.make_case("evict_fmt", seq_lens=[400, 150], seed=16, key_format=key, latent_format=fmt)
    mass = totals(2, case.max_len, "ties", 1)
    r = evict(case, synth.device_case(case), mass, 150, 5, 20, with_mass=False)
    assert r["status"] == 0
    check_evict(case, mass, 150, 5, 20, r)


@pytest.mark.parametrize("kind", ["plain", "ties", "equal"])
def test_evict_long_sequences(kind):
    """Every cluster size's worth of tokens a sequence, and shares that end inside the protected ranges."""
    for lens, keep, sink, recent in (([70001, 33000], 5000, 4000, 900), ([9000, 16385], 8000, 10, 7000)):
        case = synth.make_case("evict_long", seq_lens=lens, seed=17, key_format=synth.KEY_MXFP4, latent_format=NV)
        mass = totals(2, case.max_len, kind, 2)
        r = evict(case, synth.device_case(case), mass, keep, sink, recent)
        assert r["status"] == 0
        check_evict(case, mass, keep, sink, recent, r)


@pytest.mark.parametrize("lens,width", [([800_001], 800_001), ([50_000] + [70, 0, 300] * 53, 50_000),
                                        ([200_000, 7, 150_001], 720_897)])
def test_evict_with_totals_too_many_for_shared_memory(lens, width):
    """Contexts (or bounds) whose shares a CTA does not keep on chip: one sequence over the largest cluster, and more
    sequences than SMs.  The table lists a few pages over and over."""
    case = synth.make_case("evict_wide", seq_lens=[640] * len(lens), seed=30, key_format=synth.KEY_MXFP4, latent_format=NV)
    table = np.take(case.block_table, np.arange(-(-width // 64)) % 10, axis=1)
    case = dataclasses.replace(case, seq_lens=np.array(lens, dtype=np.int32), block_table=np.ascontiguousarray(table))
    dc = synth.device_case(case)
    dc.batch.max_seq_len = width
    mass = totals(case.batch, width, "ties", 7)
    r = evict(case, dc, mass, 1000, 9, 130)
    assert r["status"] == 0
    check_evict(case, mass, 1000, 9, 130, r)


def test_two_calls_at_once():
    """The three calls of two batches on two streams at the same time, each with its own workspaces."""
    cases = [synth.make_case("at_once", seq_lens=[9000, 400, 2500], nq=nq, seed=31 + nq, latent_format=fmt)
             for nq, fmt in ((1, NV), (3, FP8))]
    steps, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for case in cases:
        rows, keep = case.rows, 500
        dc = synth.device_case(case)
        rec, key = case.latent_bytes(), case.token_bytes()
        pool = torch.zeros((24, 64 * (rec + key)), dtype=torch.uint8, device="cuda")
        dst = binding.PagedCache(pool, pool.shape[1], 0, 64 * rec, case.key_format, case.latent_scale, case.latent_format)
        steps.append(dict(case=case, dc=dc, dst=dst, pool=pool, keep=keep,
                          out=torch.zeros((rows, 96, 512), dtype=torch.bfloat16, device="cuda"),
                          lse=torch.zeros((rows, 96), device="cuda"), mass=torch.zeros((3, 9000), device="cuda"),
                          table=torch.arange(24, dtype=torch.int32, device="cuda").view(3, 8),
                          kept=torch.zeros((3, keep), dtype=torch.int32, device="cuda"),
                          lens=torch.zeros(3, dtype=torch.int32, device="cuda"),
                          st=torch.zeros(1, dtype=torch.int32, device="cuda"),
                          w=[binding.workspace(n) for n in (binding.dense_mla_workspace_size(rows, 9000),
                                                            binding.attention_mass_workspace_size(rows, 9000, 0),
                                                            binding.cache_evict_workspace_size(3, 9000, keep))]))

    def run(s, stream):
        dc, scale = s["dc"], s["case"].sm_scale
        binding.dense_mla_decode(dc.cache, dc.batch, dc.q_mla, scale, s["out"], s["lse"], s["w"][0], s["st"], stream=stream)
        binding.attention_mass(dc.cache, dc.batch, dc.q_mla, s["lse"], scale, None, s["mass"], s["w"][1], s["st"],
                               stream=stream)
        binding.cache_evict(dc.cache, dc.batch, s["mass"], s["keep"], 2, 30, s["dst"], s["table"], s["kept"], None,
                            s["lens"], s["w"][2], s["st"], stream=stream)

    def results(s):
        assert s["st"].item() == 0
        return [s[n].clone() for n in ("out", "lse", "mass", "kept", "lens", "pool")]

    alone = []
    for s in steps:
        run(s, torch.cuda.current_stream())
        torch.cuda.synchronize()
        alone.append(results(s))
    for s in steps:
        for n in ("out", "lse", "mass", "kept", "lens", "pool"):
            s[n].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, stream in zip(steps, streams):
            run(s, stream)
    torch.cuda.synchronize()
    for s, want in zip(steps, alone):
        for a, b in zip(results(s), want):
            assert torch.equal(a, b)


def test_evict_into_spare_pages_of_the_same_pool():
    case = synth.make_case("evict_same", seq_lens=[300, 500], seed=18, spare_blocks=6)
    dc = synth.device_case(case)
    used = set(case.block_table[case.block_table >= 0].tolist())
    spare = [i for i in range(case.num_blocks) if i not in used]
    table = torch.tensor(spare, dtype=torch.int32).view(2, 3).cuda()
    mass = totals(2, 500, "plain", 3)
    r = evict(case, dc, mass, 192, 1, 64, dst=dc.cache, dst_table=table)
    assert r["status"] == 0
    check_evict(case, mass, 192, 1, 64, r)


def test_evict_reports_bad_pages_and_lengths():
    case = synth.make_case("evict_bad", seq_lens=[300, 200], seed=19)
    mass = totals(2, 300, "plain", 4)
    dc = synth.device_case(case)
    dc.batch.block_table[0, 1] = case.num_blocks
    assert evict(case, dc, mass, 250, 250, 0)["status"] == BOUNDS       # a kept token's page
    dc = synth.device_case(case)
    bad = torch.tensor([[0, 1], [2, 99]], dtype=torch.int32).cuda()
    assert evict(case, dc, mass, 128, 0, 0, dst_table=bad)["status"] == BOUNDS
    for length in (301, -1):
        dc = synth.device_case(case)
        dc.batch.seq_lens[1] = length
        r = evict(case, dc, mass, 128, 0, 0)
        assert r["status"] == BOUNDS and r["lens"][1] == 0 and np.all(r["kept"][1] == -1)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("sparse", [False, True])
def test_attend_weigh_evict_and_go_on(sparse):
    """Attention, its weights added up, eviction, and the next step on the smaller cache: the dense attention over
    the moved cache against the plain form over the kept tokens, the indexer's scores bit for bit those of the kept
    tokens, and a fused decode step that runs on it."""
    lens, keep = [1500, 700, 90], 300
    case = synth.make_case("together", seq_lens=lens, seed=20, key_format=synth.KEY_FP8, latent_format=NV)
    dc = synth.device_case(case)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if sparse:
        k = 512
        out = torch.empty((3, 96, 512), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((3, 96), device="cuda")
        idx = torch.empty((3, k), dtype=torch.int32, device="cuda")
        ws = binding.workspace(binding.workspace_size(dc.batch, k))
        binding.decode_step(dc.cache, dc.batch, dc.q_index, dc.head_w, dc.q_mla, k, case.sm_scale, out, lse, ws, st,
                            idx_out=idx)
    else:
        idx = None
        out, lse, _ = run_dense(case, dc)
    mass = torch.zeros((3, 1504), device="cuda")
    ws = binding.workspace(binding.attention_mass_workspace_size(3, dc.batch.max_seq_len, 512 if sparse else 0))
    for _ in range(2):
        binding.attention_mass(dc.cache, dc.batch, dc.q_mla, lse, case.sm_scale, mass, mass, ws, st, idx=idx)
    torch.cuda.synchronize()
    assert st.item() == 0
    # a row's softmax weights sum to one per head, twice
    np.testing.assert_allclose(mass.sum(1).cpu().numpy(), 2 * 96.0, rtol=1e-4)
    r = evict(case, dc, mass, keep, 4, 32)
    assert r["status"] == 0
    check_evict(case, mass, keep, 4, 32, r)
    small = binding.Batch(r["table"], torch.from_numpy(r["lens"]).cuda(), 1, keep)
    o2 = torch.empty((3, 96, 512), dtype=torch.bfloat16, device="cuda")
    l2 = torch.empty((3, 96), device="cuda")
    ws = binding.workspace(binding.dense_mla_workspace_size(3, keep))
    binding.dense_mla_decode(r["dst"], small, dc.q_mla, case.sm_scale, o2, l2, ws, st)
    s_old = torch.empty((3, 1504), device="cuda")
    s_new = torch.empty((3, 304), device="cuda")
    binding.index_scores(dc.cache, dc.batch, dc.q_index, dc.head_w, s_old, st)
    binding.index_scores(r["dst"], small, dc.q_index, dc.head_w, s_new, st)
    o3, l3 = torch.empty_like(o2), torch.empty_like(l2)
    ws = binding.workspace(binding.workspace_size(small, 2048))
    binding.decode_step(r["dst"], small, dc.q_index, dc.head_w, dc.q_mla, 2048, case.sm_scale, o3, l3, ws, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for b in range(3):
        n = int(r["lens"][b])
        tok = torch.from_numpy(r["kept"][b, :n].astype(np.int64))
        ro, rl, av, spread, bound = plain64.attend(case, b, tok)
        e = 576 * 2.0 ** -24 * bound
        tol = 2.0 ** -8 * (1 + 2.0 ** -7) * spread + (2 * e[:, None] + 2 * n * 2.0 ** -24 + 2.0 ** -11) * av + 2.0 ** -8 * ro.abs()
        for o, l in ((o2, l2), (o3, l3)):   # 2,048 covers the budget: the step attends to every kept token too
            assert torch.all((o[b].double().cpu() - ro).abs() <= tol)
            assert torch.all((l[b].double().cpu() - rl).abs() <= e + n * 2.0 ** -24 + 2.0 ** -20 * (1 + rl.abs()))
        assert torch.equal(s_new[b, :n].cpu(), s_old[b].cpu()[tok])


def test_calls_on_a_stream_and_in_a_graph():
    """The three calls on a side stream, and captured once and replayed on other inputs."""
    case = synth.make_case("graph", seq_lens=[900, 400], nq=2, seed=21, latent_format=NV)
    dc = synth.device_case(case)
    keep = 200
    out = torch.empty((4, 96, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((4, 96), device="cuda")
    mass = torch.zeros((2, 900), device="cuda")
    rec, key = case.latent_bytes(), case.token_bytes()
    pool = torch.zeros((8, 64 * (rec + key)), dtype=torch.uint8, device="cuda")
    dst = binding.PagedCache(pool, pool.shape[1], 0, 64 * rec, case.key_format, case.latent_scale, case.latent_format)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    kept = torch.empty((2, keep), dtype=torch.int32, device="cuda")
    lens = torch.empty(2, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    w1 = binding.workspace(binding.dense_mla_workspace_size(4, 900))
    w2 = binding.workspace(binding.attention_mass_workspace_size(4, 900, 0))
    w3 = binding.workspace(binding.cache_evict_workspace_size(2, 900, keep))

    def step(stream):
        binding.dense_mla_decode(dc.cache, dc.batch, dc.q_mla, case.sm_scale, out, lse, w1, st, stream=stream)
        binding.attention_mass(dc.cache, dc.batch, dc.q_mla, lse, case.sm_scale, None, mass, w2, st, stream=stream)
        binding.cache_evict(dc.cache, dc.batch, mass, keep, 2, 30, dst, table, kept, None, lens, w3, st, stream=stream)

    def results():
        torch.cuda.synchronize()
        assert st.item() == 0
        return [t.clone() for t in (out, lse, mass, kept, lens, pool)]

    step(torch.cuda.current_stream())
    first = results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (out, lse, mass, kept, lens, pool):
        t.zero_()
    torch.cuda.synchronize()
    step(side)
    for a, b in zip(first, results()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    q = dc.q_mla.clone()
    for turn in range(3):
        dc.q_mla.copy_(q.roll(turn, 0))
        dc.batch.seq_lens.copy_(torch.tensor([900 - 100 * turn, 400 - 7 * turn], dtype=torch.int32))
        for t in (out, lse, mass, kept, lens, pool):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        replayed = results()
        for t in (out, lse, mass, kept, lens, pool):
            t.zero_()
        torch.cuda.synchronize()
        step(torch.cuda.current_stream())
        for a, b in zip(replayed, results()):
            assert torch.equal(a, b)
