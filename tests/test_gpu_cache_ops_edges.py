"""dense_mla_decode and dsa_attention_mass where single heads, rows, pages or
entries are out of the ordinary: what is wrong with one of them stays there.

Tolerance of the attention, from the roundings on the way (half a step of bf16
is 2^-8 relative, of fp16 2^-11, of fp32 2^-24; p is normalised, sums over the
row's n tokens):
  logits   fp32 sums of 576 exact products and the scaled argument of the
           exponential, 576 * 2^-24 * Sum |q c| * sm_scale =: e; they move the
           quotient by at most 2 e * Sum p |v|
  P        fp16 in the numerator only, 2^-11 * Sum p |v|; below 2^-14 its step is
           fixed, half of it 2^-25 against a normaliser of at least 2^7 (the
           largest weight is stored as 2^7 or more): 2^-32 * Sum |v|
  sums     fp32, n * 2^-24 * Sum p |v| for the values and as much for the normaliser
  parts    fp16, 2^-11 * Sum p |v|, and 2^-25 of a latent unit below 2^-14
  output   bf16, 2^-8 of the computed value
  LSE      e + n * 2^-24 + 2^-20 * (1 + |lse|)
A head's query is bf16 times a power of two of its own: exact down to 2^-28 of the
head's largest element.
"""
import dataclasses

import numpy as np
import pytest
import torch

import plain64
from dsa_sparse_attention_index_gb300 import binding, synth
from test_gpu_cache_eviction import plain_lse, plain_mass, run_mass
from test_gpu_dense_mla import run_dense

pytestmark = pytest.mark.gpu

FP8, NV = synth.LATENT_FP8, synth.LATENT_NVFP4
HEAD = 5   # the head that is out of the ordinary


def bf16_bits(x):
    return x.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def check(case, out, lse, heads=None, rows=None, tokens=None):
    """Rows of the attention against 64 bits; tokens(row) lists what a row attends to (None: all it sees)."""
    heads = torch.arange(96) if heads is None else torch.as_tensor(heads)
    o, l = out.double().cpu(), lse.double().cpu()
    cached = {}
    for row in range(case.rows) if rows is None else rows:
        b = row // case.nq
        if b not in cached:
            cached = {b: plain64.latents(case, b)}
        vis = max(0, int(case.seq_lens[b]) - (case.nq - 1) + row % case.nq)
        see = torch.arange(vis) if tokens is None else tokens(row)
        n = len(see)
        if n == 0:
            assert torch.all(o[row] == 0) and torch.all(torch.isneginf(l[row])), row
            continue
        ro, rl, av, _, bound = plain64.attend(case, row, see, c=cached[b])
        sum_v = cached[b][see][:, :512].abs().sum(0)[None, :]
        e = (576 * 2.0 ** -24 * bound)[:, None]
        err = ((2 * e + 2 * n * 2.0 ** -24 + 2 * 2.0 ** -11) * av + 2.0 ** -32 * sum_v
               + 2.0 ** -25 * case.latent_scale)
        tol = err + 2.0 ** -8 * (ro.abs() + err)
        bad = ((o[row] - ro).abs() - tol)[heads]
        assert not torch.isnan(bad).any() and bad.max().item() <= 0, f"row {row}, {n} tokens: out off by {bad.max().item()}"
        ltol = e[:, 0] + n * 2.0 ** -24 + 2.0 ** -20 * (1 + rl.abs())
        assert torch.all(((l[row] - rl).abs() <= ltol)[heads]), f"row {row}: lse"


OTHERS = [h for h in range(96) if h != HEAD]


# ---------------------------------------------------------------- the tolerance itself
@pytest.mark.parametrize("fmt", [FP8, NV])
@pytest.mark.parametrize("lens,nq", [([1, 47, 48, 49, 0], 1), ([3000, 130], 1), ([20001], 1), ([700, 2049], 4)])
def test_dense_within_the_roundings_of_its_own_arithmetic(fmt, lens, nq):
    case = synth.make_case("edge_tol", seq_lens=lens, nq=nq, seed=500 + len(lens) + nq, latent_format=fmt)
    out, lse, st = run_dense(case, synth.device_case(case))
    assert st == 0
    check(case, out, lse)


@pytest.mark.parametrize("fmt", [FP8, NV])
def test_dense_weights_keep_eleven_bits(fmt):
    """Two tokens of opposite values and nearly equal weights: the output is the weights' small difference, and a
    weight held in bf16's 8 bits would be seen."""
    case = synth.make_case("edge_bits", seq_lens=[2], seed=515, latent_format=fmt)
    rec, at = case.latent_bytes(), case.latent_off
    pool = case.pool.copy()
    row = pool[case.block_table[0, 0], at:at + 2 * rec].reshape(2, rec)
    row[:, rec - 64:] = 0                      # no key-only dimensions
    row[1] = row[0]
    row[1, :512 if fmt == FP8 else 256] ^= 0x80 if fmt == FP8 else 0x88
    pool[case.block_table[0, 0], at:at + 2 * rec] = row.reshape(-1)
    q = 0.05 * torch.randn((1, 96, 576), generator=torch.Generator().manual_seed(4))
    case = dataclasses.replace(case, pool=pool, q_mla=bf16_bits(q))
    c = plain64.latents(case, 0)
    ro, rl, av, _, bound = plain64.attend(case, 0, c=c)
    err = (2 * 576 * 2.0 ** -24 * bound[:, None] + 4 * 2.0 ** -24 + 2.0 ** -11) * av + 2.0 ** -31 * c.abs().max()
    tol = err + 2.0 ** -8 * (ro.abs() + err)   # one part, so no rounding of parts
    x = plain64.queries(case, 0) @ c.T * case.sm_scale
    p = torch.exp(x - x.amax(1, keepdim=True))
    in8 = (p * 128).to(torch.bfloat16).double() / 128 @ c[:, :512] / p.sum(1, keepdim=True)
    assert bool(((in8 - ro).abs() > tol).any())
    out, lse, st = run_dense(case, synth.device_case(case))
    assert st == 0
    assert torch.all((out[0].double().cpu() - ro).abs() <= tol)


# ---------------------------------------------------------------- infinities and NaN
def constant_dim(case, kind):
    """Latent dimension 550 (E4M3 in either format) of every token: 1.0; "first": 1.0 in each tile's first token
    and 0 in the others."""
    rec = case.latent_bytes()
    pool = case.pool.copy()
    at = case.latent_off + (550 if rec == 576 else 288 + 550 - 512)
    for b in range(case.batch):
        for t in range(int(case.seq_lens[b])):
            one = kind == "same" or t % 48 == 0
            pool[case.block_table[b, t // 64], at + t % 64 * rec] = 0x38 if one else 0
    return dataclasses.replace(case, pool=pool)


@pytest.mark.parametrize("fmt", [FP8, NV])
@pytest.mark.parametrize("kind", ["same", "first"])
@pytest.mark.parametrize("bits,sign", [(0x7F80, 1), (0xFF80, 1), (0x7F80, -1), (0xFF80, -1), (0x7FC0, 1)])
def test_dense_infinite_query_whose_products_share_a_sign(fmt, kind, bits, sign):
    """inf - inf is NaN whatever the sign: one token, one tile, several tiles and several parts."""
    lens = [1, 2, 48, 60, 7000]
    case = constant_dim(synth.make_case("edge_inf", seq_lens=lens, seed=501, latent_format=fmt), kind)
    q = case.q_mla.copy()
    q[:, HEAD, 550] = bits
    case = dataclasses.replace(case, q_mla=q, sm_scale=sign * case.sm_scale)
    out, lse, st = run_dense(case, synth.device_case(case))
    assert st == 0
    assert bool(torch.isnan(out[:, HEAD].float()).all()) and bool(torch.isnan(lse[:, HEAD]).all())
    clean = case.q_mla.copy()
    clean[:, HEAD, 550] = 0
    check(dataclasses.replace(case, q_mla=clean), out, lse, heads=OTHERS)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_dense_scale_that_is_no_number(scale):
    """NaN for every row that sees a token; a row that sees none stays as documented."""
    case = dataclasses.replace(synth.make_case("edge_scale", seq_lens=[300, 0, 1], seed=502, latent_format=NV), sm_scale=scale)
    out, lse, st = run_dense(case, synth.device_case(case))
    assert st == 0
    for row in (0, 2):
        assert bool(torch.isnan(out[row].float()).all()) and bool(torch.isnan(lse[row]).all())
    assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))


# ---------------------------------------------------------------- heads of very different size
@pytest.mark.parametrize("fmt", [FP8, NV])
@pytest.mark.parametrize("power", [28, 34, 45, 60, 100])
def test_dense_one_head_far_above_the_others(fmt, power):
    """A finite outlier in one head takes nothing from the other heads of its row."""
    case = synth.make_case("edge_far", seq_lens=[700, 48, 6000], seed=503, latent_format=fmt)
    q = torch.randn((3, 96, 576), generator=torch.Generator().manual_seed(power))
    q[:, HEAD, 17] = 2.0 ** power
    case = dataclasses.replace(case, q_mla=bf16_bits(q))
    out, lse, st = run_dense(case, synth.device_case(case))
    assert st == 0
    check(case, out, lse, heads=OTHERS)


@pytest.mark.parametrize("fmt", [FP8, NV])
@pytest.mark.parametrize("power", [16, 24, 30, 45, 60, 100])
def test_dense_logits_beyond_the_steps_of_fp32(fmt, power):
    """Logits whose fp32 steps exceed 1, up to 2^100: one token takes a head, and it is the largest one's value."""
    case = synth.make_case("edge_steep", seq_lens=[700, 48, 6000], seed=509, latent_format=fmt)
    q = torch.randn((3, 96, 576), generator=torch.Generator().manual_seed(power)) * 2.0 ** power
    case = dataclasses.replace(case, q_mla=bf16_bits(q))
    out, lse, st = run_dense(case, synth.device_case(case))
    assert st == 0
    check(case, out, lse)   # this tolerance grows with the logits
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
    for b in range(3):
        c = plain64.latents(case, b)
        x = plain64.queries(case, b) @ c.T * case.sm_scale
        top, runner = x.topk(2, 1).values.T
        # where the runner-up is further behind than the logits' error, and 6,000 of its weight vanish
        bound = (plain64.queries(case, b).abs() @ c.abs().T * case.sm_scale).amax(1)
        clear = top - runner > 2 * 576 * 2.0 ** -24 * bound + 30
        assert bool(clear.any())
        v = c[x.argmax(1)][:, :512]
        tol = 2.0 ** -8 * v.abs() + 2.0 ** -11 * v.abs() + 2.0 ** -20 * c.abs().max()
        assert torch.all(((out[b].double().cpu() - v).abs() <= tol)[clear]), b


@pytest.mark.parametrize("fmt", [FP8, NV])
@pytest.mark.parametrize("power", [28, 34, 45, 60, 100])
@pytest.mark.parametrize("nq,k", [(1, 0), (3, 0), (1, 200)])
def test_mass_one_head_far_above_the_others(fmt, power, nq, k):
    """The same for the weights; the outlier's own LSE is set so high that it adds nothing."""
    case = synth.make_case("edge_mass_far", seq_lens=[700, 140], nq=nq, seed=504, latent_format=fmt)
    idx = None
    if k:
        g = torch.Generator().manual_seed(k)
        idx = torch.full((case.rows, k), -1, dtype=torch.int32)
        for r, vis in enumerate(case.row_lens()):
            idx[r, :min(k, int(vis))] = torch.randperm(int(vis), generator=g)[:k].to(torch.int32)
    q = torch.randn((case.rows, 96, 576), generator=torch.Generator().manual_seed(power))
    q[:, HEAD, 17] = 2.0 ** power
    case = dataclasses.replace(case, q_mla=bf16_bits(q))
    lse = plain_lse(case, idx)
    lse[:, HEAD] = 1e38
    before = torch.rand((2, case.max_len + 3), generator=torch.Generator().manual_seed(3))
    want, tol = plain_mass(case, before, lse, idx)
    got, st = run_mass(case, synth.device_case(case), lse, before, idx)
    assert st == 0
    for b, L in enumerate(case.seq_lens):
        assert torch.all((got[b, :L].double() - want[b, :L]).abs() <= tol[b, :L]), b


# ---------------------------------------------------------------- bad pages and entries
def seen(case, table):
    def tokens(row):
        b = row // case.nq
        t = torch.arange(max(0, int(case.seq_lens[b]) - (case.nq - 1) + row % case.nq))
        page = torch.from_numpy(table[b].astype(np.int64))[t // 64]
        return t[(page >= 0) & (page < case.num_blocks)]
    return tokens


@pytest.mark.parametrize("fmt", [FP8, NV])
@pytest.mark.parametrize("bad", [-1, 1 << 30, None])
def test_dense_bad_pages_take_no_part(fmt, bad):
    """The tokens of a page outside the pool are masked, in the first, an inner, the last and every page."""
    case = synth.make_case("edge_page", seq_lens=[40, 500, 300, 130, 6000, 64, 190], nq=2, seed=505, latent_format=fmt)
    table = case.block_table.copy()
    bad = case.num_blocks if bad is None else bad
    table[0, 0] = table[1, 0] = table[2, 2] = table[3, 2] = bad
    table[4, 5:9] = table[4, 40] = table[4, 93] = bad
    table[6, :3] = bad
    out, lse, st = run_dense(case, synth.device_case(dataclasses.replace(case, block_table=table)))
    assert st == binding.ERR_BOUNDS
    check(case, out, lse, tokens=seen(case, table))


@pytest.mark.parametrize("fmt", [FP8, NV])
@pytest.mark.parametrize("nq", [1, 3])
def test_mass_bad_pages_add_nothing(fmt, nq):
    case = synth.make_case("edge_mass_page", seq_lens=[40, 500, 1300], nq=nq, seed=506, latent_format=fmt)
    table = case.block_table.copy()
    table[0, 0], table[1, 3], table[2, 20] = -1, case.num_blocks, 1 << 30
    tokens = seen(case, table)
    lse = torch.stack([plain64.attend(case, r, tokens(r))[1] for r in range(case.rows)]).float()
    lse[:nq] = 0.0   # nothing attended; a finite LSE all the same
    before = torch.rand((3, case.max_len + 3), generator=torch.Generator().manual_seed(5))
    listed = torch.full((case.rows, case.max_len), -1, dtype=torch.int32)
    for r in range(case.rows):
        listed[r, :len(tokens(r))] = tokens(r).to(torch.int32)
    want, tol = plain_mass(case, before, lse, listed)
    got, st = run_mass(case, synth.device_case(dataclasses.replace(case, block_table=table)), lse, before)
    assert st == binding.ERR_BOUNDS
    for b, L in enumerate(case.seq_lens):
        assert torch.all((got[b, :L].double() - want[b, :L]).abs() <= tol[b, :L]), b


@pytest.mark.parametrize("fmt", [FP8, NV])
def test_mass_bad_entries_add_nothing(fmt):
    """Entries behind what their row sees, below and above the sequence's length, and on a bad page."""
    case = synth.make_case("edge_entries", seq_lens=[500, 200], nq=2, seed=507, latent_format=fmt)
    table = case.block_table.copy()
    table[1, 1] = -1
    idx = torch.full((4, 150), -1, dtype=torch.int32)
    for r, vis in enumerate(case.row_lens()):
        idx[r, :120] = torch.randperm(int(vis), generator=torch.Generator().manual_seed(r))[:120].to(torch.int32)
    good = idx.clone()
    idx[0, 3], idx[0, 130], idx[1, 149], idx[2, 7] = 499, 499, 1 << 30, 199   # row 0 sees 499 tokens, row 2 199
    good[0, 3], good[2, 7] = -1, -1
    good[2:][(good[2:] >= 64) & (good[2:] < 128)] = -1
    lse = plain_lse(case, good)
    before = torch.rand((2, case.max_len + 3), generator=torch.Generator().manual_seed(6))
    want, tol = plain_mass(case, before, lse, good)
    got, st = run_mass(case, synth.device_case(dataclasses.replace(case, block_table=table)), lse, before, idx)
    assert st == binding.ERR_BOUNDS
    for b, L in enumerate(case.seq_lens):
        assert torch.all((got[b, :L].double() - want[b, :L]).abs() <= tol[b, :L]), b


@pytest.mark.parametrize("fmt", [FP8, NV])
@pytest.mark.parametrize("nq", [1, 2])
def test_mass_rows_that_attended_to_nothing_over_unwritten_pages(fmt, nq):
    """A row whose LSEs are all -inf adds nothing, whatever lies in its pages (NaN codes here)."""
    case = synth.make_case("edge_unwritten", seq_lens=[300, 200], nq=nq, seed=508, latent_format=fmt)
    lse = plain_lse(case)
    pool = case.pool.copy()
    for page in case.block_table[1][case.block_table[1] >= 0]:
        pool[page, case.latent_off:case.latent_off + 64 * case.latent_bytes()] = 0x7F
    lse[nq:] = -float("inf")
    before = torch.rand((2, case.max_len + 3), generator=torch.Generator().manual_seed(7))
    want, tol = plain_mass(case, before, lse)
    got, st = run_mass(dataclasses.replace(case, pool=pool), synth.device_case(dataclasses.replace(case, pool=pool)), lse,
                       before)
    assert st == 0
    assert torch.equal(got[1, :200], before[1, :200])
    assert torch.all((got[0, :300].double() - want[0, :300]).abs() <= tol[0, :300])


# ---------------------------------------------------------------- sizes and bounds
def loose(dc, blocks):
    """The same batch under a table and a bound far beyond its lengths, as a captured graph has them."""
    table = torch.full((dc.batch.batch, blocks), -1, dtype=torch.int32, device="cuda")
    table[:, :dc.batch.block_table.shape[1]] = dc.batch.block_table
    dc.batch.block_table, dc.batch.max_seq_len = table, 64 * blocks
    return dc


@pytest.mark.parametrize("invariant", [False, True])
def test_dense_prompt_chunk_of_2048_rows(invariant):
    case = synth.make_case("edge_chunk", seq_lens=[4300], nq=2048, seed=510, latent_format=NV)
    prev = binding.batch_invariant(invariant)
    try:
        out, lse, st = run_dense(case, synth.device_case(case))
    finally:
        binding.batch_invariant(prev)
    assert st == 0
    check(case, out, lse, rows=[0, 1, 479, 480, 1023, 1587, 1588, 2047])


@pytest.mark.parametrize("fmt", [FP8, NV])
def test_dense_context_of_150001_tokens(fmt):
    case = synth.make_case("edge_long", seq_lens=[150_001], seed=511, latent_format=fmt)
    out, lse, st = run_dense(case, synth.device_case(case))
    assert st == 0
    check(case, out, lse)


@pytest.mark.parametrize("invariant", [False, True])
def test_dense_under_a_loose_bound(invariant):
    case = synth.make_case("edge_loose", seq_lens=[700, 0, 4100], nq=2, seed=512, latent_format=NV)
    prev = binding.batch_invariant(invariant)
    try:
        out, lse, st = run_dense(case, loose(synth.device_case(case), 2048))
    finally:
        binding.batch_invariant(prev)
    assert st == 0
    check(case, out, lse)


@pytest.mark.parametrize("nq,k", [(1, 0), (3, 0), (1, 150), (3, 150)])
def test_mass_under_a_loose_bound(nq, k):
    case = synth.make_case("edge_mass_loose", seq_lens=[700, 5, 4100], nq=nq, seed=513, latent_format=NV)
    idx = None
    if k:
        idx = torch.full((case.rows, k), -1, dtype=torch.int32)
        for r, vis in enumerate(case.row_lens()):
            n = min(k, int(vis))
            idx[r, :n] = torch.randperm(int(vis), generator=torch.Generator().manual_seed(r))[:n].to(torch.int32)
    lse = plain_lse(case, idx)
    before = torch.rand((3, 64 * 2048 + 5), generator=torch.Generator().manual_seed(8))
    want, tol = plain_mass(case, before, lse, idx)
    got, st = run_mass(case, loose(synth.device_case(case), 2048), lse, before, idx, in_place=True)
    assert st == 0
    for b, L in enumerate(case.seq_lens):
        assert torch.all((got[b, :L].double() - want[b, :L]).abs() <= tol[b, :L]), b
        assert torch.equal(got[b, L:], before[b, L:])


@pytest.mark.parametrize("nq,k", [(512, 0), (300, 40)])
def test_mass_of_a_prompt_chunk(nq, k):
    case = synth.make_case("edge_mass_chunk", seq_lens=[900, 310], nq=nq, seed=514, latent_format=NV)
    idx = None
    if k:
        idx = torch.full((case.rows, k), -1, dtype=torch.int32)
        for r, vis in enumerate(case.row_lens()):
            n = min(k, int(vis))
            idx[r, :n] = torch.randperm(int(vis), generator=torch.Generator().manual_seed(r))[:n].to(torch.int32)
    lse = plain_lse(case, idx)
    before = torch.rand((2, case.max_len + 3), generator=torch.Generator().manual_seed(9))
    want, tol = plain_mass(case, before, lse, idx)
    got, st = run_mass(case, synth.device_case(case), lse, before, idx)
    assert st == 0
    for b, L in enumerate(case.seq_lens):
        assert torch.all((got[b, :L].double() - want[b, :L]).abs() <= tol[b, :L]), b
