"""dense_mla_decode (exact MLA over every visible token) against a plain
64-bit form, at lengths around pages and runs, both latent formats, ragged
batches, draft rows and prefill chunks, offsets and strides of the pool, and
its device-side refusals.

Tolerances, from the roundings on the way (half a step of bf16 is 2^-8
relative, of fp16 2^-11, of fp32 2^-24):
  logits   fp32 sums of 576 exact products: |dl| <= 576 * 2^-24 * Sum |q c| * sm_scale
           =: e (plus 2^-22 * |l| for the scaling and the exponential's argument,
           inside e as Sum |q c| >= |l|)
  P        rounded to bf16 on both sides of the quotient, which is normalised by the
           sum of the rounded values: Sum p |v - o| * 2^-8 * (1 + 2^-7)
  logits   move the quotient by at most 2 e * Sum p |v|
  sums     fp32 over n tokens, n * 2^-24 * Sum p |v| twice (values, normaliser)
  parts    fp16, 2^-11 * Sum p |v|;  output bf16, 2^-8 |o|
  LSE      e + n * 2^-24 + 2^-20 * (1 + |lse|)
"""
import dataclasses

import numpy as np
import pytest
import torch

import plain64
from dsa_sparse_attention_index_gb300 import binding, synth

pytestmark = pytest.mark.gpu

FP8, NV = synth.LATENT_FP8, synth.LATENT_NVFP4


def run_dense(case, dc, stream=None, ws=None):
    rows = case.rows
    out = torch.full((rows, 96, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, 96), float("nan"), dtype=torch.float32, device="cuda")
    if ws is None:
        ws = binding.workspace(binding.dense_mla_workspace_size(rows, dc.batch.max_seq_len))
        ws.fill_(255)   # NaN patterns wherever a part is read that was not written
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.dense_mla_decode(dc.cache, dc.batch, dc.q_mla, case.sm_scale, out, lse, ws, st, stream=stream)
    torch.cuda.synchronize()
    return out, lse, st.item()


def check_rows(case, out, lse, rows=None):
    o, l = out.double().cpu(), lse.double().cpu()
    cached = {}
    for row in range(case.rows) if rows is None else rows:
        b = row // case.nq
        if b not in cached:
            cached = {b: plain64.latents(case, b)}
        ro, rl, av, spread, bound = plain64.attend(case, row, c=cached[b])
        n = max(0, int(case.seq_lens[b]) - (case.nq - 1) + row % case.nq)
        if n == 0:
            assert torch.all(o[row] == 0) and torch.all(torch.isneginf(l[row]))
            continue
        e = (576 * 2.0 ** -24 * bound)[:, None]
        tol = 2.0 ** -8 * (1 + 2.0 ** -7) * spread + (2 * e + 2 * n * 2.0 ** -24 + 2.0 ** -11) * av + 2.0 ** -8 * ro.abs()
        excess = ((o[row] - ro).abs() - tol).max().item()
        assert excess <= 0, f"row {row}, {n} tokens: out off by {excess} more than {tol.max().item()}"
        ltol = e[:, 0] + n * 2.0 ** -24 + 2.0 ** -20 * (1 + rl.abs())
        assert torch.all((l[row] - rl).abs() <= ltol), f"row {row}: lse"


@pytest.mark.parametrize("fmt", [FP8, NV])
@pytest.mark.parametrize("lens,nq", [([1], 1), ([64], 1), ([65], 1), ([63, 0, 1, 130], 1), ([997], 1),
                                     ([129, 700, 2049], 4), ([2, 5, 66], 3), ([5000, 64, 20001, 1], 1),
                                     ([400], 64), ([100, 31], 32)])
def test_dense_mla_matches_plain(fmt, lens, nq):
    case = synth.make_case("dense", seq_lens=lens, nq=nq, seed=100 + len(lens) + nq, latent_format=fmt)
    out, lse, st = run_dense(case, synth.device_case(case))
    assert st == 0
    check_rows(case, out, lse)


def test_dense_mla_many_sequences():
    """More sequences than SMs, so a CTA's run holds several rows and a row crosses CTAs."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 400, 333)
    case = synth.make_case("dense_many", seq_lens=lens, seed=7, latent_format=NV)
    out, lse, st = run_dense(case, synth.device_case(case))
    assert st == 0
    check_rows(case, out, lse)


def test_dense_mla_prefill_chunk():
    case = synth.make_case("dense_chunk", seq_lens=[1500], nq=512, seed=8, latent_format=NV)
    out, lse, st = run_dense(case, synth.device_case(case))
    assert st == 0
    check_rows(case, out, lse, rows=[0, 1, 63, 64, 255, 256, 300, 510, 511])


@pytest.mark.parametrize("fmt", [FP8, NV])
def test_dense_mla_sharp_heads(fmt):
    """Logits that grow along the context (the running maximum moves many times) and heads that one token takes."""
    case = synth.make_case("dense_sharp", seq_lens=[3000], seed=9, latent_format=fmt)
    q = torch.randn((1, 96, 576), generator=torch.Generator().manual_seed(1)) * torch.linspace(0.0, 60.0, 96)[None, :, None]
    case = dataclasses.replace(case, q_mla=q.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16))
    out, lse, st = run_dense(case, synth.device_case(case))
    assert st == 0
    check_rows(case, out, lse)


@pytest.mark.parametrize("fmt", [FP8, NV])
def test_dense_mla_single_tokens_are_bit_exact(fmt):
    """One token a row: out is its value rounded to bf16, for every E2M1 code under every E4M3 block scale (each in
    some sequence), and every E4M3 code."""
    n = 32
    case = synth.make_case("dense_one", seq_lens=[1] * n, seed=22, latent_format=fmt)
    rec = case.latent_bytes()
    codes = [c for c in range(256) if c & 0x7F != 0x7F]
    for b in range(n):
        if fmt == NV:
            r = np.zeros(352, dtype=np.uint8)
            r[:256] = [((i + b) % 16) | (((5 * i + 2) % 16) << 4) for i in range(256)]
            r[256:288] = [codes[(8 * b + i) % len(codes)] for i in range(32)]
            r[288:] = [codes[(3 * i + b) % len(codes)] for i in range(64)]
        else:
            r = np.array([codes[(i + 7 * b) % len(codes)] for i in range(576)], dtype=np.uint8)
        case.pool[case.block_table[b, 0], case.latent_off:case.latent_off + rec] = r
    for scale in (1.0, 0.75):
        one = dataclasses.replace(case, latent_scale=scale)
        out, lse, st = run_dense(one, synth.device_case(one))
        assert st == 0
        for b in range(n):
            v = (plain64.latents(case, b)[0, :512] / case.latent_scale).float() * np.float32(scale)
            assert torch.equal(out[b].float().cpu(), v.to(torch.bfloat16).float().expand(96, 512)), b


def test_dense_mla_layout_and_filler():
    """Index pages before the latent pages, padding between rows, and NaN codes in every slot behind a context."""
    case = synth.make_case("dense_layout", seq_lens=[70, 129], seed=10, key_format=synth.KEY_MXFP4, latent_format=NV,
                           spare_blocks=2)
    n, rec = case.num_blocks, 64 * 352
    pool = np.full((n, 384 + rec + 64 * 68 + 256), 0x7F, dtype=np.uint8)
    pool[:, 256 + 64 * 68 + 128:256 + 64 * 68 + 128 + rec] = case.pool[:, :rec]
    for b, L in enumerate([70, 129]):
        r = case.block_table[b, (L - 1) // 64]
        pool[r, 256 + 64 * 68 + 128 + (L % 64) * 352:256 + 64 * 68 + 128 + rec] = 0x7F
    moved = dataclasses.replace(case, pool=pool, row_stride=pool.shape[1], latent_off=256 + 64 * 68 + 128, index_off=256)
    out, lse, st = run_dense(moved, synth.device_case(moved))
    assert st == 0
    check_rows(moved, out, lse)


def test_dense_mla_invariant_mode():
    """In the batch-invariant mode a row's bits do not depend on its batch, and stay within the tolerance."""
    lens = [9000, 4097, 300]
    case = synth.make_case("dense_inv", seq_lens=lens, seed=11, latent_format=NV)
    prev = binding.batch_invariant(True)
    try:
        out, lse, st = run_dense(case, synth.device_case(case))
        assert st == 0
        check_rows(case, out, lse)
        for b in range(3):
            one = dataclasses.replace(case, batch=1, seq_lens=case.seq_lens[b:b + 1].copy(),
                                      block_table=case.block_table[b:b + 1].copy(), q_mla=case.q_mla[b:b + 1].copy(),
                                      q_index=case.q_index[b:b + 1].copy(), head_w=case.head_w[b:b + 1].copy())
            o1, l1, st = run_dense(one, synth.device_case(one))
            assert st == 0
            assert torch.equal(o1[0], out[b]) and torch.equal(l1[0], lse[b])
    finally:
        binding.batch_invariant(prev)


def test_dense_mla_invariant_mode_over_the_batch_size():
    """Bit for bit the same row alone, among a few and among many, with several parts a row."""
    case = synth.make_case("dense_inv", seq_lens=[20000, 12000, 3841], seed=33, latent_format=NV)
    try:
        binding.batch_invariant(True)
        alone = run_dense(case, synth.device_case(case))
        assert alone[2] == 0
        for copies in (6, 30):
            many = dataclasses.replace(case, batch=3 * copies, q_mla=np.tile(case.q_mla, (copies, 1, 1)),
                                       seq_lens=np.tile(case.seq_lens, copies),
                                       block_table=np.tile(case.block_table, (copies, 1)))
            dc = synth.device_case(many)
            out, lse, st = run_dense(many, dc)
            assert st == 0
            for i in range(copies):
                assert torch.equal(out[3 * i:3 * i + 3], alone[0]) and torch.equal(lse[3 * i:3 * i + 3], alone[1]), i
    finally:
        binding.batch_invariant(False)


def test_dense_mla_bad_page_is_reported():
    case = synth.make_case("dense_bad", seq_lens=[500, 300], seed=12)
    for bad in (case.num_blocks, -1, 1 << 30):
        table = case.block_table.copy()
        table[1, 2] = bad
        broken = dataclasses.replace(case, block_table=table)
        _, _, st = run_dense(broken, synth.device_case(broken))
        assert st == binding.ERR_BOUNDS


def test_dense_mla_lengths_outside_the_table():
    """A length above the table reads as the table's bound, a negative one as 0."""
    case = synth.make_case("dense_len", seq_lens=[128, 64], seed=13)
    dc = synth.device_case(case)
    dc.batch.seq_lens.copy_(torch.tensor([1 << 30, -5], dtype=torch.int32))
    out, lse, st = run_dense(case, dc)
    assert st == 0
    check_rows(case, out, lse, rows=[0])
    assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))


@pytest.mark.parametrize("scale", [-1.0 / 24, 0.0, 3.0])
def test_dense_mla_scales(scale):
    """A negative scale (the smallest products weigh most), none at all (uniform weights), and a large one."""
    case = dataclasses.replace(synth.make_case("dense_scale", seq_lens=[1000, 47, 49], seed=23, latent_format=NV),
                               sm_scale=scale)
    out, lse, st = run_dense(case, synth.device_case(case))
    assert st == 0
    check_rows(case, out, lse)


def test_dense_mla_rising_logits():
    """Tokens sorted by one head's logit, so that its maximum grows along the whole context and the others' do not."""
    case = synth.make_case("dense_rising", seq_lens=[2500], seed=24, latent_format=FP8)
    c = plain64.latents(case, 0)
    q = plain64.queries(case, 0) * 8
    case = dataclasses.replace(case, q_mla=q.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)[None].copy())
    for head in (0, 50, 95):
        order = torch.argsort(c @ q[head]).numpy()
        pool = case.pool.copy()
        flat = pool[case.block_table[0], :64 * 576].reshape(-1, 576)
        flat[:2500] = flat[:2500][order]
        pool[case.block_table[0], :64 * 576] = flat.reshape(-1, 64 * 576)
        sorted_case = dataclasses.replace(case, pool=pool)
        out, lse, st = run_dense(sorted_case, synth.device_case(sorted_case))
        assert st == 0
        check_rows(sorted_case, out, lse)


@pytest.mark.parametrize("bits", [0x7FC0, 0x7F80])
def test_dense_mla_nan_or_inf_in_a_query(bits):
    """A NaN or an infinity in one head's query leaves NaN in that head and nothing in the others or the other rows."""
    case = synth.make_case("dense_nan", seq_lens=[500, 300], seed=25, latent_format=NV)
    q = case.q_mla.copy()
    q[0, 5, 17] = bits
    out, lse, st = run_dense(dataclasses.replace(case, q_mla=q), synth.device_case(dataclasses.replace(case, q_mla=q)))
    assert st == 0
    assert bool(torch.isnan(out[0, 5].float()).all()) and bool(torch.isnan(lse[0, 5]))
    clean, clean_lse, _ = run_dense(case, synth.device_case(case))
    out[0, 5], lse[0, 5] = clean[0, 5], clean_lse[0, 5]
    check_rows(case, out, lse)


def test_dense_mla_tiny_and_huge_queries():
    """Query magnitudes far outside fp16's range, and heads of very different size in one row."""
    case = synth.make_case("dense_range", seq_lens=[300], seed=26, latent_format=FP8)
    q = torch.randn((1, 96, 576), generator=torch.Generator().manual_seed(2))
    for factor, scale in ((2.0 ** -100, 2.0 ** 95), (2.0 ** 60, 2.0 ** -64), (0.0, 1.0)):
        size = factor * torch.logspace(-6, 0, 96)[None, :, None]
        bits = (q * size).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
        one = dataclasses.replace(case, q_mla=bits, sm_scale=scale)
        out, lse, st = run_dense(one, synth.device_case(one))
        assert st == 0
        check_rows(one, out, lse)


def test_cache_beyond_4_gib():
    """Pages past the 4 GiB mark of a pool: attention, weights and eviction address them with 64 bits."""
    small = synth.make_case("dense_far", seq_lens=[200, 130], seed=27, key_format=synth.KEY_MXFP4, latent_format=NV)
    stride = small.row_stride
    blocks = (1 << 32) // stride + 200
    pool = torch.empty((blocks, stride), dtype=torch.uint8, device="cuda")
    far = torch.arange(blocks - 1, blocks - 1 - small.num_blocks, -1, device="cuda")   # page p of the case lies there
    pool[far] = torch.from_numpy(small.pool).cuda()
    dc = synth.device_case(small)
    table = torch.from_numpy(small.block_table).cuda()
    table = torch.where(table >= 0, far[table.clamp(min=0).long()].to(torch.int32), table)
    dc.cache.pool, dc.batch.block_table = pool, table.contiguous()
    out, lse, st = run_dense(small, dc)
    assert st == 0
    check_rows(small, out, lse)
    mass = torch.zeros((2, 200), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = binding.workspace(binding.attention_mass_workspace_size(2, 200, 0))
    binding.attention_mass(dc.cache, dc.batch, dc.q_mla, lse, small.sm_scale, None, mass, ws, status)
    torch.testing.assert_close(mass.sum(1), torch.full((2,), 96.0, device="cuda"), rtol=1e-4, atol=0)
    # evicted within the far end of the same pool
    to = torch.arange(blocks - 100, blocks - 96, dtype=torch.int32, device="cuda").view(2, 2)
    kept = torch.empty((2, 100), dtype=torch.int32, device="cuda")
    lens = torch.empty(2, dtype=torch.int32, device="cuda")
    ws = binding.workspace(binding.cache_evict_workspace_size(2, 200, 100))
    binding.cache_evict(dc.cache, dc.batch, mass, 100, 3, 20, dc.cache, to, kept, None, lens, ws, status)
    after = binding.Batch(to, lens, 1, 100)
    o2 = torch.empty_like(out)
    l2 = torch.empty_like(lse)
    ws = binding.workspace(binding.dense_mla_workspace_size(2, 100))
    binding.dense_mla_decode(dc.cache, after, dc.q_mla, small.sm_scale, o2, l2, ws, status)
    torch.cuda.synchronize()
    assert status.item() == 0 and lens.tolist() == [100, 100]
    for b in range(2):
        ro, rl, av, spread, bound = plain64.attend(small, b, kept[b].long().cpu())
        e = 576 * 2.0 ** -24 * bound
        tol = 2.0 ** -8 * (1 + 2.0 ** -7) * spread + (2 * e[:, None] + 200 * 2.0 ** -24 + 2.0 ** -11) * av + 2.0 ** -8 * ro.abs()
        assert torch.all((o2[b].double().cpu() - ro).abs() <= tol)
