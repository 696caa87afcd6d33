"""Host-side checks of dense_mla_decode, dsa_attention_mass and dsa_cache_evict:
refused synchronously, before anything is launched, so no device is needed; the
sizes of their workspaces; and the binding's checks of shapes and types."""
import ctypes

import pytest
import torch

from dsa_sparse_attention_index_gb300 import binding as B
from dsa_sparse_attention_index_gb300 import build

FAKE = 1 << 20   # an aligned address that the host checks never follow


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def cache(**kw):
    c = B.PagedCacheT(FAKE, 45312, 0, 36864, 64, 10, B.KEY_FP8_E4M3, 1.0, B.LATENT_FP8_E4M3)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def batch(**kw):
    b = B.BatchT(FAKE, 2 * FAKE, 8, 2, 1, 500)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def refs(*structs):
    return [ctypes.byref(s) for s in structs]


def dense(lib, c=None, b=None, q=FAKE, out=FAKE, lse=FAKE, ws=FAKE, n=1 << 40, st=FAKE):
    return lib.dense_mla_decode(*refs(c or cache(), b or batch()), q, 1.0, out, lse, ws, n, st, None)


def test_dense_mla_refusals(lib):
    assert dense(lib, c=cache(base=None)) == B.ERR_INVALID_ARG
    assert dense(lib, c=cache(block_size=32)) == B.ERR_UNSUPPORTED
    assert dense(lib, c=cache(latent_format=2)) == B.ERR_INVALID_ARG
    assert dense(lib, c=cache(row_stride=45312 + 64)) == B.ERR_INVALID_ARG
    assert dense(lib, b=batch(queries_per_seq=2049)) == B.ERR_UNSUPPORTED
    assert dense(lib, b=batch(block_table=None)) == B.ERR_INVALID_ARG
    assert dense(lib, b=batch(max_seq_len=-1)) == B.ERR_INVALID_ARG
    assert dense(lib, st=None) == B.ERR_INVALID_ARG
    for bad in (dict(q=None), dict(out=None), dict(lse=None), dict(q=FAKE + 8), dict(out=FAKE + 4), dict(lse=FAKE + 2)):
        assert dense(lib, **bad) == B.ERR_INVALID_ARG
    need = lib.dense_mla_workspace_size(2, 500)
    for bad in (dict(ws=None), dict(ws=FAKE + 128), dict(n=need - 1)):
        assert dense(lib, **bad) == B.ERR_WORKSPACE
    assert dense(lib, b=batch(batch=0)) == B.OK     # nothing to do


def mass(lib, c=None, b=None, q=FAKE, lse=FAKE, idx=None, k=0, mi=None, mo=FAKE, ld=500, ws=FAKE, n=1 << 40, st=FAKE):
    return lib.dsa_attention_mass(*refs(c or cache(), b or batch()), q, lse, idx, k, 1.0, mi, mo, ld, ws, n, st, None)


def test_attention_mass_refusals(lib):
    assert mass(lib, c=cache(num_blocks=0)) == B.ERR_INVALID_ARG
    for bad in (dict(q=None), dict(lse=None), dict(mo=None), dict(q=FAKE + 8), dict(lse=FAKE + 1), dict(mi=FAKE + 2),
                dict(mo=FAKE + 2), dict(ld=499), dict(k=5), dict(idx=FAKE, k=0), dict(idx=FAKE, k=2049),
                dict(idx=FAKE, k=-1), dict(idx=FAKE + 2, k=7), dict(st=None)):
        assert mass(lib, **bad) == B.ERR_INVALID_ARG, bad
    for nq, k in ((1, 0), (4, 0), (1, 100)):
        need = lib.dsa_attention_mass_workspace_size(2 * nq, 500, k)
        kw = dict(b=batch(queries_per_seq=nq), idx=FAKE if k else None, k=k)
        for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(n=need - 1)):
            assert mass(lib, **kw, **bad) == B.ERR_WORKSPACE
    assert mass(lib, b=batch(batch=0)) == B.OK


def evict(lib, c=None, b=None, d=None, m=FAKE, ld=500, keep=128, sink=4, recent=32, table=FAKE, blocks=2, kept=FAKE,
          mo=2 * FAKE, ldo=128, lens=FAKE, ws=FAKE, n=1 << 40, st=FAKE):
    cs, bs, ds = refs(c or cache(), b or batch(), d or cache())
    return lib.dsa_cache_evict(cs, bs, m, ld, keep, sink, recent, ds, table, blocks, kept, mo, ldo, lens, ws, n, st, None)


def test_cache_evict_refusals(lib):
    for bad in (dict(keep=0), dict(sink=-1), dict(recent=-1), dict(sink=100, recent=29), dict(blocks=1), dict(blocks=0),
                dict(m=None), dict(table=None), dict(kept=None), dict(lens=None), dict(ld=499), dict(ldo=127),
                dict(m=FAKE + 2), dict(mo=2 * FAKE + 1), dict(kept=FAKE + 3), dict(st=None),
                dict(sink=(1 << 31) - 1, recent=(1 << 31) - 1)):
        assert evict(lib, **bad) == B.ERR_INVALID_ARG, bad
    assert evict(lib, lens=2 * FAKE) == B.ERR_INVALID_ARG          # the lengths themselves
    assert evict(lib, mo=FAKE) == B.ERR_INVALID_ARG                # the totals themselves
    assert evict(lib, mo=FAKE + 4 * 900) == B.ERR_INVALID_ARG      # overlapping the totals
    assert evict(lib, d=cache(base=None)) == B.ERR_INVALID_ARG
    # records move as they are
    nv = dict(latent_format=B.LATENT_NVFP4, row_stride=64 * 352 + 64 * 132, index_off=64 * 352)
    assert evict(lib, d=cache(**nv)) == B.ERR_UNSUPPORTED
    assert evict(lib, d=cache(latent_scale=2.0)) == B.ERR_UNSUPPORTED
    assert evict(lib, d=cache(key_format=B.KEY_MXFP4)) == B.ERR_UNSUPPORTED
    need = lib.dsa_cache_evict_workspace_size(2, 500, 128)
    for bad in (dict(ws=None), dict(ws=FAKE + 4), dict(n=need - 1)):
        assert evict(lib, **bad) == B.ERR_WORKSPACE
    assert evict(lib, b=batch(batch=0)) == B.OK
    # one page layout, two names: MXFP4 keys for either query format
    c1, c2 = cache(key_format=B.KEY_MXFP4), cache(key_format=B.KEY_MXFP4_NATIVE)
    assert evict(lib, c=c1, d=c2, ws=None) == B.ERR_WORKSPACE


def test_workspace_sizes(lib):
    q16 = 96 * 576 * 2
    assert lib.dense_mla_workspace_size(-1, 10) == 0 and lib.dense_mla_workspace_size(1, -1) == 0
    # the queries in fp16 and two partials for each of up to 256 CTAs
    assert lib.dense_mla_workspace_size(32, 65536) >= 32 * q16 + 512 * 96 * 512 * 2
    assert lib.dense_mla_workspace_size(1, 100) < 1 << 20
    assert lib.dsa_batch_invariant(1) == 0
    try:   # a partial every 3,840 tokens
        assert lib.dense_mla_workspace_size(4, 100000) >= 4 * 27 * 96 * 512 * 2
    finally:
        assert lib.dsa_batch_invariant(0) == 1
    assert lib.dsa_attention_mass_workspace_size(4, 1000, 0) >= 4 * (q16 + 4000)
    assert lib.dsa_attention_mass_workspace_size(4, 100000, 64) < 4 * q16 + 4 * 64 * 4 + 4096
    assert lib.dsa_attention_mass_workspace_size(4, 1000, 2049) == 0
    assert lib.dsa_attention_mass_workspace_size(4, 1000, -1) == 0
    assert lib.dsa_cache_evict_workspace_size(3, 1000, 100) >= 1200
    assert lib.dsa_cache_evict_workspace_size(3, 1000, 0) == 0


def test_binding_checks_shapes_and_types():
    x = torch.zeros((2, 96), dtype=torch.float32)
    for shape, types in (((2, 95), B._F32), ((3, 96), B._F32), ((2, 96, 1), B._F32), ((2, 96), B._I32)):
        with pytest.raises(ValueError):
            B._want("lse", x, shape, types)
    with pytest.raises(ValueError):
        B._want("lse", x, (2, 96), B._F32)       # a host tensor
    assert B._want("mass_in", None, (2, 96), B._F32) is None


def test_contexts_beyond_32_bit_tiles_and_overlapping_totals(lib):
    far = batch(max_blocks_per_seq=1 << 25, max_seq_len=(1 << 30) + 1)
    assert dense(lib, b=far) == B.ERR_UNSUPPORTED
    assert evict(lib, b=far, ld=1 << 31, mo=None) == B.ERR_UNSUPPORTED
    # a loose bound over a short table is none
    loose = batch(max_seq_len=(1 << 31) - 1)
    assert dense(lib, b=loose, ws=None) == B.ERR_WORKSPACE
    assert evict(lib, b=loose, ld=1 << 31, mo=None, ws=None) == B.ERR_WORKSPACE
    for rows in (1, 3):   # and takes as many partial results as any long one
        assert lib.dense_mla_workspace_size(rows, (1 << 31) - 1) == lib.dense_mla_workspace_size(rows, 1 << 20)
    for mi in (FAKE + 4 * 900, FAKE - 4 * 900):
        assert mass(lib, mi=mi) == B.ERR_INVALID_ARG
    for mi in (FAKE, FAKE + 4 * 1000, FAKE - 4 * 1000):
        assert mass(lib, mi=mi, ws=None) == B.ERR_WORKSPACE


def test_an_empty_batch_has_nothing_to_do_whatever_the_selection(lib):
    """No sequence, so no row of idx, whose tensor then has no address."""
    none = batch(batch=0, block_table=None, seq_lens=None)
    assert mass(lib, b=none, idx=None, k=64, q=None, lse=None, mo=None, ws=None, n=0) == B.OK
    assert mass(lib, b=none, q=None, lse=None, mo=None, ws=None, n=0) == B.OK
    assert dense(lib, b=none, q=None, out=None, lse=None, ws=None, n=0) == B.OK
    assert evict(lib, b=none, m=None, table=None, kept=None, mo=None, lens=None, ws=None, n=0) == B.OK
    assert mass(lib, b=none, idx=None, k=2049) == B.ERR_INVALID_ARG
