"""Host-side checks of dsa_assign_slots, dsa_cache_append_slots and the gated
delta calls: refused synchronously, before anything is launched, so no device is
needed; and the binding's checks of shapes, types and strides."""
import ctypes

import pytest
import torch

from dsa_sparse_attention_index_gb300 import binding as B
from dsa_sparse_attention_index_gb300 import build
from test_binding_cache_ops import Library, Tensor

FAKE = 1 << 20   # an aligned address that the host checks never follow


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def assign(lib, cached=FAKE, new=2 * FAKE, batch=3, free=FAKE, cap=10, count=FAKE, left=FAKE, blocks=10, table=FAKE,
           width=4, lens=FAKE, starts=FAKE, pos=FAKE, slots=FAKE, rows=5, st=FAKE):
    return lib.dsa_assign_slots(cached, new, batch, free, cap, count, left, blocks, table, width, lens, starts, pos, slots,
                                rows, st, None)


def test_assign_refusals(lib):
    for bad in ("cached", "new", "free", "count", "left", "table", "lens", "starts", "pos", "slots", "st"):
        assert assign(lib, **{bad: None}) == B.ERR_INVALID_ARG, bad
        if bad != "st":
            assert assign(lib, **{bad: FAKE + 2}) == B.ERR_INVALID_ARG, bad
    for bad in (dict(batch=-1), dict(cap=-1), dict(blocks=0), dict(width=0), dict(rows=-1), dict(lens=2 * FAKE)):
        assert assign(lib, **bad) == B.ERR_INVALID_ARG, bad
    for bad in (dict(batch=(1 << 24) + 1), dict(blocks=(1 << 25) + 1), dict(width=(1 << 24) + 1), dict(rows=(1 << 30) + 1)):
        assert assign(lib, **bad) == B.ERR_UNSUPPORTED, bad


def append(lib, base=FAKE, slots=FAKE, rows=4, lat=FAKE, key=FAKE, st=FAKE, **kw):
    c = B.PagedCacheT(base, 45312, 0, 36864, 64, 10, B.KEY_FP8_E4M3, 1.0, B.LATENT_FP8_E4M3)
    for k, v in kw.items():
        setattr(c, k, v)
    return lib.dsa_cache_append_slots(ctypes.byref(c), slots, rows, lat, key, st, None)


def test_append_slots_refusals(lib):
    for bad in (dict(base=None), dict(slots=None), dict(lat=None), dict(key=None), dict(st=None), dict(rows=-1),
                dict(slots=FAKE + 2), dict(lat=FAKE + 8), dict(key=FAKE + 8), dict(row_stride=64), dict(key_format=9)):
        assert append(lib, **bad) == B.ERR_INVALID_ARG, bad
    assert append(lib, rows=(1 << 24) + 1) == B.ERR_UNSUPPORTED
    assert append(lib, rows=0, slots=None, lat=None, key=None) == B.OK    # nothing to do


def delta(lib, prefill=False, batch=2, nq=1, rows=8, slots_in=FAKE, slots_out=FAKE, out=FAKE, starts=FAKE, ws=FAKE,
          n=1 << 50, st=FAKE, **kw):
    pool = B.StatePoolT(FAKE, 4 * 65536, 10, 4)
    x = B.DeltaRowsT(FAKE, FAKE, FAKE, FAKE, FAKE, 256, 256, 512, 512, 4, 2, 128, 1.0)
    for k, v in kw.items():
        setattr(pool if hasattr(pool, k) else x, k, v)
    if prefill:
        return lib.gated_delta_prefill(ctypes.byref(pool), ctypes.byref(x), starts, batch, rows, slots_in, slots_out, out,
                                       ws, n, st, None)
    return lib.gated_delta_decode(ctypes.byref(pool), ctypes.byref(x), batch, nq, slots_in, slots_out, out, st, None)


@pytest.mark.parametrize("prefill", [False, True])
def test_gated_delta_refusals(lib, prefill):
    for bad in (dict(base=None), dict(base=FAKE + 64), dict(slot_stride=4 * 65536 - 128), dict(slot_stride=4 * 65536 + 64),
                dict(num_slots=0), dict(heads=0), dict(qk_heads=3), dict(qk_heads=0), dict(gate_dim=64), dict(q=None),
                dict(k=None), dict(v=None), dict(gate=None), dict(beta=None), dict(q=FAKE + 8), dict(k=FAKE + 8),
                dict(v=FAKE + 2), dict(gate=FAKE + 4), dict(beta=FAKE + 1), dict(ld_q=248), dict(ld_k=260), dict(ld_v=511),
                dict(ld_gate=514), dict(ld_beta=3), dict(slots_in=None), dict(slots_out=None), dict(out=None),
                dict(out=FAKE + 8), dict(st=None), dict(batch=-1), dict(slots_in=FAKE + 2)):
        assert delta(lib, prefill, **bad) == B.ERR_INVALID_ARG, bad
    assert delta(lib, prefill, gate_dim=1, gate=FAKE + 2) == B.ERR_INVALID_ARG
    big = dict(heads=8192, slot_stride=8192 * 65536, ld_v=1 << 20, ld_gate=1 << 20, ld_beta=8192)
    assert delta(lib, prefill, **big) == B.ERR_UNSUPPORTED
    assert delta(lib, prefill, batch=1 << 23) == B.ERR_UNSUPPORTED
    assert delta(lib, prefill, batch=0, slots_in=None, slots_out=None) == B.OK      # nothing to do
    if not prefill:
        assert delta(lib, nq=0) == B.ERR_INVALID_ARG
        assert delta(lib, nq=1 << 24) == B.ERR_UNSUPPORTED
        return
    assert delta(lib, True, starts=None) == B.ERR_INVALID_ARG
    assert delta(lib, True, rows=(1 << 24) + 1) == B.ERR_UNSUPPORTED
    need = lib.gated_delta_prefill_workspace_size(8, 2, 4)
    assert need > 0 and lib.gated_delta_prefill_workspace_size(-1, 2, 4) == 0
    for bad in (dict(ws=None), dict(ws=FAKE + 128), dict(n=need - 1)):
        assert delta(lib, True, **bad) == B.ERR_WORKSPACE, bad


@pytest.fixture
def calls(monkeypatch):
    library = Library()
    monkeypatch.setattr(B, "lib", lambda: library)
    monkeypatch.setattr(B, "_stream", lambda s: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return library


def i32(*shape):
    return Tensor(shape, torch.int32)


def test_binding_assign(calls):
    def go(batch=3, rows=9, **kw):
        a = dict(cached_lens=i32(batch), new_lens=i32(batch), free_blocks=i32(20), free_count=i32(1), num_blocks=20,
                 block_table=i32(batch, 4), seq_lens=i32(batch), row_starts=i32(batch + 1), positions=i32(rows),
                 slots=i32(rows), free_left=i32(1), status=i32(1))
        B.assign_slots(**{**a, **kw})

    go()
    go(rows=0)
    assert calls.calls == 2
    for bad in (dict(new_lens=i32(2)), dict(block_table=i32(2, 4)), dict(row_starts=i32(3)), dict(positions=i32(8)),
                dict(free_left=i32(2)), dict(cached_lens=Tensor((3,), torch.int64)), dict(free_count=i32(0)),
                dict(slots=Tensor((9,), torch.int64))):
        with pytest.raises(ValueError):
            go(**bad)
    assert calls.calls == 2


class Rows(Tensor):
    """A stand-in with strides: `apart` more elements between rows."""

    def __init__(self, shape, dtype, apart=0, cuda=True, order=None):
        super().__init__(shape, dtype)
        self.is_cuda, inner, strides = cuda, 1, []
        for size in reversed(shape[1:]):
            strides.append(inner)
            inner *= size
        self._strides = order or (inner + apart, *reversed(strides))

    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]


def layer(rows=6, qk=2, heads=4, wide=True, **kw):
    bf, f32 = torch.bfloat16, torch.float32
    t = dict(q=Rows((rows, qk, 128), bf, 64), k=Rows((rows, qk, 128), bf), v=Rows((rows, heads, 128), bf),
             gate=Rows((rows, heads, 128) if wide else (rows, heads), f32), beta=Rows((rows, heads), f32, 3), scale=0.5)
    return B.DeltaRows(**{**t, **kw})


def test_binding_descriptors():
    x = layer().layout
    assert (x.ld_q, x.ld_k, x.ld_v, x.ld_gate, x.ld_beta, x.qk_heads, x.gate_dim) == (320, 256, 512, 512, 7, 2, 128)
    assert layer(wide=False).layout.gate_dim == 1 and layer(rows=1).layout.ld_q == 256
    bf, f32 = torch.bfloat16, torch.float32
    for bad in (dict(q=Rows((6, 2, 64), bf)), dict(q=Rows((6, 256), bf)), dict(k=Rows((5, 2, 128), bf)),
                dict(v=Rows((6, 4, 128), f32)), dict(gate=Rows((6, 4, 64), f32)), dict(beta=Rows((6, 3), f32)),
                dict(gate=Rows((6, 4, 128), bf)), dict(v=Rows((6, 4, 128), bf, cuda=False)),
                dict(k=Rows((6, 2, 128), bf, order=(256, 1, 2)))):
        with pytest.raises(ValueError):
            layer(**bad)
    p = B.StatePool(Rows((5, 4, 128, 128), f32, 32)).layout
    assert (p.slot_stride, p.num_slots, p.heads) == (4 * (4 * 16384 + 32), 5, 4)
    for bad in (Rows((5, 4, 128, 64), f32), Rows((5, 4, 16384), f32), Rows((5, 4, 128, 128), bf),
                Rows((5, 4, 128, 128), f32, cuda=False), Rows((5, 4, 128, 128), f32, order=(65536, 16384, 1, 128))):
        with pytest.raises(ValueError):
            B.StatePool(bad)


def test_binding_gated_delta(calls):
    f32, bf = torch.float32, torch.bfloat16
    pool, x, out, ws = B.StatePool(Rows((9, 4, 128, 128), f32)), layer(), Tensor((6, 4, 128), bf), Tensor((99,), torch.uint8)

    def decode(pool=pool, x=x, nq=3, slots_in=i32(2), slots_out=i32(2, 3), out=out, status=i32(1)):
        B.gated_delta_decode(pool, x, nq, slots_in, slots_out, out, status)

    def prefill(pool=pool, x=x, starts=i32(3), slots_in=i32(2), slots_out=i32(2), out=out, ws=ws, status=i32(1)):
        B.gated_delta_prefill(pool, x, starts, slots_in, slots_out, out, ws, status)

    decode()
    prefill()
    assert calls.calls == 2
    other = B.StatePool(Rows((9, 8, 128, 128), f32))
    for bad in (dict(nq=2), dict(slots_out=i32(2, 2)), dict(slots_in=Tensor((2,), torch.int64)), dict(pool=other),
                dict(out=Tensor((6, 4, 128), f32)), dict(out=Tensor((5, 4, 128), bf)), dict(status=i32(0))):
        with pytest.raises(ValueError):
            decode(**bad)
    for bad in (dict(starts=i32(2)), dict(slots_out=i32(2, 1)), dict(slots_in=i32(3)), dict(pool=other),
                dict(out=Tensor((6, 3, 128), bf)), dict(starts=Tensor((3,), torch.int64))):
        with pytest.raises(ValueError):
            prefill(**bad)
    assert calls.calls == 2


def test_binding_append_slots(calls):
    bf = torch.bfloat16
    cache = B.PagedCache(Tensor((3, 45312), torch.uint8), 45312, 0, 36864, B.KEY_FP8_E4M3, 1.0)

    def go(cache=cache, slots=i32(4), lat=Tensor((4, 576), bf), key=Tensor((4, 128), bf), status=i32(1)):
        B.cache_append_slots(cache, slots, lat, key, status)

    go()
    small = B.PagedCache(Tensor((3, 45000), torch.uint8), 45312, 0, 36864, B.KEY_FP8_E4M3, 1.0)
    for bad in (dict(lat=Tensor((3, 576), bf)), dict(key=Tensor((4, 64), bf)), dict(slots=Tensor((4,), torch.int64)),
                dict(cache=small), dict(lat=Tensor((4, 576), torch.float32))):
        with pytest.raises(ValueError):
            go(**bad)
    assert calls.calls == 1
