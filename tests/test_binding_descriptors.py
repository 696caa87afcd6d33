"""StatePool and DeltaRows over tensors whose storage changes after the descriptor
was made: the call takes the tensors as they are, or is refused."""
import ctypes

import pytest
import torch

from dsa_sparse_attention_index_gb300 import binding as B
from test_abi_step_ops import Rows, i32, layer
from test_binding_cache_ops import Tensor


class Moving(Rows):
    """A stand-in whose address, shape and strides a test changes."""

    at = 1 << 20

    def data_ptr(self):
        return self.at

    def move(self, at=None, shape=None, strides=None):
        self.at = at or self.at
        self.shape = torch.Size(shape or self.shape)
        self._strides = strides or self._strides


class Recorder:
    """Keeps the descriptors that reach the library."""

    def __getattr__(self, name):
        def call(pool, x, *args):
            pool, x = (ctypes.cast(p, ctypes.POINTER(t)).contents for p, t in ((pool, B.StatePoolT), (x, B.DeltaRowsT)))
            self.pool = {n: getattr(pool, n) for n, _ in pool._fields_}
            self.x = {n: getattr(x, n) for n, _ in x._fields_}
            return B.OK
        return call


@pytest.fixture
def library(monkeypatch):
    fake = Recorder()
    monkeypatch.setattr(B, "lib", lambda: fake)
    monkeypatch.setattr(B, "_stream", lambda s: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return fake


NAMES = dict(q=(6, 2, 128), k=(6, 2, 128), v=(6, 4, 128), gate=(6, 4, 128), beta=(6, 4))


def things():
    t = {n: Moving(s, torch.bfloat16 if n in "qkv" else torch.float32) for n, s in NAMES.items()}
    return Moving((9, 4, 128, 128), torch.float32), t


def decode(pool, x):
    B.gated_delta_decode(pool, x, 3, i32(2), i32(2, 3), Tensor((6, 4, 128), torch.bfloat16), i32(1))


def prefill(pool, x):
    B.gated_delta_prefill(pool, x, i32(3), i32(2), i32(2), Tensor((6, 4, 128), torch.bfloat16), Tensor((99,), torch.uint8), i32(1))


@pytest.mark.parametrize("call", [decode, prefill])
def test_tensors_that_move_are_followed(library, call):
    states, t = things()
    pool, x = B.StatePool(states), layer(**t)
    call(pool, x)
    assert library.pool["base"] == 1 << 20 and library.x["q"] == 1 << 20
    states.move(1 << 30, strides=(4 * 16384 + 32, 16384, 128, 1))
    for i, (name, tensor) in enumerate(t.items()):
        wide = 1024 + 64 * i
        tensor.move((1 << 31) + 4096 * i, strides=(wide, *tensor.stride()[1:]))
        call(pool, x)
        assert library.x[name] == (1 << 31) + 4096 * i and library.x["ld_" + name] == wide
    assert library.pool["base"] == 1 << 30 and library.pool["slot_stride"] == 4 * (4 * 16384 + 32)


@pytest.mark.parametrize("call", [decode, prefill])
@pytest.mark.parametrize("name", NAMES)
def test_tensors_that_no_longer_fit_are_refused(library, call, name):
    states, t = things()
    pool, x = B.StatePool(states), layer(**t)
    call(pool, x)
    t[name].move(1 << 30, shape=(5, *NAMES[name][1:]))
    with pytest.raises(ValueError):
        call(pool, x)
    t[name].move(1 << 31, shape=NAMES[name])
    call(pool, x)
    t[name].move(1 << 32, strides=tuple(2 * s for s in t[name].stride()))
    with pytest.raises(ValueError):
        call(pool, x)


@pytest.mark.parametrize("call", [decode, prefill])
def test_rows_that_grow_in_place_are_refused(library, call):
    """Values of a buffer with room for more rows, the others without."""
    states, t = things()
    pool, x = B.StatePool(states), layer(**t)
    t["v"].move(shape=(12, 4, 128))
    with pytest.raises(ValueError):
        call(pool, x)


@pytest.mark.parametrize("call", [decode, prefill])
def test_states_that_no_longer_fit_are_refused(library, call):
    states, t = things()
    pool, x = B.StatePool(states), layer(**t)
    states.move(shape=(9, 8, 128, 128), strides=(8 * 16384, 16384, 128, 1))
    with pytest.raises(ValueError):
        call(pool, x)
    states.move(shape=(5, 4, 128, 128), strides=(4 * 16384, 16384, 128, 1))
    call(pool, x)
    assert library.pool["num_slots"] == 5
