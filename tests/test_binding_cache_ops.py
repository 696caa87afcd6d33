"""The binding's own checks in front of dense_mla_decode, dsa_attention_mass and
dsa_cache_evict: what the C side cannot see (shapes, types and sizes behind its
pointers) is refused before the library is called.  Stand-ins take the tensors'
place, so no device is needed."""
import math

import pytest
import torch

from dsa_sparse_attention_index_gb300 import binding as B

ITEM = {torch.int32: 4, torch.int64: 8, torch.float32: 4, torch.uint8: 1, torch.bfloat16: 2, torch.int16: 2}


class Tensor:
    """What the binding asks of a CUDA tensor."""

    is_cuda = True

    def __init__(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.nbytes = math.prod(shape) * ITEM[dtype]

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 20 if self.numel() else 0   # as torch: an empty tensor has no address


class Library:
    """Counts the calls that reach the library; each succeeds."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return B.OK
        return call


@pytest.fixture
def lib(monkeypatch):
    fake = Library()
    monkeypatch.setattr(B, "lib", lambda: fake)
    monkeypatch.setattr(B, "_stream", lambda stream: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return fake


def cache(blocks=10, row=45312, stride=45312):
    return B.PagedCache(Tensor((blocks, row), torch.uint8), stride, 0, 36864, B.KEY_FP8_E4M3, 1.0)


def batch(table=(3, 8), lens=(3,), types=(torch.int32, torch.int32), nq=2):
    return B.Batch(Tensor(table, types[0]), Tensor(lens, types[1]), nq, 500)


def arguments():
    rows = 6
    return dict(q=Tensor((rows, 96, 576), torch.bfloat16), out=Tensor((rows, 96, 512), torch.bfloat16),
                lse=Tensor((rows, 96), torch.float32), mass=Tensor((3, 500), torch.float32),
                table=Tensor((3, 2), torch.int32), kept=Tensor((3, 100), torch.int32), lens=Tensor((3,), torch.int32),
                ws=Tensor((1 << 30,), torch.uint8), status=Tensor((1,), torch.int32), idx=Tensor((rows, 64), torch.int32))


def calls(c=None, b=None, d=None, **kw):
    """The three calls (four: the weights with and without a selection), each with these arguments replaced."""
    a = {**arguments(), **kw}
    c, b, d = c or cache(), b or batch(), d or cache()
    return [lambda: B.dense_mla_decode(c, b, a["q"], 1.0, a["out"], a["lse"], a["ws"], a["status"]),
            lambda: B.attention_mass(c, b, a["q"], a["lse"], 1.0, a["mass"], a["mass"], a["ws"], a["status"]),
            lambda: B.attention_mass(c, b, a["q"], a["lse"], 1.0, None, a["mass"], a["ws"], a["status"], idx=a["idx"]),
            lambda: B.cache_evict(c, b, a["mass"], 100, 4, 16, d, a["table"], a["kept"], None, a["lens"], a["ws"], a["status"])]


def refused(lib, bad):
    before = lib.calls
    with pytest.raises(ValueError):
        bad()
    assert lib.calls == before


def test_good_calls_pass(lib):
    for call in calls() + calls(b=batch(table=(5, 8))):   # a table of more rows than sequences has what is read
        call()
    assert lib.calls == 8


@pytest.mark.parametrize("bad", [dict(table=(2, 8)), dict(table=(3,)), dict(table=(3, 8, 1)), dict(lens=(3, 1)),
                                 dict(types=(torch.int64, torch.int32)), dict(types=(torch.int32, torch.int64))])
def test_tables_and_lengths(lib, bad):
    """Fewer table rows than sequences would be read past their end, 64-bit entries as twice as many."""
    for call in calls(b=batch(**bad)):
        refused(lib, call)


def test_pools_smaller_than_their_rows(lib):
    for call in calls(c=cache(row=45312 - 128)):
        refused(lib, call)
    refused(lib, calls(d=cache(row=45312 - 128))[3])


@pytest.mark.parametrize("shape,dtype", [((0,), torch.int32), ((1,), torch.int64), ((1,), torch.uint8)])
def test_status_words(lib, shape, dtype):
    for call in calls(status=Tensor(shape, dtype)):
        refused(lib, call)


def test_a_selection_of_no_entries(lib):
    """An empty idx has no address, which the library would take for "every visible token"."""
    refused(lib, calls(idx=Tensor((6, 0), torch.int32))[2])


def test_no_status_word_is_left_to_the_library(lib):
    """Which refuses it by its own code."""
    none = {**arguments(), "status": None}
    for call in calls(**none):
        call()
    assert lib.calls == 4
