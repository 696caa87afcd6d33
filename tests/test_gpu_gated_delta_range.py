"""gated_delta_prefill where the rows of a chunk differ widely in size, and how
many bits it keeps: long keys and values with small betas among ordinary rows,
states that decay by many powers of two, large and small queries, scales,
states that are no finite numbers, the paths beside the tensor cores for one
decay a head and for shared query and key heads, and states and outputs held to
the operands' bits instead of to a bound that grows with the rows; descriptors
over storage that changes."""
import math

import pytest
import torch

from dsa_sparse_attention_index_gb300 import binding as B
from plain_delta import DIM, inputs, out_tolerance, rule, state_tolerance

pytestmark = pytest.mark.gpu
SCALE = DIM ** -0.5


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def state(heads, seed=1):
    return 0.3 * torch.randn((1, heads, DIM, DIM), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def prefill(x, s0, scale=SCALE):
    """(outputs, last state) of one sequence."""
    rows, heads = x[2].shape[:2]
    pool, out, st = torch.cat([s0, torch.zeros_like(s0)]), torch.zeros((rows, heads, DIM), dtype=torch.bfloat16, device="cuda"), ints(0)
    ws = B.workspace(B.gated_delta_prefill_workspace_size(rows, 1, heads))
    B.gated_delta_prefill(B.StatePool(pool), B.DeltaRows(*x, scale), ints(0, rows), ints(0), ints(1), out, ws, st)
    assert st.item() == 0
    return out, pool[1]


def norms(s):
    return s.double().flatten(1).norm(dim=1)


# Six operands meet a state in 64 rows (S, K P, R, T, U, K D).  Each is two fp16 parts of 11 bits: what the second leaves is at
# most 2^-22 of the number, and the product of two second parts, which is left out, at most 2^-20 of a product; counted together
# as 2^-21 for each operand, relative to the state, since the updates (beta |k|^2 <= 1) and the decays do not enlarge it.
# (An emulation of the chunks on these inputs stays within 0.06 of it; without any one of the cross products of first and
# second parts it is 13 to 137 times over it.)
BITS = 6 * 2.0 ** -21


def check_bits(got, want, size):
    off = norms(got.double() - want) / size
    assert (off <= BITS).all(), off / BITS


def check_out(out, want, rows, size, mass, q, scale=SCALE):
    off, tol = (out.double() - want).abs(), out_tolerance(want, rows, size, mass, q, scale, True)
    assert (off <= tol).all(), (off / tol).max()


@pytest.mark.parametrize("length", [1e2, 1e3, 1e4, 1e6])
@pytest.mark.parametrize("at", [[63], [20, 21, 100]], ids=str)
def test_long_keys_among_ordinary_ones(length, at):
    """beta |k|^2 = 1 whatever the key's length: the update is of the state's size."""
    x, s0 = inputs(130, 2, 2, seed=41), state(2)
    q, k, v, g, beta = x
    k[at] = (k[at].float() * length).to(torch.bfloat16)
    beta[at] = 1 / k[at].float().square().sum(2)
    out, last = prefill(x, s0)
    want, states, size, mass = rule(*x, SCALE, s0[0])
    check_bits(last, states[-1], torch.stack([norms(s) for s in states]).amax(0))
    check_out(out, want, 130, size, mass, q)


@pytest.mark.parametrize("beta", [1e-38, 1e-40, 1e-45, -0.5, 0.0])
@pytest.mark.parametrize("length", [1.0, 1e-15, 1e15])
def test_betas_at_the_ends_of_their_range(beta, length):
    """Every third row: betas below the normal numbers, negative ones, and none; beside keys of any length."""
    x, s0 = inputs(130, 2, 2, seed=53), state(2)
    q, k, v, g, b = x
    k[1::5] = (k[1::5].float() * length).to(torch.bfloat16)
    b[1::5] *= length ** -2
    b[::3] = beta if beta > -0.1 else beta * b[::3].sign() / k[::3].float().square().sum(2).clamp(min=1.0)
    out, last = prefill(x, s0)
    want, states, size, mass = rule(*x, SCALE, s0[0])
    check_bits(last, states[-1], torch.stack([norms(s) for s in states]).amax(0))


@pytest.mark.parametrize("length", [1e3, 1e5])
def test_long_values_with_small_betas(length):
    x, s0 = inputs(130, 2, 2, seed=42), state(2)
    q, k, v, g, beta = x
    at = [17, 63, 90]
    v[at] = (v[at].float() * length).to(torch.bfloat16)
    beta[at] = 1 / length
    out, last = prefill(x, s0)
    want, states, _, _ = rule(*x, SCALE, s0[0])
    check_bits(last, states[-1], torch.stack([norms(s) for s in states]).amax(0))


@pytest.mark.parametrize("gate,beta", [(-0.41, 1e-16), (-0.5, 0.5), (-1.2, 0.5), (-0.5, 1e-12)])
def test_state_that_decayed_without_updates(gate, beta):
    """64 rows take a state down by 2^-38 to 2^-111 and bring nothing; the next rows act on what is left of it."""
    x, s0 = inputs(256, 2, 2, seed=43), state(2)
    q, k, v, g, b = x
    g[:64], g[64:] = gate, 0.0
    b[:64], b[64:] = 0.0, beta
    if beta > 1e-3:
        v[64:] = 0.0                # beta erases
    out, last = prefill(x, s0)
    want, states, _, _ = rule(*x, SCALE, s0[0])
    left = [norms(s) for s in states[63:]]
    assert torch.isfinite(last).all() and torch.isfinite(out).all()
    check_bits(last, states[-1], torch.stack(left).amax(0))
    # outputs behind the decay, relative to what is left: half a bf16 step and the operands' 11 bits
    tol = 2.0 ** -8 * want[64:].abs() + 2.0 ** -8 * SCALE * q[64:].double().norm(dim=2)[..., None] * torch.stack(left).amax(0)[None, :, None]
    assert ((out[64:].double() - want[64:]).abs() <= tol).all()


@pytest.mark.parametrize("size", [1e-30, 1e-36, 0.0])
def test_states_that_are_nothing_beside_their_updates(size):
    x, s0 = inputs(200, 2, 2, seed=49), size * state(2)
    x[2][:64] *= 1e-30
    x[2][64:] *= 1e8
    out, last = prefill(x, s0)
    want, states, grown, mass = rule(*x, SCALE, s0[0])
    check_bits(last, states[-1], grown)
    check_out(out, want, 200, grown, mass, x[0])


@pytest.mark.parametrize("length", [1e15, 1e22, 1e26])
def test_large_queries_where_a_block_decays(length):
    """A channel that keeps its size for 15 rows and then falls by 2^-115."""
    x, s0 = inputs(130, 2, 2, seed=44), state(2)
    q, k, v, g, beta = x
    q.copy_((q.float() * length).to(torch.bfloat16))
    g[:, :, 3] = -0.001
    g[15::16, :, 3] = -79.0
    out, last = prefill(x, s0)
    want, states, size, mass = rule(*x, SCALE, s0[0])
    check_out(out, want, 130, size, mass, q)
    check_bits(last, states[-1], size)


@pytest.mark.parametrize("power", [-20, -30, -40, -60])
def test_small_queries_among_ordinary_ones(power):
    """A row's outputs are relative to its own query."""
    x, s0 = inputs(130, 2, 2, seed=45), state(2)
    x[0][::3] *= 2.0 ** power
    out, last = prefill(x, s0)
    want, states, size, mass = rule(*x, SCALE, s0[0])
    check_out(out, want, 130, size, mass, x[0])


@pytest.mark.parametrize("scale", [0.0, -0.25, 1e20, 1e-20, -1e-3])
def test_scales(scale):
    x, s0 = inputs(130, 2, 2, seed=46), state(2)
    out, last = prefill(x, s0, scale)
    want, states, size, mass = rule(*x, scale, s0[0])
    check_out(out, want, 130, size, mass, x[0], scale)
    check_bits(last, states[-1], size)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("rows", [10, 130])
def test_states_that_are_no_numbers(bad, rows):
    """Their value row is lost, the others are not."""
    x, s0 = inputs(rows, 2, 2, seed=47), state(2)
    good, good_last = prefill(x, s0)
    s0[0, 1, 77, 5] = bad
    out, last = prefill(x, s0)
    keep = torch.ones((2, DIM), dtype=torch.bool, device="cuda")
    keep[1, 77] = False
    assert not torch.isfinite(out[:, 1, 77]).any() and not torch.isfinite(last[1, 77]).any()
    assert torch.equal(out[:, keep], good[:, keep]) and torch.equal(last[keep], good_last[keep])


@pytest.mark.parametrize("heads,qk,gate", [(2, 2, "head"), (6, 2, "channel"), (6, 2, "head")])
@pytest.mark.parametrize("what", ["fast", "resets", "growing", "nan", "inf"])
def test_paths_beside_the_tensor_cores(heads, qk, gate, what):
    """Decays that leave a block's range, and chunks that go row by row: one decay a head, shared queries and keys."""
    n, at = 150, 77
    x, s0 = inputs(n, heads, qk, gate, seed=48), state(heads)
    q, k, v, g, beta = x
    if what == "fast":
        g.fill_(-8.0)
        g[:, ::2] = -0.01
    elif what == "resets":
        g[::7] = -math.inf
    elif what == "growing":
        g[30:90] = 0.2
    elif what == "nan":
        v[at, 1, 9] = math.nan
    else:
        beta[at, 1] = math.inf
    out, last = prefill(x, s0)
    want, states, size, mass = rule(*x, SCALE, s0[0])
    if what in ("nan", "inf"):
        check_out(out[:at], want[:at], n, rule(*(t[:at] for t in x), SCALE, s0[0])[2], mass[:at], q[:at])
        assert torch.equal(torch.isfinite(out), torch.isfinite(want)) and torch.equal(torch.isfinite(last), torch.isfinite(states[-1]))
    else:
        check_out(out, want, n, size, mass, q)
        assert (norms(last.double() - states[-1]) <= state_tolerance(n, size)).all()


def test_descriptors_follow_tensors_that_get_other_storage():
    x, s0 = inputs(40, 2, 2, seed=51), state(2)
    y, s1 = inputs(40, 2, 2, seed=52), state(2, seed=9)
    pool, rows = torch.cat([s0, torch.zeros_like(s0)]), B.DeltaRows(*x, SCALE)
    states, out, st = B.StatePool(pool), torch.zeros((40, 2, DIM), dtype=torch.bfloat16, device="cuda"), ints(0)
    ws = B.workspace(B.gated_delta_prefill_workspace_size(40, 1, 2))
    for new, first in ((x, s0), (y, s1)):
        for t, n in zip(x, new):
            t.data = n.clone()
        pool.data = torch.cat([first, torch.zeros_like(first)])
        B.gated_delta_prefill(states, rows, ints(0, 40), ints(0), ints(1), out, ws, st)
        want, after, size, mass = rule(*new, SCALE, first[0])
        assert st.item() == 0
        check_out(out, want, 40, size, mass, new[0])
        check_bits(pool[1], after[-1], size)


@pytest.mark.parametrize("rows,heads,qk,gate", [(n, 4, qk, gate) for n in (21, 64, 65, 130, 333, 2085)
                                                for qk, gate in ((4, "channel"), (2, "head"))] + [(16385, 1, 1, "channel")])
def test_states_keep_the_operands_bits(rows, heads, qk, gate):
    x, s0 = inputs(rows, heads, qk, gate, seed=rows), state(heads)
    out, last = prefill(x, s0)
    want, states, size, mass = rule(*x, SCALE, s0[0])
    check_bits(last, states[-1], size)


@pytest.mark.parametrize("gate", ["channel", "head"])
def test_outputs_have_no_bias(gate):
    """Over a million outputs.  A rounding to nearest has no bias, and to bf16 a relative error of 1.7e-3 rms, so the factor
    that fits the outputs best is within 2e-6 of one; operands cut to 11 bits instead of rounded make it 3.5e-4 smaller."""
    x, s0 = inputs(2048, 4, 4, gate, seed=50), state(4)
    out, last = prefill(x, s0)
    want = rule(*x, SCALE, s0[0])[0]
    assert abs(float((out.double() * want).sum() / want.square().sum()) - 1) <= 2.0 ** -15


@pytest.mark.parametrize("gate", ["channel", "head"])
def test_outputs_are_hardly_less_exact_than_bf16(gate):
    """The roundings to 11 bits (S, U, Q P, B and the queries in B, each within 2^-11 and 2^-11 / sqrt(3) / 2 = 1.4e-4 rms) add
    sqrt(1 + 5 (1.4e-4 / 1.66e-3)^2) - 1 = 2 % to the rounding to bf16; one operand of 8 bits (1.1e-3) can add a fifth."""
    x, s0 = inputs(2048, 4, 4, gate, seed=50), state(4)
    out, last = prefill(x, s0)
    want = rule(*x, SCALE, s0[0])[0]
    least = (want.to(torch.bfloat16).double() - want).square().mean().sqrt()
    assert float((out.double() - want).square().mean().sqrt() / least) <= 1.05
