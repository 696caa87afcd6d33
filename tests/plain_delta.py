"""The gated delta rule row by row in 64 bits, and inputs for its tests.  It
shares no code with the package's kernels."""
import torch

DIM = 128


def rule(q, k, v, gate, beta, scale, S):
    """(out [n, heads, 128], the states after each row, the largest Frobenius norm a head's state and value had, the
    outputs' magnitude) of one sequence's rows in float64, from the state S [heads, 128, 128].  The magnitude is the sum
    of the magnitudes of what a chunk of 64 rows adds up to an output: of the products of its first state's elements, and
    of its rows' updates, with the query."""
    heads = v.shape[1]
    of = torch.arange(heads, device=v.device) // (heads // q.shape[1])
    q, k, v, beta = q.double()[:, of], k.double()[:, of], v.double(), beta.double()
    decay = torch.exp(gate.double())
    decay = decay if decay.dim() == 3 else decay[:, :, None].expand(-1, -1, DIM)
    S, out, states, mass = S.double(), [], [], []
    size = S.flatten(1).norm(dim=1)
    for t in range(v.shape[0]):
        if t % 64 == 0:
            parts = S.abs()
        parts = parts * decay[t][:, None, :]
        S = S * decay[t][:, None, :]
        u = beta[t][:, None] * (v[t] - (S @ k[t][:, :, None])[..., 0])
        S = S + u[:, :, None] * k[t][:, None, :]
        parts = parts + (u[:, :, None] * k[t][:, None, :]).abs()
        mass.append(abs(scale) * (parts @ q[t].abs()[:, :, None])[..., 0])
        out.append(scale * (S @ q[t][:, :, None])[..., 0])
        states.append(S)
        size = torch.maximum(size, S.flatten(1).norm(dim=1) + v[t].norm(dim=1))
    none = torch.zeros((0, heads, DIM), dtype=torch.float64, device=v.device)
    return (torch.stack(out) if out else none), states, size, (torch.stack(mass) if out else none)


def inputs(rows, heads, qk_heads, gate="channel", seed=0, device="cuda", apart=0):
    """Rows of a layer: queries and keys of at most length one, decays from 0.999 to 0.2 a row; `apart` more elements between rows."""
    g = torch.Generator(device=device).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=device)

    def spread(t):
        if not apart:
            return t.contiguous()
        wide = torch.full((rows, t[0].numel() + apart if rows else apart), float("nan"), device=device, dtype=t.dtype)
        wide[:, :wide.shape[1] - apart] = t.flatten(1)
        return wide[:, :wide.shape[1] - apart].unflatten(1, t.shape[1:])

    # 2^-8 below one, which bf16's rounding cannot make up for
    q, k = ((0.996 * torch.nn.functional.normalize(randn(rows, qk_heads, DIM), dim=2)).to(torch.bfloat16) for _ in "qk")
    v = randn(rows, heads, DIM).to(torch.bfloat16)
    rate = torch.exp(-7 + 7.4 * torch.rand((heads, DIM), generator=g, device=device))
    gate = -rate * torch.nn.functional.softplus(randn(rows, heads, DIM)) if gate == "channel" else \
        -rate[:, 0] * torch.nn.functional.softplus(randn(rows, heads))
    beta = torch.sigmoid(randn(rows, heads))
    return [spread(t) for t in (q, k, v, gate, beta)]


def state_tolerance(rows, size):
    """Largest |S - S64|_F of a head after `rows` rows, for keys no longer than one and beta in [0, 2].

    A step takes an error E to (E diag(decay)) (I - beta k k^T), no larger in the Frobenius norm, and adds roundings of
    half a step, 2^-24 relative, to numbers of the state's size: the decayed state 1, the decay itself 4 (two units in
    the last place of the exponential, counted as four halves), the product with the key 16 fused additions along a
    thread, three between lanes and beta's factor two (40), beta (v - p) 4, the update 1: 50 in all.  Prompts in chunks,
    whose operands are two fp16 parts (21 bits, one product of three left out), are held to the same."""
    return 50 * max(rows, 1) * 2.0 ** -24 * size


def out_tolerance(out64, rows, size, mass, q, scale, chunked):
    """|out - out64| elementwise: half a bf16 step, 2^-8 of the value, and the state's error and the product's own
    roundings (24) with a query, all in fp32.  Prompts in chunks also round the operands of the outputs' products, each
    relative to what it adds (`mass`): the state and the updates are cut to 11 bits (2^-10), the decayed queries and the
    products of queries and keys rounded to fp16 (2^-11), and in those products the query to bf16 (2^-8)."""
    fp32 = (state_tolerance(rows, size) + 24 * 2.0 ** -24 * size)[None, :, None] * abs(scale)
    of = torch.arange(out64.shape[1], device=q.device) // (out64.shape[1] // q.shape[1])
    off = fp32 * q.double().norm(dim=2)[:, of, None]
    if chunked:
        off = off + (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -11) * mass
    return 2.0 ** -8 * (out64.abs() + off) + off
