"""Plain 64-bit forms (torch, CPU) of attention over a synthetic case's whole
context: latents decoded from the pool's bytes, logits, softmax, outputs, and
the attention weight of every token.  They share no code with the package's
kernels or with the C oracle."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def e4m3(b):
    return torch.from_numpy(np.ascontiguousarray(b)).view(torch.float8_e4m3fn).to(torch.float64)


def latents(case, b, length=None):
    """float64 [L, 576]: sequence b's latents with the layer's scale."""
    L = int(case.seq_lens[b]) if length is None else length
    rec = case.latent_bytes()
    n = -(-L // 64)
    page = case.pool[case.block_table[b, :n], case.latent_off:case.latent_off + 64 * rec]
    r = page.reshape(n * 64, rec)[:L]
    if rec == 576:
        c = e4m3(r)
    else:
        c = torch.empty((L, 576), dtype=torch.float64)
        c[:, 0:512:2] = torch.from_numpy(E2M1[r[:, :256] & 15])
        c[:, 1:512:2] = torch.from_numpy(E2M1[r[:, :256] >> 4])
        c[:, :512] *= e4m3(r[:, 256:288]).repeat_interleave(16, 1)
        c[:, 512:] = e4m3(r[:, 288:])
    return c * case.latent_scale


def queries(case, row):
    return torch.from_numpy(case.q_mla[row].view(np.int16).copy()).view(torch.bfloat16).to(torch.float64)


def attend(case, row, tokens=None, c=None):
    """(out [96, 512], lse [96], weight bound Sum_t p |v|, Sum_t p |v - out|, logits' bound) of one row over
    the given tokens (None: every visible one)."""
    b, j = row // case.nq, row % case.nq
    c = latents(case, b) if c is None else c
    vis = max(0, int(case.seq_lens[b]) - (case.nq - 1) + j)
    c = c[:vis] if tokens is None else c[tokens]
    if c.shape[0] == 0:
        z = torch.zeros((96, 512), dtype=torch.float64)
        return z, torch.full((96,), -np.inf, dtype=torch.float64), z, z, torch.zeros(96, dtype=torch.float64)
    q = queries(case, row)
    x = q @ c.T * case.sm_scale
    p = torch.softmax(x, 1)
    v = c[:, :512]
    out = p @ v
    # Sum p |v - out| <= sqrt(Sum p (v - out)^2), as p sums to one
    spread = torch.sqrt(torch.clamp(p @ (v * v) - out * out, min=0.0))
    bound = (q.abs() @ c.abs().T * abs(case.sm_scale)).amax(1)
    return out, torch.logsumexp(x, 1), p @ v.abs(), spread, bound
