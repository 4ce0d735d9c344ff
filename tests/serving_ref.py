"""Definitions in 64 bits of the packed convolution, the SSD over packed
sequences and single tokens, and the norms, for their tests. Every reference
also gives the sum of the absolute values of what it adds up, from which the
tests derive how far a result may be off."""
import torch

F64 = torch.float64


def half(dtype):
    """Largest relative error of one rounding to this type."""
    return torch.finfo(dtype).eps / 2


U32 = half(torch.float32)


def silu(v):
    return v * torch.sigmoid(v)


def live_sequences(nseq, slots, idx):
    """[(sequence, slot)] of the sequences that run: the first user of every slot inside the cache."""
    seen, out = set(), []
    for s in range(nseq):
        slot = s if idx is None else int(idx[s])
        if 0 <= slot < slots and slot not in seen:
            seen.add(slot)
            out.append((s, slot))
    return out


def conv(x, weight, cu, bias=None, act=True, state=None, idx=None, init=None, y=None):
    """(y, state, absolute sums) of the packed convolution; y starts as given."""
    width = weight.shape[1]
    x, w = x.to(F64), weight.to(F64)
    y = y.to(F64).clone()
    mag = torch.zeros_like(y)
    new = None if state is None else state.to(F64).clone()
    nseq = len(cu) - 1
    b = torch.zeros(x.shape[1], dtype=F64, device=x.device) if bias is None else bias.to(F64)
    slots = nseq if state is None and idx is None else (len(state) if state is not None else 1 << 30)
    for s, slot in live_sequences(nseq, slots, idx):
        rows = x[cu[s]:cu[s + 1]]
        past = torch.zeros(width - 1, x.shape[1], dtype=F64, device=x.device)
        if state is not None and (init is None or init[s]) and width > 1 and init is not None:
            past = state[slot].to(F64)
        full = torch.cat([past, rows])
        n = len(rows)
        v, m = b.expand(n, -1).clone(), b.abs().expand(n, -1).clone()
        for k in range(width):
            v = v + w[:, k] * full[k:k + n]
            m = m + (w[:, k] * full[k:k + n]).abs()
        y[cu[s]:cu[s + 1]] = silu(v) if act else v
        mag[cu[s]:cu[s + 1]] = m
        if new is not None and width > 1:
            new[slot] = full[len(full) - (width - 1):]
    return y, new, mag


def ssd(x, dt, A, B, C, cu, D=None, z=None, dt_bias=None, softplus=True, state=None, idx=None, init=None, y=None,
        always=False):
    """(y, state, absolute sums of y, of state) of the SSD recurrence, token by token."""
    x, B, C, A = x.to(F64), B.to(F64), C.to(F64), A.to(F64)
    H, G = x.shape[1], B.shape[1]
    heads = torch.arange(H, device=x.device) // (H // G)
    B, C = B[:, heads], C[:, heads]
    delta = dt.to(F64) + (0 if dt_bias is None else dt_bias.to(F64))
    if softplus:
        delta = torch.logaddexp(delta, torch.zeros_like(delta))
    decay = (delta * A).exp()
    y = y.to(F64).clone()
    ymag = torch.zeros_like(y)
    new = None if state is None else state.to(F64).clone()
    smag = None if state is None else state.to(F64).abs()
    nseq = len(cu) - 1
    for s, slot in live_sequences(nseq, nseq if state is None else len(state), idx):
        h = torch.zeros(H, x.shape[2], B.shape[2], dtype=F64, device=x.device)
        if state is not None and (always or (init is not None and bool(init[s]))):
            h = state[slot].to(F64).clone()
        m = h.abs()
        for t in range(cu[s], cu[s + 1]):
            add = (delta[t][:, None] * x[t])[..., None] * B[t][:, None]
            h = h * decay[t][:, None, None] + add
            m = m * decay[t][:, None, None] + add.abs()
            y[t] = torch.einsum("hpn,hn->hp", h, C[t])
            ymag[t] = torch.einsum("hpn,hn->hp", m, C[t].abs())
            if D is not None:
                y[t] += D.to(F64)[:, None] * x[t]
                ymag[t] += (D.to(F64)[:, None] * x[t]).abs()
            if z is not None:
                g = silu(z[t].to(F64))
                y[t] *= g
                ymag[t] *= g.abs()
        if new is not None:
            new[slot], smag[slot] = h, m
    return y, new, ymag, smag


def norm(x, weight=None, z=None, residual=None, scale=1.0, eps=1e-5, group=None, gate_first=True, stored=None):
    """(y, sum) in 64 bits, differentiable; ``stored``: the value of the sum, with the gradients of its parts."""
    rows, dim = x.shape
    v = x * silu(z) if z is not None and gate_first else x
    if residual is not None:
        v = residual + scale * v
        if stored is not None:
            v = v + (stored - v).detach()
    g = v.reshape(rows, -1, group or dim)
    y = (g * torch.rsqrt(g.square().mean(-1, keepdim=True) + eps)).reshape(rows, dim)
    if weight is not None:
        y = y * weight
    if z is not None and not gate_first:
        y = y * silu(z)
    return y, v
