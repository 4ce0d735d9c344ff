"""Cases and plain forms of the Mamba-2 serving and normalisation operators.

Four families, as a program that serves or trains Mamba-2 layers calls them:

* ``prompt``: the scalar-decay scan (SSD) over packed prompts of different
  lengths, with the requests' states in slots of a cache
  (``ssd_packed_fwd``).
* ``token``: one decode step of the same recurrence for a batch of requests
  (``ssd_state_update``).
* ``conv``: the short causal depthwise convolution in front of it, over
  packed prompts (``conv_packed_fwd``) or one token per request
  (``conv_packed_update``).
* ``norm``: the RMS norm before a block (fused with the residual sum and its
  scale) and after it (fused with the SiLU gate, by groups of channels),
  forward (``norm_fwd``) and backward (``norm_bwd``).

Where ``own`` is false, ``run`` computes the same from elementary torch
operations in 32 bits (in 64 bits where running sums of the decay are
subtracted), rounding once at the end.
"""
import math
import random

import torch

own = False

P, N = 64, 128   # head dimension and state size of the scan over prompts


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # three short prompts that arrive together at a 24-head layer (d_inner 1536): latency counts;
        # the gate is applied in the scan
        dict(name="prompt_short", op="prompt", nseq=3, shortest=1, total=378, heads=24, groups=1, z=True,
             resumed=False, lens=1),
        # a serving step of 16 ragged prompts through a 64-head layer (d_inner 4096), half of them
        # continuing from a cached state (chunked prefill)
        dict(name="prompt_ragged", op="prompt", nseq=16, shortest=64, total=24000, heads=64, groups=1,
             z=False, resumed=True, lens=2),
        # one long document through a 24-head layer: fewer heads than SMs, a long token axis
        dict(name="prompt_long", op="prompt", nseq=1, shortest=32768, total=32768, heads=24, groups=1,
             z=False, resumed=False, lens=3),
        # decode of a few requests (80 heads, d_inner 5120): latency counts
        dict(name="token_few", op="token", batch=2, slots=5, heads=80, groups=1, headdim=64, dstate=128,
             dtype="bf16", pads=0, z=True),
        # decode of a full batch of 256 requests, padded to it with a few empty places
        dict(name="token_many", op="token", batch=256, slots=270, heads=64, groups=1, headdim=64, dstate=128,
             dtype="bf16", pads=5, z=False),
        # the convolution over x, B and C of the ragged prompts (4096 + 2 * 128 channels)
        dict(name="conv_prompts", op="conv", tokens=24000, nseq=16, channels=4352, width=4, dtype="bf16", update=False,
             resumed=True, lens=2),
        # short prompts in float32, a channel count that is no multiple of 8, width 3
        dict(name="conv_odd_f32", op="conv", tokens=777, nseq=9, channels=1333, width=3, dtype="f32", update=False,
             resumed=True, lens=5),
        # decode step of the convolution for 256 requests
        dict(name="conv_tokens", op="conv", tokens=256, nseq=256, channels=4352, width=4, dtype="bf16", update=True,
             resumed=True, lens=6),
        # the norm after the scan, gated, in 8 groups (training or prefill of 16384 tokens, d_inner 4096)
        dict(name="norm_gated", op="norm", rows=16384, dim=4096, group=512, dtype="bf16", res="", z=True,
             gate_first=True, back=False),
        # the norm before a block at decode: 64 rows of d_model 2048, residual stream in float32
        dict(name="norm_residual_decode", op="norm", rows=64, dim=2048, group=2048, dtype="bf16", res="f32", z=False,
             gate_first=True, back=False),
        # backward of the gated norm
        dict(name="norm_gated_back", op="norm", rows=16384, dim=4096, group=512, dtype="bf16", res="", z=True,
             gate_first=True, back=True),
        # backward of the norm before a block, float32, odd sizes
        dict(name="norm_residual_back_f32", op="norm", rows=4099, dim=1530, group=1530, dtype="f32", res="f32",
             z=False, gate_first=True, back=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "token", "conv", "conv", "norm", "norm", "norm"])
    if op == "prompt":
        heads, groups = rng.choice([(24, 1), (64, 1), (80, 1), (64, 8), (5, 1), (12, 3), (32, 2)])
        nseq = _log(rng, 1, 48)
        total = max(nseq, _log(rng, 64, 1500000 // heads))
        return dict(op=op, nseq=nseq, shortest=rng.choice([0, 1, 1, 64]), total=total, heads=heads,
                    groups=groups, z=rng.random() < 0.4, resumed=rng.random() < 0.6, lens=rng.randrange(1 << 20))
    if op == "token":
        heads, groups = rng.choice([(24, 1), (64, 1), (80, 1), (64, 8), (7, 1), (32, 2)])
        headdim, dstate = rng.choice([(64, 128), (64, 128), (64, 64), (32, 16), (48, 96), (128, 256), (64, 37)])
        batch = _log(rng, 1, max(1, min(512, 130000000 // (heads * headdim * dstate))))
        return dict(op=op, batch=batch, slots=batch + rng.randrange(1, 20), heads=heads, groups=groups,
                    headdim=headdim, dstate=dstate, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    pads=rng.randrange(0, 1 + batch // 4), z=rng.random() < 0.5)
    if op == "conv":
        channels = rng.choice([1792, 4352, 5376, 8448, 100, 1333, _log(rng, 8, 6000)])
        update = rng.random() < 0.4
        nseq = _log(rng, 1, 600) if update else _log(rng, 1, 64)
        tokens = nseq if update else max(nseq, _log(rng, 1, 100000000 // max(channels, 3500)))
        return dict(op=op, tokens=tokens, nseq=nseq, channels=channels, width=rng.choice([4, 4, 4, 2, 3]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), update=update, resumed=rng.random() < 0.7,
                    lens=rng.randrange(1 << 20))
    dim = rng.choice([768, 1536, 2048, 2560, 4096, 5120, 8192, 1530, _log(rng, 1, 10000)])
    group = rng.choice([dim, dim] + [dim // k for k in (2, 8, 10) if dim % k == 0])
    rows = _log(rng, 1, 32000000 // max(dim, 1000))
    res = rng.choice(["", "", "f32", "same"])
    return dict(op=op, rows=rows, dim=dim, group=group, dtype=rng.choice(["bf16", "bf16", "f32"]), res=res,
                z=(res == "" and rng.random() < 0.7) or rng.random() < 0.15, gate_first=rng.random() < 0.7,
                back=rng.random() < 0.5)


def _lens(case, total, shortest=0):
    """Ragged sequence lengths that sum to ``total``, the case's own."""
    g = random.Random(case["lens"])
    n = case["nseq"]
    lo = min(shortest, total // n)
    w = [g.random() ** 2 + 0.02 for _ in range(n)]
    s = sum(w)
    lens = [lo + int((total - lo * n) * v / s) for v in w]
    lens[g.randrange(n)] += total - sum(lens)
    return lens


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


# ---- inputs ----------------------------------------------------------------

class _Rng:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=self.g) * scale).to(dtype)

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, device="cuda", generator=self.g) * (hi - lo) + lo

    def slots(self, slots, n, pads=0):
        """n distinct slots in a random order, the last ``pads`` places empty (-1)."""
        idx = torch.randperm(slots, device="cuda", generator=self.g)[:n].to(torch.int32)
        if pads:
            idx[n - pads:] = -1
        return idx


def _head_params(r, heads):
    dt = torch.exp(r.uniform(heads, lo=math.log(1e-3), hi=math.log(1e-1)))
    return dict(A=-r.uniform(heads, lo=1.0, hi=16.0), D=r.uniform(heads, lo=0.5, hi=1.5),
                dt_bias=torch.log(torch.expm1(dt)))


def prepare(case, seed):
    r = _Rng(seed)
    s = dict(case=dict(case))
    if case["op"] == "prompt":
        lens = _lens(case, case["total"], case["shortest"])
        T, H, G, n = sum(lens), case["heads"], case["groups"], len(lens)
        # x, B and C are slices of the convolution's output, dt and z of the input projection
        xbc = r.normal(T, H * P + 2 * G * N, dtype=torch.bfloat16)
        proj = r.normal(T, H * P + (H + 7) // 8 * 8, dtype=torch.bfloat16)
        proj[:, H * P:] *= 0.5
        s.update(_head_params(r, H), x=xbc[:, :H * P].unflatten(1, (H, P)),
                 B=xbc[:, H * P:H * P + G * N].unflatten(1, (G, N)), C=xbc[:, H * P + G * N:].unflatten(1, (G, N)),
                 z=proj[:, :H * P].unflatten(1, (H, P)) if case["z"] else None, dt=proj[:, H * P:H * P + H],
                 cu=torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32), longest=max(lens),
                 cache=r.normal(n + 3, H, P, N), slots=r.slots(n + 3, n),
                 resumed=torch.arange(n, device="cuda") % 2 == 0 if case["resumed"] else None,
                 y=torch.zeros(T, H, P, dtype=torch.bfloat16, device="cuda"))
    elif case["op"] == "token":
        b, H, G, p, N_ = (case[k] for k in ("batch", "heads", "groups", "headdim", "dstate"))
        dt = _dtype(case["dtype"])
        xbc = r.normal(b, H * p + 2 * G * N_, dtype=dt)
        s.update(_head_params(r, H), x=xbc[:, :H * p].unflatten(1, (H, p)),
                 B=xbc[:, H * p:H * p + G * N_].unflatten(1, (G, N_)), C=xbc[:, H * p + G * N_:].unflatten(1, (G, N_)),
                 z=r.normal(b, H, p, dtype=dt) if case["z"] else None, dt=r.normal(b, H, dtype=dt, scale=0.5),
                 cache=r.normal(case["slots"], H, p, N_), slots=r.slots(case["slots"], b, case["pads"]),
                 y=torch.zeros(b, H, p, dtype=dt, device="cuda"))
    elif case["op"] == "conv":
        c, w, n, dt = case["channels"], case["width"], case["nseq"], _dtype(case["dtype"])
        lens = [1] * n if case["update"] else _lens(case, case["tokens"])
        proj = r.normal(sum(lens), c + 64, dtype=dt)   # a slice of the input projection
        s.update(x=proj[:, 64:], weight=r.uniform(c, w, lo=-0.5, hi=0.5), bias=r.uniform(c, lo=-0.5, hi=0.5),
                 cu=torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32),
                 cache=r.normal(n + 3, w - 1, c, dtype=dt), slots=r.slots(n + 3, n),
                 resumed=torch.arange(n, device="cuda") % 3 != 1 if case["resumed"] else None,
                 y=torch.zeros(sum(lens), c, dtype=dt, device="cuda"))
    else:
        R, d, dt = case["rows"], case["dim"], _dtype(case["dtype"])
        s.update(x=r.normal(R, d, dtype=dt), weight=r.uniform(d, lo=0.5, hi=1.5),
                 z=r.normal(R, d, dtype=dt) if case["z"] else None, residual=None, scale=1.0, dsum=None)
        if case["res"]:
            s.update(residual=r.normal(R, d, dtype=dt if case["res"] == "same" else torch.float32), scale=0.75)
        if case["back"]:
            s.update(dy=r.normal(R, d, dtype=dt))
            if case["res"]:   # the sum that the forward stored, and the gradient that reaches it from later blocks
                s.update(dsum=r.normal(R, d, dtype=s["residual"].dtype))
                s.update(total=(s["residual"].float() + s["scale"] * _branch(s)).to(s["residual"].dtype))
    return s


# ---- the operators in their plain form -------------------------------------

def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _branch(s):
    """What enters the norm or the residual sum: x, or x silu(z)."""
    x = s["x"].float()
    return x * _silu(s["z"].float()) if s["z"] is not None and s["case"]["gate_first"] else x


def _live(s):
    """Requests that run (slot >= 0) and their slots."""
    run = torch.nonzero(s["slots"] >= 0)[:, 0] if s["case"].get("pads") else torch.arange(len(s["slots"]), device="cuda")
    return run, s["slots"][run].long()


def _prompt(s):
    """Chunks of 128 tokens of the padded sequences: the quadratic form inside a
    chunk, and a decay matrix over the chunks for the states between them."""
    Q = 128
    cu, n, H = s["cu"].long(), len(s["slots"]), s["case"]["heads"]
    hpg = H // s["case"]["groups"]
    nc = max(1, -(-s["longest"] // Q))
    at = cu[:-1, None] + torch.arange(nc * Q, device="cuda")
    inside = at < cu[1:, None]
    rows = torch.where(inside, at, 0)

    def padded(v):   # (n, nc, Q, heads or groups, ...)
        v = v.float()[rows] * inside.view(n, nc * Q, *[1] * (v.dim() - 1))
        return v.unflatten(1, (nc, Q))

    x, B, C = padded(s["x"]), padded(s["B"]), padded(s["C"])
    delta = _softplus(padded(s["dt"]) + s["dt_bias"]) * inside.view(n, nc, Q, 1)
    a = torch.cumsum((delta * s["A"]).double().permute(0, 3, 1, 2), -1)   # (n, H, nc, Q)
    xd = x * delta[..., None]
    causal = torch.ones(Q, Q, dtype=torch.bool, device="cuda").tril()
    scores = torch.einsum("nctgk,ncugk->ngctu", C, B)
    y = torch.empty_like(x)
    start = s["cache"][s["slots"].long()] if s["resumed"] is not None else torch.zeros_like(s["cache"][:n])
    if s["resumed"] is not None:
        start = start * s["resumed"].view(n, 1, 1, 1)
    last = torch.empty_like(start)
    ends = a[..., -1]                                                       # (n, H, nc)
    before = torch.cumsum(ends, -1) - ends                                  # decay up to each chunk
    steps = torch.cat([before, (before + ends)[..., -1:]], -1)              # (n, H, nc + 1)
    earlier = torch.ones(nc + 1, nc, dtype=torch.bool, device="cuda").tril(-1)
    for h in range(0, H, 8):                                                # 8 heads at a time: bounded memory
        k = slice(h, min(h + 8, H))
        g = torch.arange(k.start, k.stop, device="cuda") // hpg
        decay = torch.where(causal, a[:, k, :, :, None] - a[:, k, :, None, :], -math.inf).exp().float()
        yd = torch.einsum("nhctu,ncuhp->ncthp", scores[:, g] * decay, xd[..., k, :])
        w = (ends[:, k, :, None] - a[:, k]).exp().float()
        states = torch.einsum("nhcu,ncuhk,ncuhp->nchpk", w, B[:, :, :, g], xd[..., k, :])
        between = torch.where(earlier, steps[:, k, :, None] - (before + ends)[:, k, None, :], -math.inf).exp().float()
        into = torch.einsum("nhic,nchpk->nihpk", between, states)
        into = into + steps[:, k].exp().float().permute(0, 2, 1)[..., None, None] * start[:, None, k]
        yo = torch.einsum("nhct,ncthk,nchpk->ncthp", a[:, k].exp().float(), C[:, :, :, g], into[:, :-1])
        y[..., k, :] = yd + yo
        last[:, k] = into[:, -1]
    y = y + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(padded(s["z"]))
    s["y"][at[inside]] = y.flatten(1, 2)[inside].to(s["y"].dtype)
    s["cache"][s["slots"].long()] = last
    return {"y": s["y"], "state": s["cache"]}


def _token(s):
    run, slots = _live(s)
    hpg = s["case"]["heads"] // s["case"]["groups"]
    x, B, C = s["x"][run].float(), s["B"][run].float(), s["C"][run].float()
    delta = _softplus(s["dt"][run].float() + s["dt_bias"])
    B, C = B.repeat_interleave(hpg, 1), C.repeat_interleave(hpg, 1)
    h = s["cache"][slots] * torch.exp(delta * s["A"])[..., None, None]
    h = h + (delta[..., None] * x)[..., None] * B[:, :, None]
    y = (h * C[:, :, None]).sum(-1) + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(s["z"][run].float())
    s["cache"][slots] = h
    s["y"][run] = y.to(s["y"].dtype)
    return {"y": s["y"], "state": s["cache"]}


def _conv(s):
    cu, n, w = s["cu"].long(), len(s["slots"]), s["case"]["width"]
    T = s["x"].shape[0]
    slots = s["slots"].long()
    history = s["cache"][slots]
    if s["resumed"] is not None and not s["case"]["update"]:
        history = torch.where(s["resumed"].view(n, 1, 1), history, 0)
    elif not s["case"]["update"]:
        history = torch.zeros_like(history)
    # every sequence behind its history, in one row list
    rows = torch.cat([history.flatten(0, 1), s["x"]]).float()
    seq = torch.bucketize(torch.arange(T, device="cuda"), cu[1:], right=True)
    t = torch.arange(T, device="cuda") - cu[seq]
    acc = s["bias"].expand(T, -1)
    for k in range(w):
        back = t - (w - 1 - k)
        at = torch.where(back >= 0, n * (w - 1) + cu[seq] + back, seq * (w - 1) + (w - 1) + back)
        acc = acc + rows[at] * s["weight"][:, k]
    j = torch.arange(w - 1, device="cuda") + (cu[1:] - cu[:-1])[:, None]    # the last w - 1 rows of history and inputs
    first = torch.arange(n, device="cuda")[:, None]
    at = torch.where(j < w - 1, first * (w - 1) + j, n * (w - 1) + cu[:-1, None] + j - (w - 1))
    s["cache"][slots] = rows[at].to(s["cache"].dtype)
    s["y"].copy_(_silu(acc))
    return {"y": s["y"], "state": s["cache"]}


def _norm(s):
    case = s["case"]
    gs = case["group"]
    v = _branch(s)
    if s["residual"] is not None:
        v = s["residual"].float() + s["scale"] * v
    g = v.unflatten(1, (-1, gs))
    y = (g * torch.rsqrt((g * g).mean(-1, keepdim=True) + 1e-5)).flatten(1) * s["weight"]
    if s["z"] is not None and not case["gate_first"]:
        y = y * _silu(s["z"].float())
    out = {"y": y.to(s["x"].dtype)}
    if s["residual"] is not None:
        out["sum"] = v.to(s["residual"].dtype)
    return out


def _norm_back(s):
    case = s["case"]
    gs = case["group"]
    x, dy, w = s["x"].float(), s["dy"].float(), s["weight"]
    v = s["total"].float() if s["residual"] is not None else _branch(s)
    g = v.unflatten(1, (-1, gs))
    rstd = torch.rsqrt((g * g).mean(-1, keepdim=True) + 1e-5)
    unit = (g * rstd).flatten(1)
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        sig = 1 / (1 + torch.exp(-z))
        slope = sig * (1 + z * (1 - sig))
        if not case["gate_first"]:
            out["dz"] = (dy * unit * w * slope).to(s["x"].dtype)
            dy = dy * z * sig
    out["dweight"] = (dy * unit).sum(0)
    u = (dy * w).unflatten(1, (-1, gs))
    n = unit.unflatten(1, (-1, gs))
    dv = ((u - n * (u * n).mean(-1, keepdim=True)) * rstd).flatten(1)
    if s["residual"] is not None:
        dv = dv + s["dsum"].float()
        out["dresidual"] = dv.to(s["residual"].dtype)
        dv = s["scale"] * dv
    if s["z"] is not None and case["gate_first"]:
        out["dz"] = (dv * x * slope).to(s["x"].dtype)
        dv = dv * z * sig
    out["dx"] = dv.to(s["x"].dtype)
    return out


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    if op == "prompt":
        return _prompt(s)
    if op == "token":
        return _token(s)
    if op == "conv":
        return _conv(s)
    return _norm_back(s) if s["case"]["back"] else _norm(s)


def _own(s):
    import selective_state_space_27_b200 as ms
    case = s["case"]
    if case["op"] == "prompt":
        ms.ssd_packed_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                          state=s["cache"], state_indices=s["slots"], has_initial_state=s["resumed"],
                          max_seqlen=s["longest"], out=s["y"], check=False)
        return {"y": s["y"], "state": s["cache"]}
    if case["op"] == "token":
        ms.ssd_state_update(s["cache"], s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                            dt_bias=s["dt_bias"], state_indices=s["slots"], out=s["y"])
        return {"y": s["y"], "state": s["cache"]}
    if case["op"] == "conv":
        if case["update"]:
            ms.conv_packed_update(s["cache"], s["x"], s["weight"], bias=s["bias"], state_indices=s["slots"],
                                  out=s["y"])
        else:
            ms.conv_packed_fwd(s["x"], s["weight"], s["cu"], bias=s["bias"], state=s["cache"],
                               state_indices=s["slots"], has_initial_state=s["resumed"], out=s["y"])
        return {"y": s["y"], "state": s["cache"]}
    kw = dict(weight=s["weight"], z=s["z"], group_size=case["group"], gate_first=case["gate_first"])
    if case["back"]:
        g = ms.norm_bwd(s["dy"], s["x"], residual_out=s["total"] if s["residual"] is not None else None,
                        dresidual_out=s["dsum"], residual_scale=s["scale"], **kw)
        return {k: v for k, v in g.items() if v is not None}
    y, total = ms.norm_fwd(s["x"], residual=s["residual"], residual_scale=s["scale"], **kw)
    return {"y": y} if total is None else {"y": y, "sum": total}


# ---- work ------------------------------------------------------------------

def work(case):
    eb = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "prompt":
        lens = _lens(case, case["total"], case["shortest"])
        T, H, G, n = sum(lens), case["heads"], case["groups"], len(lens)
        state = n * H * P * N * 4
        read = (n + 1) // 2 if case["resumed"] else 0
        return {"bytes": T * H * P * 2 * (3 if case["z"] else 2) + T * G * N * 4 + T * H * 2 + state + state * read // n,
                "flops": 4 * T * H * P * N}
    if case["op"] == "token":
        b, H, G, p, N_ = case["batch"] - case["pads"], case["heads"], case["groups"], case["headdim"], case["dstate"]
        return {"bytes": b * H * p * N_ * 8 + b * H * p * eb * (3 if case["z"] else 2) + b * G * N_ * 2 * eb,
                "flops": 5 * b * H * p * N_}
    if case["op"] == "conv":
        T, c, w, n = case["tokens"], case["channels"], case["width"], case["nseq"]
        return {"bytes": 2 * T * c * eb + n * (w - 1) * c * eb * (2 if case["resumed"] or case["update"] else 1)
                + c * (w + 1) * 4, "flops": T * c * (2 * w + 4)}
    R, d = case["rows"], case["dim"]
    rb = 0 if not case["res"] else 4 if case["res"] == "f32" else eb
    if case["back"]:
        # dy and dx; x (and z, dz) where the branch enters by itself or through the gate; the stored sum, the
        # gradients that reach and leave it
        per = 2 * eb + (2 * eb if case["z"] else 0) + 3 * rb
        per += eb if not rb or (case["z"] and case["gate_first"]) else 0
        return {"bytes": R * d * per + 2 * d * 4, "flops": 12 * R * d}
    return {"bytes": R * d * (2 * eb + (eb if case["z"] else 0) + 2 * rb) + d * 4, "flops": 6 * R * d}


# ---- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    """The recurrences token by token, the sums and the gradients in 64 bits."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "prompt":
        lens = (s["cu"][1:] - s["cu"][:-1]).tolist()
        starts = s["cu"].tolist()
        if max(lens) * len(lens) * case["heads"] > 16_000_000:
            return None
        order = sorted(range(len(lens)), key=lambda i: -lens[i])            # the running ones stay in front
        slot = s["slots"].long()[order]
        hpg = case["heads"] // case["groups"]
        h = torch.zeros(len(lens), case["heads"], P, N, dtype=f64, device="cuda")
        if s["resumed"] is not None:
            keep = s["resumed"][order]
            h[keep] = s["cache"][slot][keep].to(f64)
        delta = torch.logaddexp(s["dt"].to(f64) + s["dt_bias"].to(f64), torch.zeros((), dtype=f64, device="cuda"))
        factor = (delta * s["A"].to(f64)).exp()
        y = s["y"].to(f64)
        first = torch.tensor([starts[i] for i in order], device="cuda")
        alive = len(lens)
        for t in range(max(lens)):
            while alive and lens[order[alive - 1]] <= t:
                alive -= 1
            at = first[:alive] + t
            xt, dt = s["x"][at].to(f64), delta[at]
            Bt = s["B"][at].to(f64).repeat_interleave(hpg, 1)
            Ct = s["C"][at].to(f64).repeat_interleave(hpg, 1)
            ht = h[:alive]
            ht.mul_(factor[at][..., None, None]).addcmul_((dt[..., None] * xt)[..., None], Bt[:, :, None])
            y[at] = torch.matmul(ht, Ct[..., None])[..., 0]
        y = y + s["D"].to(f64)[:, None] * s["x"].to(f64)
        if s["z"] is not None:
            z = s["z"].to(f64)
            y = y * z * torch.sigmoid(z)
        state = s["cache"].to(f64)
        state[slot] = h
        return {"y": y, "state": state}
    if case["op"] == "token":
        state, y = s["cache"].to(f64), s["y"].to(f64)
        hpg = case["heads"] // case["groups"]
        for i, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            x, dt = s["x"][i].to(f64), s["dt"][i].to(f64) + s["dt_bias"].to(f64)
            dt = torch.logaddexp(dt, torch.zeros_like(dt))
            heads = torch.arange(case["heads"], device="cuda") // hpg
            B, C = s["B"][i].to(f64)[heads], s["C"][i].to(f64)[heads]
            h = state[slot] * (dt * s["A"].to(f64)).exp()[:, None, None] + torch.einsum("h,hp,hk->hpk", dt, x, B)
            state[slot] = h
            y[i] = torch.einsum("hpk,hk->hp", h, C) + s["D"].to(f64)[:, None] * x
            if s["z"] is not None:
                z = s["z"][i].to(f64)
                y[i] *= z * torch.sigmoid(z)
        return {"y": y, "state": state}
    if case["op"] == "conv":
        w = case["width"]
        y, state, starts = s["y"].to(f64), s["cache"].to(f64), s["cu"].tolist()
        filt = s["weight"].to(f64).flip(1)
        for i, slot in enumerate(s["slots"].tolist()):
            x = s["x"][starts[i]:starts[i + 1]].to(f64)
            past = state[slot].clone()
            if not case["update"] and (s["resumed"] is None or not bool(s["resumed"][i])):
                past.zero_()
            x = torch.cat([past, x])
            state[slot] = x[x.shape[0] - (w - 1):]
            n = x.shape[0] - (w - 1)
            v = s["bias"].to(f64) + sum(filt[:, k] * x[w - 1 - k:w - 1 - k + n] for k in range(w))
            y[starts[i]:starts[i + 1]] = v * torch.sigmoid(v)
        return {"y": y, "state": state}
    x, w = s["x"].to(f64).requires_grad_(), s["weight"].to(f64).requires_grad_()
    z = None if s["z"] is None else s["z"].to(f64).requires_grad_()
    v = x * z * torch.sigmoid(z) if z is not None and case["gate_first"] else x
    res = None
    if s["residual"] is not None:
        # the backward starts from the sum as it was stored: its value, with the gradients of its parts
        res = s["residual"].to(f64).requires_grad_()
        v = res + s["scale"] * v
        if case["back"]:
            v = v + (s["total"].to(f64) - v).detach()
    g = v.reshape(case["rows"], -1, case["group"])
    y = (g / torch.sqrt(g.square().mean(-1, keepdim=True) + 1e-5)).reshape(case["rows"], -1) * w
    if z is not None and not case["gate_first"]:
        y = y * z * torch.sigmoid(z)
    if not case["back"]:
        return {"y": y.detach()} if res is None else {"y": y.detach(), "sum": v.detach()}
    loss = (y * s["dy"].to(f64)).sum()
    if s["dsum"] is not None:
        loss = loss + (v * s["dsum"].to(f64)).sum()
    leaves = {"dx": x, "dweight": w}
    if z is not None:
        leaves["dz"] = z
    if res is not None:
        leaves["dresidual"] = res
    return dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
