"""GPU tests of the serving operators and norms against their definitions in 64
bits (serving_ref.py).

Tolerances are per element and count roundings: u(t) = finfo(t).eps / 2 is the
largest relative error of one rounding to type t, and a sum of n terms in
float32 is off by at most about n u(f32) times the sum of its terms' absolute
values, which the references give ("mag").
* convolution: at most width + 1 terms, the SiLU and its steps (below 16 more
  float32 roundings; SiLU's slope is below 1.1), the rounding of y.
* single tokens: the state is two products and a sum with a decay whose
  exponent is rounded (|delta A| log2(e) u) and a step of a few roundings: 64
  roundings of its terms; y is a sum of dstate terms of that.
* SSD over prompts: y is built from M' and the state, each rounded to bf16
  once: u(bf16) of every term, u(bf16) of y itself, and a tenth of that for all
  float32 work. The state's terms are split into two bf16 values, off by
  u(bf16)^2 = 2^-16 of each, and as much again for the float32 work.
* norm: the mean is a sum of up to 32 terms per thread and a tree, so below 64
  roundings; every value is that many roundings of what it is made of.
"""
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

F64 = torch.float64
U32, UB = ref.U32, ref.half(torch.bfloat16)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ms():
    import selective_state_space_27_b200 as m
    return m


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def offsets(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu, torch.tensor(cu, dtype=torch.int32, device="cuda")


def close(got, want, tol):
    got = got.to(F64)
    assert torch.isfinite(got).all()
    over = (got - want).abs() - tol
    assert over.max().item() <= 0, f"over by {over.max().item():.3e} at a tolerance of {tol.flatten()[over.argmax()].item():.3e}"


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ---- convolution -----------------------------------------------------------------

def conv_tol(mag, want, dtype, width):
    return (width + 17) * 1.1 * U32 * (mag + want.abs()) + ref.half(dtype) * want.abs() * (1 if dtype != torch.float32 else 2)


CONV = [
    # lens, channels, width, dtype, slots, indices, resumed
    ([1], 8, 4, "bf16", 3, [2], [True]),
    ([0, 1, 2, 3, 4, 5], 100, 4, "f32", 6, None, [True, True, False, True, True, False]),
    ([3, 0, 0, 40, 129, 1], 1333, 3, "bf16", 9, [8, 7, 0, 1, 4, 2], [False, True, False, True, True, True]),
    ([700, 33, 1], 64, 4, "bf16", 3, [2, 1, 0], None),
    ([17, 250], 1, 2, "f32", 4, [3, 1], [True, False]),
    ([5, 300, 64], 24, 1, "bf16", 5, [1, 2, 3], None),
    # skipped: outside the cache, and the second user of a slot
    ([9, 40, 40, 2, 70], 48, 4, "bf16", 4, [1, -1, 1, 4, 0], [True] * 5),
    # more sequences than threads in a block, most of them short
    ([(7 * i) % 11 for i in range(400)], 40, 4, "f32", 500, list(range(499, 99, -1)), [i % 2 == 0 for i in range(400)]),
]


@pytest.mark.parametrize("lens,channels,width,dtype,slots,idx,resumed", CONV)
def test_conv_packed(ms, lens, channels, width, dtype, slots, idx, resumed):
    g, dt = rng(len(lens) + channels), DTYPES[dtype]
    cu, cu_t = offsets(lens, first=2)   # two rows in front and three behind belong to no sequence
    T = cu[-1] + 3
    wide = normal(g, T, channels + 16, dtype=dt)
    wide[:2] = float("nan")
    wide[cu[-1]:] = float("nan")
    x = wide[:, 16:]                    # a slice of wider rows
    weight, bias = normal(g, channels, width, scale=0.5), normal(g, channels)
    state = normal(g, slots, width - 1, channels, dtype=dt) if width > 1 else None
    flags = None if resumed is None else torch.tensor(resumed, device="cuda")
    out = torch.full((T, channels), 7.0, dtype=dt, device="cuda")
    index = idx if idx is not None else None
    want, new, mag = ref.conv(x, weight, cu, bias, True, state, index, resumed or [False] * len(lens), out)
    if width == 1:
        want, new, mag = ref.conv(x, weight, cu, bias, True, None, None, None, out)
        idx = None
    got = ms.conv_packed_fwd(x, weight, cu_t, bias=bias, state=state, state_indices=None if idx is None else i32(idx),
                             has_initial_state=flags if width > 1 else None, out=out)
    assert got is out
    close(got, want, conv_tol(mag, want, dt, width))
    if state is not None:
        assert torch.equal(state.to(F64), new)   # inputs are copied, not computed


@pytest.mark.parametrize("batch,channels,width,dtype,idx", [
    (1, 8, 4, "bf16", [0]), (5, 1333, 3, "f32", [6, 2, -1, 2, 99]), (300, 64, 4, "bf16", None), (2, 40, 1, "f32", None)])
def test_conv_packed_update(ms, batch, channels, width, dtype, idx):
    g, dt = rng(batch), DTYPES[dtype]
    x = normal(g, batch, channels, dtype=dt)
    weight = normal(g, channels, width)
    state = normal(g, max(batch, 7), width - 1, channels, dtype=dt)
    out = torch.full((batch, channels), -3.0, dtype=dt, device="cuda")
    cu = list(range(batch + 1))
    want, new, mag = ref.conv(x, weight, cu, None, False, state, idx, [True] * batch, out)
    got = ms.conv_packed_update(state, x, weight, silu=False, state_indices=None if idx is None else i32(idx), out=out)
    close(got, want, conv_tol(mag, want, dt, width))
    assert torch.equal(state.to(F64), new)


def test_conv_packed_stateless_and_unaligned(ms):
    """No state: every sequence starts from zero. A pointer that is aligned to its elements only."""
    g = rng(3)
    x = normal(g, 60 * 33 + 1, dtype=torch.bfloat16)[1:].view(60, 33)
    weight = normal(g, 33, 4)
    cu, cu_t = offsets([20, 40])
    want, _, mag = ref.conv(x, weight, cu, None, True, None, None, None, torch.zeros(60, 33, device="cuda"))
    close(ms.conv_packed_fwd(x, weight, cu_t), want, conv_tol(mag, want, torch.bfloat16, 4))


# ---- single tokens -----------------------------------------------------------------

def heads(g, n):
    return (-torch.rand(n, device="cuda", generator=g) * 15 - 1, normal(g, n), normal(g, n, scale=0.5) - 3.0)


@pytest.mark.parametrize("batch,H,G,P,N,dtype,idx,gate,softplus", [
    (1, 1, 1, 64, 128, "bf16", [0], False, True), (3, 4, 2, 64, 128, "bf16", [4, -1, 0], True, True),
    (5, 3, 1, 48, 96, "f32", [1, 5, 1, 9, 3], True, True), (2, 2, 1, 7, 16, "f32", None, False, False),
    (4, 6, 3, 32, 64, "bf16", None, True, True), (2, 3, 3, 130, 256, "bf16", [1, 0], False, True),
    (2, 2, 2, 5, 37, "f32", None, True, True), (3, 1, 1, 1, 1, "bf16", None, False, True),
    (2, 2, 1, 64, 20, "f32", [1, 0], True, False), (70, 2, 1, 16, 128, "bf16", None, False, True)])
def test_ssd_state_update(ms, batch, H, G, P, N, dtype, idx, gate, softplus):
    g, dt = rng(batch * H + N), DTYPES[dtype]
    A, D, bias = heads(g, H)
    wide = normal(g, batch, H * P + 2 * G * N, dtype=dt)
    x = wide[:, :H * P].unflatten(1, (H, P))
    B, C = wide[:, H * P:H * P + G * N].unflatten(1, (G, N)), wide[:, H * P + G * N:].unflatten(1, (G, N))
    step = normal(g, batch, H, dtype=dt, scale=0.5)
    z = normal(g, batch, H, P, dtype=dt) if gate else None
    state = normal(g, max(batch, 6), H, P, N)
    out = torch.full((batch, H, P), 5.0, dtype=dt, device="cuda")
    kw = dict(D=D, z=z, dt_bias=bias if softplus else None)
    want, new, ymag, smag = ref.ssd(x, step, A, B, C, list(range(batch + 1)), softplus=softplus, state=state, idx=idx,
                                    y=out, always=True, **kw)
    got = ms.ssd_state_update(state, x, step, A, B, C, dt_softplus=softplus,
                              state_indices=None if idx is None else i32(idx), out=out, **kw)
    close(state, new, 64 * U32 * smag)
    close(got, want, (64 + N) * U32 * ymag + 2 * ref.half(dt) * want.abs())


# ---- SSD over prompts ------------------------------------------------------------------

def ssd_inputs(g, T, H, G, gate):
    A, D, bias = heads(g, H)
    xbc = normal(g, T, H * 64 + 2 * G * 128, dtype=torch.bfloat16)
    pad = (H + 7) // 8 * 8
    proj = normal(g, T, H * 64 + pad, dtype=torch.bfloat16, scale=0.7)
    return dict(x=xbc[:, :H * 64].unflatten(1, (H, 64)), dt=proj[:, H * 64:H * 64 + H], A=A,
                B=xbc[:, H * 64:H * 64 + G * 128].unflatten(1, (G, 128)),
                C=xbc[:, H * 64 + G * 128:].unflatten(1, (G, 128))), \
        dict(D=D, dt_bias=bias, z=proj[:, :H * 64].unflatten(1, (H, 64)) if gate else None), (xbc, proj)


def ssd_close(y, state, want, new, ymag, smag):
    close(y, want, 1.1 * UB * (ymag + want.abs()))
    if state is not None:
        close(state, new, 2 * UB * UB * smag)


SSD = [
    # lens, heads, groups, gate, slots, indices, resumed, max_seqlen
    ([1], 1, 1, False, 2, [1], None, 0),
    ([5, 128, 129], 2, 1, True, 4, [3, 0, 1], [True, False, True], 129),
    ([0, 77, 0, 1, 256], 3, 1, False, 6, [5, 0, 2, 1, 3], [True, True, False, False, True], 0),
    ([300, 64], 6, 2, True, 2, None, [True, True], 300),
    ([130, 3], 5, 5, False, 2, None, None, 130),
    # skipped sequences between others
    ([40, 200, 40, 130], 2, 2, False, 3, [1, -1, 1, 7], [True] * 4, 200),
    # cut into segments: two, and more than two (the states pass through them)
    ([1500], 1, 1, False, 1, None, [True], 1500),
    ([2000, 0, 17, 1025], 2, 1, True, 4, [2, 0, 3, 1], [True, False, True, False], 2000),
    ([3000, 500, 100], 3, 3, False, 3, [1, 1, 0], [True, True, False], 3000),
    # more sequences than a warp has lanes
    ([(37 * i) % 150 for i in range(45)], 2, 1, False, 50, list(range(45)), [i % 3 == 0 for i in range(45)], 0),
]


@pytest.mark.parametrize("lens,H,G,gate,slots,idx,resumed,longest", SSD)
def test_ssd_packed(ms, lens, H, G, gate, slots, idx, resumed, longest):
    g = rng(sum(lens) + H)
    cu, cu_t = offsets(lens, first=3)
    T = cu[-1] + 130                    # rows of no sequence in front and behind, any bits in them
    a, kw, wide = ssd_inputs(g, T, H, G, gate)
    for w in wide:
        w[:3] = float("nan")
        w[cu[-1]:] = float("inf")
    state = normal(g, slots, H, 64, 128)
    out = torch.full((T, H, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    want, new, ymag, smag = ref.ssd(*a.values(), cu, state=state, idx=idx, init=resumed, y=out, **kw)
    got = ms.ssd_packed_fwd(*a.values(), cu_t, state=state, state_indices=None if idx is None else i32(idx),
                            has_initial_state=None if resumed is None else torch.tensor(resumed, device="cuda"),
                            max_seqlen=longest, out=out, **kw)
    ssd_close(got, state, want, new, ymag, smag)


def test_ssd_packed_rows_of_other_sequences(ms):
    """What a sequence's neighbours hold (infinities, NaN) does not reach it."""
    g = rng(8)
    cu, cu_t = offsets([70, 100, 60])
    a, kw, wide = ssd_inputs(g, 230, 2, 1, False)
    kw.pop("z")
    for w in wide:
        w[70:170] = float("nan")
    y = ms.ssd_packed_fwd(*a.values(), cu_t, **kw)
    want, _, ymag, _ = ref.ssd(*a.values(), cu, y=torch.zeros(230, 2, 64, device="cuda"), **kw)
    for s in (slice(0, 70), slice(170, 230)):
        close(y[s], want[s], 1.1 * UB * (ymag[s] + want[s].abs()))


@pytest.mark.parametrize("scale,A,softplus", [(40.0, -16.0, True), (0.0, 0.0, True), (0.02, -1.0, False),
                                              (-0.02, -1.0, False), (300.0, -50.0, True)])
def test_ssd_packed_steps(ms, scale, A, softplus):
    """Steps that wipe the state at once, no decay at all, raw and negative steps."""
    g = rng(11)
    lens = [400]
    cu, cu_t = offsets(lens)
    a, kw, _ = ssd_inputs(g, 400, 2, 1, False)
    a["A"] = torch.full((2,), A, device="cuda")
    if softplus:
        a["dt"] = normal(g, 400, 2, dtype=torch.bfloat16, scale=max(scale, 0.5))
    else:
        a["dt"] = torch.full((400, 2), scale, dtype=torch.bfloat16, device="cuda")
        kw["dt_bias"] = None
    state = normal(g, 1, 2, 64, 128)
    y = torch.zeros(400, 2, 64, dtype=torch.bfloat16, device="cuda")
    want, new, ymag, smag = ref.ssd(*a.values(), cu, softplus=softplus, state=state, init=[True], y=y, **kw)
    got = ms.ssd_packed_fwd(*a.values(), cu_t, dt_softplus=softplus, state=state, out=y,
                            has_initial_state=torch.ones(1, dtype=torch.uint8, device="cuda"), **kw)
    ssd_close(got, state, want, new, ymag, smag)


def test_ssd_packed_no_tokens(ms):
    """Only empty sequences: the resumed one keeps its state, the fresh one leaves zero."""
    g = rng(2)
    a, kw, _ = ssd_inputs(g, 0, 2, 1, False)
    state = normal(g, 3, 2, 64, 128)
    before = state.clone()
    y = ms.ssd_packed_fwd(*a.values(), i32([0, 0, 0]), state=state, state_indices=i32([2, 0]),
                          has_initial_state=torch.tensor([True, False], device="cuda"), **kw)
    assert y.shape == (0, 2, 64)
    assert torch.equal(state[1:], before[1:]) and not state[0].any()


def test_ssd_packed_longest_is_a_hint(ms):
    """A max_seqlen that is too small, exact or too large changes the schedule, not what is computed."""
    g = rng(41)
    cu, cu_t = offsets([2500, 40, 700])
    a, kw, _ = ssd_inputs(g, cu[-1], 2, 1, False)
    y = torch.zeros(cu[-1], 2, 64, dtype=torch.bfloat16, device="cuda")
    first = normal(g, 3, 2, 64, 128)
    want, new, ymag, smag = ref.ssd(*a.values(), cu, state=first, init=[True] * 3, y=y, **kw)
    for longest in (1, 300, 1000, 2500, 10 ** 6):
        state = first.clone()
        got = ms.ssd_packed_fwd(*a.values(), cu_t, state=state, max_seqlen=longest,
                                has_initial_state=torch.ones(3, dtype=torch.bool, device="cuda"), **kw)
        ssd_close(got, state, want, new, ymag, smag)


@pytest.mark.parametrize("lens", [[300, 77], [3000]])
def test_ssd_packed_in_place(ms, lens):
    """y in the place of x, and of z."""
    g = rng(43)
    _, cu = offsets(lens)
    for name in ("x", "z"):
        a, kw, _ = ssd_inputs(g, sum(lens), 2, 1, True)
        want = ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=max(lens), **kw)
        out = a["x"] if name == "x" else kw["z"]
        got = ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=max(lens), out=out, **kw)
        assert got is out and torch.equal(got, want)


@pytest.mark.parametrize("lens,H,must", [([2000, 300], 4, False), ([40000], 2, False), ([1100] * 8, 64, True)])
def test_ssd_packed_reports_a_wait_that_ran_out(ms, lens, H, must):
    """A limit of a microsecond: the call ends, says whether a wait ran out, and leaves nothing behind.
    The step warps run four chunks ahead and then wait for each chunk's products: 48 MMAs of 64 clocks for two
    heads, 1.6 us at 1965 MHz, less a step's own quarter of a microsecond. Where 256 pairs of heads share 148 SMs
    a CTA takes two heads and waits run out, though the device's timer may step too rarely to show it in every
    call; where the CTAs have room, a chunk of one head may take less than the limit."""
    g = rng(47)
    _, cu = offsets(lens)
    a, kw, _ = ssd_inputs(g, sum(lens), H, 1, False)
    want = ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=max(lens), **kw)
    ran_out = 0
    for _ in range(300 if must else 3):
        try:
            got = ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=max(lens), wait_limit_us=1, **kw)
            assert torch.equal(got, want)
        except ms.MambaScanError as e:
            assert e.status == 5                             # MS_ERR_TIMEOUT
            ran_out += 1
        if ran_out and must:
            break
    assert ran_out or not must
    assert torch.equal(ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=max(lens), **kw), want)


@pytest.mark.parametrize("lens,H", [([32768], 24), ([5000, 1, 0, 20000], 3), ([200, 150, 28], 24)])
def test_ssd_packed_many_calls_in_a_graph(ms, lens, H):
    """Calls one right behind the other, with one workspace: no wait runs out, every call gives the same."""
    g = rng(59)
    _, cu = offsets(lens)
    a, kw, _ = ssd_inputs(g, sum(lens), H, 1, False)
    state = torch.zeros(len(lens), H, 64, 128, device="cuda")
    out = torch.zeros(sum(lens), H, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")

    def call():
        ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=max(lens), state=state, out=out, workspace=ws, check=False, **kw)

    call()
    ms.ssd_check(ws)
    want = out.clone(), state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(20):
            call()
    for _ in range(20):
        out.fill_(float("nan"))
        state.fill_(float("nan"))
        graph.replay()
        ms.ssd_check(ws)
        assert torch.equal(out, want[0]) and torch.equal(state, want[1])


def test_cache_beyond_32_bits(ms):
    """Slots whose offset in the cache passes 2^31 elements (8 GB of states)."""
    g = rng(53)
    H, slots = 64, 4100                                      # 524288 values per slot
    state = torch.empty(slots, H, 64, 128, device="cuda")
    small = torch.zeros(2, H, 64, 128, device="cuda")
    at = [4099, 4097]
    a, kw, _ = ssd_inputs(g, 40, H, 1, False)
    kw.pop("z")
    _, cu = offsets([30, 10])
    want = ms.ssd_packed_fwd(*a.values(), cu, state=small, **kw)
    got = ms.ssd_packed_fwd(*a.values(), cu, state=state, state_indices=i32(at), **kw)
    assert torch.equal(got, want) and torch.equal(state[at], small)
    token = [t[:2] if t.dim() > 1 else t for t in a.values()]
    want = ms.ssd_state_update(small, *token, **kw)
    got = ms.ssd_state_update(state, *token, state_indices=i32(at), **kw)
    assert torch.equal(got, want) and torch.equal(state[at], small)


def test_ssd_packed_agrees_with_the_dense_forward(ms):
    """Equal lengths: the same layer through ssd_fwd, whose operands are rounded alike."""
    g = rng(21)
    a, kw, _ = ssd_inputs(g, 600, 4, 2, True)
    cu, cu_t = offsets([300, 300])
    state = torch.empty(2, 4, 64, 128, device="cuda")
    y = ms.ssd_packed_fwd(*a.values(), cu_t, state=state, **kw)
    dense = {k: v if k == "A" else v.reshape(2, 300, *v.shape[1:]) for k, v in a.items()}
    yd, hd = ms.ssd_fwd(*dense.values(), D=kw["D"], dt_bias=kw["dt_bias"], z=kw["z"].reshape(2, 300, 4, 64))
    want, new, ymag, smag = ref.ssd(*a.values(), cu, state=state, y=torch.zeros_like(y), **kw)
    ssd_close(y, state, want, new, ymag, smag)
    assert (yd.reshape(600, 4, 64).to(F64) - y.to(F64)).abs().max() <= 5e-3 * want.abs().max() * 2
    assert (hd - state).abs().max() <= 5e-3 * new.abs().max()


# ---- norms ---------------------------------------------------------------------------------

NORM = [
    # rows, dim, group, dtype, residual, gate, gate_first, weight
    (1, 1, 1, "f32", None, False, True, True), (3, 2048, 2048, "bf16", "f32", False, True, True),
    (130, 4096, 512, "bf16", None, True, True, True), (7, 4096, 4096, "bf16", None, True, False, True),
    (65, 1530, 1530, "f32", "f32", False, True, True), (40, 96, 12, "bf16", "bf16", True, True, True),
    (33, 777, 777, "bf16", None, False, True, False), (19, 200, 50, "f32", "f32", True, False, True),
    (9, 20000, 20000, "f32", None, True, True, True), (5, 40000, 40000, "bf16", "f32", True, True, True),
    (4, 5001, 5001, "bf16", "bf16", False, True, True), (1000, 64, 64, "bf16", None, True, False, False),
    (6, 16384, 16384, "bf16", None, False, True, True), (257, 8, 4, "f32", None, True, True, True),
]


def norm_inputs(rows, dim, dtype, residual, gate, weight):
    g, dt = rng(rows + dim), DTYPES[dtype]
    x = normal(g, rows, dim + 8, dtype=dt)[:, 8:]
    rd = None if residual is None else DTYPES[residual]
    return dict(x=x, z=normal(g, rows, dim, dtype=dt) if gate else None,
                residual=None if rd is None else normal(g, rows, dim, dtype=rd),
                weight=normal(g, dim) if weight else None), g


@pytest.mark.parametrize("rows,dim,group,dtype,residual,gate,first,weight", NORM)
def test_norm_fwd(ms, rows, dim, group, dtype, residual, gate, first, weight):
    a, _ = norm_inputs(rows, dim, dtype, residual, gate, weight)
    scale = 0.75 if residual else 1.0
    y, total = ms.norm_fwd(a["x"], weight=a["weight"], z=a["z"], residual=a["residual"], residual_scale=scale,
                           group_size=group, gate_first=first)
    d = {k: None if v is None else v.to(F64) for k, v in a.items()}
    want, v = ref.norm(d["x"], d["weight"], d["z"], d["residual"], scale, 1e-5, group, first)
    # what v is made of, and the size it reaches y with
    branch = d["x"].abs() * (ref.silu(d["z"]).abs() if gate and first else 1)
    mag = scale * branch + (0 if residual is None else d["residual"].abs())
    gain = torch.rsqrt(v.reshape(rows, -1, group).square().mean(-1, keepdim=True) + 1e-5).expand(-1, -1, group)
    gain = gain.reshape(rows, dim) * (1 if d["weight"] is None else d["weight"].abs())
    if gate and not first:
        gain = gain * ref.silu(d["z"]).abs()
    close(y, want, 64 * U32 * (want.abs() + mag * gain) + ref.half(y.dtype) * want.abs())
    if residual is None:
        assert total is None
    else:
        close(total, v, 16 * U32 * mag + ref.half(total.dtype) * v.abs())


@pytest.mark.parametrize("rows,dim,group,dtype,residual,gate,first,weight,later",
                         [(*c, later) for c in NORM for later in (False, True) if c[4] or not later])
def test_norm_bwd(ms, rows, dim, group, dtype, residual, gate, first, weight, later):
    a, g = norm_inputs(rows, dim, dtype, residual, gate, weight)
    scale = 0.75 if residual else 1.0
    dy = normal(g, rows, dim, dtype=a["x"].dtype)
    total = None if residual is None else normal(g, rows, dim, dtype=a["residual"].dtype)
    dtotal = normal(g, rows, dim, dtype=total.dtype) if later else None
    got = ms.norm_bwd(dy, a["x"], weight=a["weight"], z=a["z"], residual_out=total, dresidual_out=dtotal,
                      residual_scale=scale, group_size=group, gate_first=first)
    d = {k: None if v is None else v.to(F64).requires_grad_() for k, v in a.items()}
    y, v = ref.norm(d["x"], d["weight"], d["z"], d["residual"], scale, 1e-5, group, first,
                    None if total is None else total.to(F64))
    loss = (y * dy.to(F64)).sum() + (0 if dtotal is None else (v * dtotal.to(F64)).sum())
    names = [k for k in ("x", "z", "residual", "weight") if d[k] is not None]
    want = dict(zip(names, torch.autograd.grad(loss, [d[k] for k in names])))
    # sizes of what each gradient is made of
    with torch.no_grad():
        x, z, w = d["x"], d["z"], torch.ones(dim, dtype=F64, device="cuda") if d["weight"] is None else d["weight"].abs()
        gs = ref.silu(z).abs() if gate else torch.ones_like(x)
        slope = (torch.sigmoid(z) * (1 + z.abs() * (1 - torch.sigmoid(z)))) if gate else None
        r = torch.rsqrt(v.reshape(rows, -1, group).square().mean(-1, keepdim=True) + 1e-5)
        n = (v.reshape(rows, -1, group) * r).abs()
        e = dy.to(F64).abs() * (gs if gate and not first else 1)
        u = (e * w).reshape(rows, -1, group)
        dv = ((u + n * (u * n).mean(-1, keepdim=True)) * r).reshape(rows, dim)
        n = n.reshape(rows, dim)
        if dtotal is not None:
            dv = dv + dtotal.to(F64).abs()
        size = {"residual": dv, "x": scale * dv * (gs if gate and first else 1), "weight": (e * n).sum(0)}
        if gate:
            size["z"] = scale * dv * x.abs() * slope if first else dy.to(F64).abs() * n * w * slope
    key = {"x": "dx", "z": "dz", "residual": "dresidual", "weight": "dweight"}
    for k in names:
        t = got[key[k]]
        count = 128 + (rows if k == "weight" else 0)   # (dweight: a sum over the rows)
        close(t, want[k], count * U32 * size[k] + ref.half(t.dtype) * want[k].abs())
    for k in set(key) - set(names):
        assert got[key[k]] is None


@pytest.mark.parametrize("rows,dim,group,dtype,residual,gate,first", [
    (9001, 512, 512, "bf16", None, True, True), (2500, 1530, 1530, "f32", "f32", False, True),
    (750, 16384, 16384, "bf16", None, True, False), (1999, 2048, 2048, "bf16", "f32", False, True),
    (20011, 48, 16, "bf16", "bf16", False, True), (1200, 4096, 4096, "f32", None, False, True),
    # every number of vectors per thread, for warps and blocks, with the most bytes per row on their way
    (64, 2048, 2048, "f32", "f32", False, True), (300, 1024, 512, "f32", "f32", False, True),
    (300, 512, 256, "f32", "f32", False, True), (70, 8192, 8192, "f32", "f32", False, True),
    (70, 16384, 16384, "f32", None, True, True), (90, 4096, 4096, "bf16", "f32", False, True),
    (90, 8192, 8192, "bf16", "f32", False, True), (90, 8192, 8192, "bf16", None, True, True),
    (90, 2048, 1024, "bf16", "bf16", False, True), (200, 640, 128, "bf16", "f32", False, True),
    (200, 66, 66, "f32", "f32", False, True), (100, 3330, 3330, "f32", None, True, False),
])
def test_norm_bwd_many_rows(ms, rows, dim, group, dtype, residual, gate, first):
    """More rows than a team of threads has on their way together."""
    test_norm_bwd(ms, rows, dim, group, dtype, residual, gate, first, True, residual is not None)


def test_norm_bwd_against_differences(ms):
    """The gradients of x, z and weight against central differences of the forward in 64 bits."""
    g = rng(77)
    x, z, w, dy = (normal(g, 3, 24) for _ in range(4))
    w = w[0].contiguous()
    got = ms.norm_bwd(dy, x, weight=w, z=z, group_size=8)

    def loss(x, z, w):
        return (ref.norm(x, w, z, group=8)[0] * dy.to(F64)).sum()

    args, h = [x.to(F64), z.to(F64), w.to(F64)], 1e-5
    for i, name in enumerate(("dx", "dz", "dweight")):
        for j in range(0, args[i].numel(), 5):
            up, down = ([a.clone() for a in args] for _ in range(2))
            up[i].view(-1)[j] += h
            down[i].view(-1)[j] -= h
            diff = ((loss(*up) - loss(*down)) / (2 * h)).item()
            # the difference's own error is about h^2 times a third derivative
            assert abs(got[name].view(-1)[j].item() - diff) <= 1e-4 * (1 + abs(diff))


@pytest.mark.parametrize("rows,dim,group", [(40, 64, 16), (9, 2048, 2048), (3, 40000, 40000)])
def test_norm_in_place(ms, rows, dim, group):
    """y in the place of x or z, the sum in the residual's."""
    g = rng(dim)
    x, z, w = normal(g, rows, dim), normal(g, rows, dim), normal(g, dim)
    res = normal(g, rows, dim)
    kw = dict(weight=w, group_size=group)
    want, sums = ms.norm_fwd(x, z=z, residual=res, **kw)
    for name in ("x", "z"):
        c = dict(x=x.clone(), z=z.clone(), residual=res.clone())
        y, ro = ms.norm_fwd(**c, **kw, out=c[name], residual_out=c["residual"])
        assert y is c[name] and ro is c["residual"]
        assert torch.equal(y, want) and torch.equal(ro, sums)


def test_norm_rows_none(ms):
    x = torch.empty(0, 64, device="cuda")
    y, total = ms.norm_fwd(x, residual=x)
    assert y.shape == total.shape == (0, 64)
    g = ms.norm_bwd(x, x, weight=torch.ones(64, device="cuda"))
    assert not g["dweight"].any() and g["dx"].shape == (0, 64)


def test_norm_bwd_sums_in_a_fixed_order(ms):
    g = rng(5)
    x, dy, w = normal(g, 3000, 1024, dtype=torch.bfloat16), normal(g, 3000, 1024, dtype=torch.bfloat16), normal(g, 1024)
    first = ms.norm_bwd(dy, x, weight=w)["dweight"]
    for _ in range(3):
        assert torch.equal(ms.norm_bwd(dy, x, weight=w)["dweight"], first)


# ---- together --------------------------------------------------------------------------------

def layer(ms, c, x, states, mode, cu=None, idx=None, init=None):
    """The inner part of a Mamba-2 layer, as a serving program runs it: the norm
    before the block, a projection, convolution, SSD and the gated norm."""
    h, stream = ms.norm_fwd(x, weight=c["w_in"], residual=c["stream"][:len(x)])
    proj = (h.float() @ c["proj"]).to(torch.bfloat16)
    H, di = c["H"], c["H"] * 64
    z, xbc, dt = proj[:, :di], proj[:, di:2 * di + 256], proj[:, 2 * di + 256:2 * di + 256 + H]
    conv_state, ssm_state = states
    if mode == "tokens":
        xbc = ms.conv_packed_update(conv_state, xbc, c["filter"], bias=c["conv_bias"], state_indices=idx)
    else:
        xbc = ms.conv_packed_fwd(xbc, c["filter"], cu, bias=c["conv_bias"], state=conv_state, state_indices=idx,
                                 has_initial_state=init)
    xs, B, C = (xbc[:, :di].unflatten(1, (H, 64)), xbc[:, di:di + 128].unflatten(1, (1, 128)),
                xbc[:, di + 128:].unflatten(1, (1, 128)))
    if mode == "tokens":
        y = ms.ssd_state_update(ssm_state, xs, dt, c["A"], B, C, D=c["D"], dt_bias=c["bias"], state_indices=idx)
    else:
        y = ms.ssd_packed_fwd(xs, dt, c["A"], B, C, cu, D=c["D"], dt_bias=c["bias"], state=ssm_state,
                              state_indices=idx, has_initial_state=init)
    return ms.norm_fwd(y.reshape(len(x), di), weight=c["w_out"], z=z, group_size=di // 2)[0], stream


def layer_params(H=4, d=96, T=400):
    g = rng(99)
    A, D, bias = heads(g, H)
    di = H * 64
    width = 2 * di + 256 + 8
    return dict(H=H, A=A, D=D, bias=bias, w_in=normal(g, d), w_out=normal(g, di), proj=normal(g, d, width, scale=d ** -0.5),
                filter=normal(g, di + 256, 4, scale=0.5), conv_bias=normal(g, di + 256),
                stream=normal(g, T, d)), g


def new_states(c, slots):
    ch = c["H"] * 64 + 256
    return (torch.zeros(slots, 3, ch, dtype=torch.bfloat16, device="cuda"),
            torch.zeros(slots, c["H"], 64, 128, device="cuda"))


def test_layer_prompts_then_tokens(ms):
    """Prompts in two chunks and then single tokens give what the whole prompts give at once."""
    c, g = layer_params()
    c["stream"].zero_()
    lens = [150, 7, 133]
    parts = [(100, 30, 20), (3, 3, 1), (129, 2, 2)]          # chunk, chunk, tokens one by one
    xs = [normal(g, n, 96, dtype=torch.bfloat16) for n in lens]
    whole_states = new_states(c, 5)
    idx = i32([4, 0, 2])
    cu, cu_t = offsets(lens)
    whole, _ = layer(ms, c, torch.cat(xs), whole_states, "prompt", cu_t, idx)
    states = new_states(c, 5)
    states[1].normal_()                                      # (what was there before a fresh start does not matter)
    states[0].fill_(1.0)
    got = [[] for _ in lens]
    at = [0, 0, 0]
    for k in (0, 1):
        _, cu_p = offsets([p[k] for p in parts])
        rows = torch.cat([x[a:a + p[k]] for x, a, p in zip(xs, at, parts)])
        out, _ = layer(ms, c, rows, states, "prompt", cu_p, idx, torch.full((3,), k == 1, device="cuda"))
        o = 0
        for s, p in enumerate(parts):
            got[s].append(out[o:o + p[k]])
            o += p[k]
            at[s] += p[k]
    for t in range(20):
        # requests that are done leave an empty place in the batch
        live = [t < p[2] for p in parts]
        rows = torch.stack([x[min(a, len(x) - 1)] for x, a in zip(xs, at)])
        out, _ = layer(ms, c, rows, states, "tokens", idx=torch.where(torch.tensor(live, device="cuda"), idx, -1))
        for s in range(3):
            if live[s]:
                got[s].append(out[s:s + 1])
                at[s] += 1
    got = torch.cat([torch.cat(v) for v in got]).to(F64)
    whole = whole.to(F64)
    assert torch.isfinite(got).all()
    # the convolution is the same; the SSD's two roundings (M', state) and its own fall differently, and
    # the norm scales them with what it norms: a few u(bf16) of the row's size
    size = whole.abs().reshape(len(whole), 2, -1).amax(-1, keepdim=True).expand(-1, -1, 128).reshape(whole.shape)
    assert ((got - whole).abs() <= 6 * UB * size).all()
    assert (states[1][[4, 0, 2]] - whole_states[1][[4, 0, 2]]).abs().max() <= 1e-4 * whole_states[1].abs().max()
    assert torch.equal(states[0][[4, 0, 2]], whole_states[0][[4, 0, 2]])


def test_captured_step_on_another_stream(ms):
    """A decode step and a prompt step captured into graphs on a side stream, replayed with new inputs."""
    c, g = layer_params()
    idx = i32([1, 0, 3])
    x = normal(g, 3, 96, dtype=torch.bfloat16)
    p = normal(g, 300, 96, dtype=torch.bfloat16)
    _, cu = offsets([200, 0, 100])
    H, di = c["H"], c["H"] * 64

    def ssd(rows, states, workspace=None):
        xbc = (rows.float() @ c["proj"][:, :di + 256]).to(torch.bfloat16)
        xbc = ms.conv_packed_fwd(xbc, c["filter"], cu, state=states[0], state_indices=idx)
        return ms.ssd_packed_fwd(xbc[:, :di].unflatten(1, (H, 64)), xbc[:, :H], c["A"],
                                 xbc[:, di:di + 128].unflatten(1, (1, 128)),
                                 xbc[:, di + 128:].unflatten(1, (1, 128)), cu, dt_bias=c["bias"], state=states[1],
                                 state_indices=idx, workspace=workspace, check=False)

    def token(rows, states):
        return layer(ms, c, rows, states, "tokens", idx=idx)[0]

    runs = {}
    for name, fn, rows in (("prompt", ssd, p), ("token", token, x)):
        states = new_states(c, 4)
        fn(rows, states)                                     # warm-up outside the capture
        for s in states:
            s.zero_()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            out = fn(rows, states)
        runs[name] = (graph, out, states, fn, rows)
    fresh = {"prompt": normal(g, 300, 96, dtype=torch.bfloat16), "token": normal(g, 3, 96, dtype=torch.bfloat16)}
    for name, (graph, out, states, fn, rows) in runs.items():
        for s in states:
            s.zero_()
        rows.copy_(fresh[name])
        graph.replay()
        torch.cuda.synchronize()
        again = new_states(c, 4)
        want = fn(fresh[name], again)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(torch.equal(a, b) for a, b in zip(states, again))


def test_two_streams_at_once(ms):
    """Two prompt calls on two streams, each with scratch of its own, against the same calls one by one."""
    g = rng(31)
    work = []
    for s in range(2):
        a, kw, _ = ssd_inputs(g, 4000, 2, 1, False)
        work.append((a, kw, i32([0, 4000])))
    alone = [ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=4000, **kw) for a, kw, cu in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(5):
        outs = []
        for st, (a, kw, cu) in zip(streams, work):
            outs.append(ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=4000, stream=st, check=False, **kw))
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, alone))


# ---- refusals ------------------------------------------------------------------------------------

def test_python_refusals(ms):
    f = lambda *s, **k: torch.zeros(*s, device="cuda", **k)   # noqa: E731
    bf = torch.bfloat16
    x, w, cu = f(8, 16), f(16, 4), i32([0, 8])
    with pytest.raises(TypeError):
        ms.conv_packed_fwd(f(8, 16, dtype=torch.float16), w, cu)
    with pytest.raises(TypeError):
        ms.conv_packed_fwd(x, w, cu.long())
    with pytest.raises(ValueError):
        ms.conv_packed_fwd(x, f(15, 4), cu)
    with pytest.raises(ValueError):
        ms.conv_packed_fwd(x, w, cu, state=f(2, 4, 16))
    with pytest.raises(TypeError):
        ms.conv_packed_fwd(x, w, cu, state=f(2, 3, 16, dtype=bf))
    with pytest.raises(ValueError):
        ms.conv_packed_fwd(x, w, cu, state=f(2, 3, 16), state_indices=i32([0, 1]))
    with pytest.raises(ValueError):
        ms.conv_packed_fwd(x, w, cu, out=f(8, 17))
    with pytest.raises(ValueError):
        ms.conv_packed_fwd(x.t().contiguous().t(), w, cu)
    with pytest.raises(ms.MambaScanError) as e:
        ms.conv_packed_fwd(x, f(16, 5), cu)
    assert e.value.status == 2
    with pytest.raises(ms.MambaScanError) as e:
        ms.conv_packed_update(f(7, 3, 16), x, w)              # fewer slots than rows and no index table
    assert e.value.status == 1
    with pytest.raises(ms.MambaScanError):
        ms.conv_packed_fwd(x, w, cu, state_indices=i32([0]))  # an index table without a state
    a, kw, _ = ssd_inputs(rng(1), 16, 2, 1, False)
    cu = i32([0, 16])
    with pytest.raises(ValueError):
        ms.ssd_packed_fwd(*{**a, "B": a["B"][:, :, :64]}.values(), cu, **kw)
    with pytest.raises(TypeError):
        ms.ssd_packed_fwd(*{**a, "dt": a["dt"].float()}.values(), cu, **kw)
    with pytest.raises(ms.MambaScanError) as e:
        ms.ssd_packed_fwd(*{k: v.float() if k != "A" else v for k, v in a.items()}.values(), cu, **kw)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        ms.ssd_packed_fwd(*a.values(), cu, state=f(1, 2, 64, 64), **kw)
    with pytest.raises(ValueError):
        ms.ssd_packed_fwd(*a.values(), cu, workspace=f(8), **kw)
    with pytest.raises(ms.MambaScanError) as e:
        ms.ssd_packed_fwd(*{**a, "x": f(17, 2 * 64 + 4, dtype=bf)[:16, :128].unflatten(1, (2, 64))}.values(), cu, **kw)
    assert e.value.status == 3
    with pytest.raises(TypeError):
        ms.norm_fwd(f(4, 8), residual=f(4, 8, dtype=bf))
    with pytest.raises(ValueError):
        ms.norm_fwd(f(4, 8), residual_out=f(4, 8))
    for kind, bad in ((TypeError, dict(z=f(4, 8, dtype=bf))), (ValueError, dict(z=f(4, 9))), (ValueError, dict(weight=f(9))),
                      (TypeError, dict(weight=f(8, dtype=bf))), (ValueError, dict(out=torch.zeros(4, 8))),
                      (ValueError, dict(z=f(8, 4).t())), (TypeError, dict(eps="x")), (TypeError, dict(z=3)), (TypeError, dict(group_size=2.5)),
                      (ValueError, dict(weight=f(16)[::2]))):
        with pytest.raises(kind):
            ms.norm_fwd(f(4, 8), **bad)
    with pytest.raises(ValueError):
        ms.norm_fwd(f(8))
    with pytest.raises(TypeError):
        ms.norm_fwd(f(4, 8, dtype=torch.float16))
    with pytest.raises(ValueError):
        ms.norm_bwd(f(4, 8), f(4, 8), weight=f(8), workspace=f(100))
    with pytest.raises(ValueError):
        ms.norm_bwd(f(4, 9), f(4, 8))
    with pytest.raises(ms.MambaScanError):
        ms.norm_fwd(f(4, 8), group_size=3)
    with pytest.raises(ValueError):
        ms.norm_bwd(f(4, 8), f(4, 8), dresidual_out=f(4, 8))
    with pytest.raises(ValueError):
        ms.ssd_state_update(f(2, 1, 4, 8), f(2, 1, 4), f(2, 1), f(2), f(2, 1, 8), f(2, 1, 8))
