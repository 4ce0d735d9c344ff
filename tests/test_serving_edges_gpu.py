"""GPU tests of calls of the serving operators and norms at their edges: NaN in the
decay, the schedules that large batches take, other streams, workspaces. Tolerances
as in test_serving_gpu.py."""
import pytest
import torch

from tests import serving_ref as ref
from tests.test_serving_gpu import (F64, UB, close, conv_tol, i32, normal, offsets, rng, ssd_close, ssd_inputs,
                                     test_ssd_packed as _test_ssd_packed)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ms():
    import selective_state_space_27_b200 as m
    return m


# ---- the schedules of large batches ---------------------------------------------------

SCHEDULES = [
    # (chunks per segment, heads per CTA) on 148 SMs: test_schedules_of_these_sizes holds them to it
    # lens, heads, groups, gate, slots, indices, resumed, longest, schedule
    # two heads per CTA, whole sequences: ragged ends, empty ones, resumed and skipped ones
    ([300, 77, 128, 5, 0, 200], 64, 1, True, 7, [6, 0, 3, -1, 1, 5], [True, False, True, True, True, False], 300, (0, 2)),
    ([257, 1, 256, 129], 80, 2, False, 4, None, [False, True, True, False], 257, (0, 2)),
    # an odd number of heads in a group: its last pair is one head
    ([200, 130, 40, 1, 0, 90, 60], 45, 3, True, 9, [8, 1, 1, 3, 4, 9, 0], [True] * 7, 200, (0, 2)),
    # more than 32 whole sequences, two heads per CTA (the last pair of nine is one head), and one
    ([40 - i % 9 for i in range(40)], 9, 1, False, 41, list(range(40, 0, -1)), [i % 2 == 0 for i in range(40)], 40, (0, 2)),
    ([(37 * i) % 150 for i in range(45)], 2, 1, True, 50, [i if i % 7 else -1 for i in range(45)],
     [i % 3 == 0 for i in range(45)], 148, (0, 1)),
    # two heads per CTA in segments of two, three, four and six chunks
    ([3000], 24, 1, False, 1, None, [True], 3000, (2, 2)),
    ([1500], 64, 2, True, 2, [1], [False], 1500, (4, 2)),
    ([4000], 48, 1, False, 1, [0], [True], 4000, (6, 2)),
    ([2500, 0, 300], 45, 3, True, 3, [2, 0, 1], [True, True, False], 2500, (3, 2)),
    # one head per CTA in segments of three chunks
    ([9000], 5, 1, False, 1, None, [True], 9000, (3, 1)),
]


@pytest.mark.parametrize("lens,H,G,gate,slots,idx,resumed,longest,schedule", SCHEDULES)
def test_ssd_packed_schedules(ms, lens, H, G, gate, slots, idx, resumed, longest, schedule):
    """The forms that large batches take, against the definition, rows of no sequence and skipped slots among them."""
    _test_ssd_packed(ms, lens, H, G, gate, slots, idx, resumed, longest)


# ---- NaN in the decay --------------------------------------------------------------

# one head per CTA; two; one sequence in segments (of two chunks)
NAN_SIZES = [([300, 20], 4, 0), ([130, 40, 70, 20, 1], 64, 130), ([1500], 4, 1500)]


@pytest.mark.parametrize("lens,H,longest", NAN_SIZES)
@pytest.mark.parametrize("how", ["rate", "infinite_rate_without_step"])
def test_nan_decay_reaches_outputs_and_states(ms, lens, H, longest, how):
    """A head whose decay exp(delta A) is NaN (A NaN, or -inf times a step of 0) gives NaN, as its definition and the
    single-token call do; the other heads are what they are without it."""
    g = rng(5)
    cu, cu_t = offsets(lens)
    a, kw, _ = ssd_inputs(g, cu[-1], H, 1, False)
    if how != "rate":
        kw["dt_bias"] = None
        a["dt"] = a["dt"].abs()
        a["dt"][:, 1] = 0.0
    first = normal(g, len(lens), H, 64, 128)
    flags = torch.ones(len(lens), dtype=torch.bool, device="cuda")

    def call(A):
        state = first.clone()
        y = ms.ssd_packed_fwd(a["x"], a["dt"], A, a["B"], a["C"], cu_t, state=state, has_initial_state=flags,
                              max_seqlen=longest, dt_softplus=how == "rate", **kw)
        return y, state

    bad = a["A"].clone()
    bad[1] = float("nan") if how == "rate" else -float("inf")
    (y, state), (y0, state0) = call(bad), call(a["A"])
    assert torch.isfinite(y0).all() and torch.isfinite(state0).all()
    assert torch.isnan(y[:, 1]).all() and torch.isnan(state[:, 1]).all()
    others = [h for h in range(H) if h != 1]
    assert torch.equal(y[:, others], y0[:, others]) and torch.equal(state[:, others], state0[:, others])
    token = first.clone()
    n = len(lens)
    yt = ms.ssd_state_update(token, a["x"][:n], a["dt"][:n], bad, a["B"][:n], a["C"][:n], dt_softplus=how == "rate", **kw)
    assert torch.isnan(yt[:, 1]).all() and torch.isnan(token[:, 1]).all()


@pytest.mark.parametrize("lens,H,longest", NAN_SIZES)
@pytest.mark.parametrize("at", [0, 17, 127])
def test_nan_step_reaches_what_follows(ms, lens, H, longest, at):
    """A step that is NaN: the rows in front of it are what they are, its own and the later ones NaN."""
    g = rng(6)
    cu, cu_t = offsets(lens)
    a, kw, _ = ssd_inputs(g, cu[-1], H, 1, False)
    a["dt"][at, 1] = float("nan")
    state = torch.zeros(len(lens), H, 64, 128, device="cuda")
    out = torch.zeros(cu[-1], H, 64, dtype=torch.bfloat16, device="cuda")
    want, new, ymag, smag = ref.ssd(*a.values(), cu, state=state, y=out, **kw)
    y = ms.ssd_packed_fwd(*a.values(), cu_t, state=state, max_seqlen=longest, **kw)
    hit = torch.isnan(want)
    assert hit[at:cu[1], 1].all() and hit.sum() == (cu[1] - at) * 64
    assert torch.equal(torch.isnan(y), hit) and torch.equal(torch.isnan(state), torch.isnan(new))
    ssd_close(y[~hit], None, want[~hit], None, ymag[~hit], None)
    clean = ~torch.isnan(new)
    close(state[clean], new[clean], 2 * UB * UB * smag[clean])


# ---- other streams --------------------------------------------------------------------

def on_stream_calls(ms, g):
    """name -> (call of a stream, shapes and types of what it allocates)."""
    bf = torch.bfloat16
    x, z, w = normal(g, 3000, 512, dtype=bf), normal(g, 3000, 512, dtype=bf), normal(g, 512)
    res = normal(g, 3000, 512)
    filt, conv_state = normal(g, 512, 4), normal(g, 3000, 3, 512, dtype=bf)
    a, kw, _ = ssd_inputs(g, 3000, 2, 1, False)
    token = dict(zip(a, [t[:700] if t.dim() > 1 else t for t in a.values()]))
    state = torch.zeros(700, 2, 64, 128, device="cuda")
    cu = i32([0, 3000])
    rows = ((3000, 512), bf)
    kept = []

    def fresh(cache):
        kept.append(cache.clone())   # (of the current stream: kept, and there before another stream uses it)
        torch.cuda.synchronize()
        return kept[-1]

    return {
        "norm_fwd": (lambda s: ms.norm_fwd(x, weight=w, residual=res, stream=s), [rows, ((3000, 512), torch.float32)]),
        "norm_bwd": (lambda s: ms.norm_bwd(x, x, weight=w, z=z, stream=s), [rows, rows, ((512,), torch.float32)]),
        "conv_packed_fwd": (lambda s: ms.conv_packed_fwd(x, filt, cu, stream=s), [rows]),
        "conv_packed_update": (lambda s: ms.conv_packed_update(fresh(conv_state), x, filt, stream=s), [rows]),
        "ssd_packed_fwd": (lambda s: ms.ssd_packed_fwd(*a.values(), cu, stream=s, check=False, **kw),
                           [((3000, 2, 64), bf), ((1 << 21,), torch.uint8)]),
        "ssd_state_update": (lambda s: ms.ssd_state_update(fresh(state), *token.values(), stream=s, **kw),
                             [((700, 2, 64), bf)]),
    }


def tensors(result):
    return [t for t in (result.values() if isinstance(result, dict) else result if isinstance(result, tuple) else [result])
            if t is not None]


@pytest.mark.parametrize("name", ["norm_fwd", "norm_bwd", "conv_packed_fwd", "conv_packed_update", "ssd_packed_fwd",
                                  "ssd_state_update"])
def test_given_stream_owns_what_the_call_allocates(ms, name):
    """With ``stream`` the outputs are not memory that the current stream has just given back (its work may still use
    it), and memory of dropped outputs does not go to the current stream while the call still writes it."""
    call, shapes = on_stream_calls(ms, rng(3))[name]
    want = [t.clone() for t in tensors(call(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty(s, dtype=t, device="cuda") for s, t in shapes for _ in range(3)]
    freed = [(b.data_ptr(), b.data_ptr() + b.numel() * b.element_size()) for b in blocks]
    del blocks
    got = tensors(call(side))
    assert len(got) == len(want)
    assert not any(lo <= t.data_ptr() < hi for t in got for lo, hi in freed)
    side.synchronize()
    assert all(torch.equal(t, w) for t, w in zip(got, want))
    for _ in range(5):
        places = [t.data_ptr() for t in tensors(call(side))]      # dropped at once
        mine = [torch.full_like(w, 3.0) for w in want]
        assert not set(places) & {t.data_ptr() for t in mine}
        torch.cuda.synchronize()
        assert all((t == 3.0).all() for t in mine)


def test_given_stream_beside_unchecked_calls_of_the_current_one(ms):
    """A call in segments whose workspace is dropped while it runs, and one of the same size on another stream right
    behind it: each keeps to its own workspace."""
    g = rng(12)
    work = [ssd_inputs(g, 16384, 4, 1, False)[:2] for _ in range(2)]
    cu = i32([0, 16384])

    def call(k, stream=None, check=False):
        a, kw = work[k]
        state = torch.zeros(1, 4, 64, 128, device="cuda")
        y = ms.ssd_packed_fwd(*a.values(), cu, state=state, max_seqlen=16384, stream=stream, check=check, **kw)
        return y, state

    want = [call(k, check=True) for k in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    states = torch.zeros(2, 1, 4, 64, 128, device="cuda")
    for _ in range(10):
        states.zero_()
        torch.cuda.synchronize()
        out = []
        for k, stream in ((0, None), (1, side)):
            a, kw = work[k]
            out.append(ms.ssd_packed_fwd(*a.values(), cu, state=states[k], max_seqlen=16384, stream=stream, check=False,
                                         **kw))
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(out[k], want[k][0]) and torch.equal(states[k], want[k][1])


def test_stream_of_the_inputs_device(ms):
    """``stream`` positional, as keyword, in a capture; with host tensors the tensor is refused."""
    g = rng(4)
    x, w = normal(g, 40, 64), normal(g, 64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = ms.norm_fwd(x, weight=w)[0]
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        y, _ = ms.norm_fwd(x, weight=w, stream=side)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    with pytest.raises(ValueError, match="CUDA"):
        ms.norm_fwd(x.cpu(), stream=side)
    with pytest.raises(ValueError, match="CUDA"):
        ms.conv_packed_update(x.cpu(), x.cpu(), w, stream=side)


# ---- workspaces ------------------------------------------------------------------------

def test_small_workspace_is_refused_where_its_status_is_read_later(ms):
    """With check=False the caller reads the status from the workspace it gave: one that is too small is refused, not
    replaced. With check=True the call reads the status itself."""
    g = rng(14)
    a, kw, _ = ssd_inputs(g, 6000, 2, 1, False)
    cu = i32([0, 6000])
    want = ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=6000, **kw)
    small = torch.full((256,), 0xAB, dtype=torch.uint8, device="cuda")
    out = torch.full_like(want, 5.0)
    for ws in (small, small[:0]):
        with pytest.raises(ms.MambaScanError) as e:
            ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=6000, out=out, workspace=ws, check=False, **kw)
        assert e.value.status == 6                               # MS_ERR_WORKSPACE
    assert (out == 5.0).all() and (small == 0xAB).all()
    assert torch.equal(ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=6000, workspace=small, **kw), want)
    large = torch.full((1 << 24,), 0xAB, dtype=torch.uint8, device="cuda")
    ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=6000, out=out, workspace=large, check=False, **kw)
    ms.ssd_check(large)
    assert torch.equal(out, want)


def test_failed_wait_of_an_unchecked_call_leaves_a_trace(ms):
    """check=False without a workspace: the status word goes with the scratch, the count of failures stays. (A limit of
    a microsecond on chunks of two heads, as in the timeout test of test_serving_gpu.py.)"""
    g = rng(47)
    a, kw, _ = ssd_inputs(g, 8 * 1100, 64, 1, False)
    cu = offsets([1100] * 8)[1]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    try:
        ms.ssd_check()                   # what earlier calls left
    except ms.MambaScanError:
        pass
    want = ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=1100, **kw)
    ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=1100, check=False, **kw)
    ms.ssd_check()
    for k in range(300):
        ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=1100, check=False, wait_limit_us=1, stream=side, **kw)
        try:
            ms.ssd_check(stream=side)
        except ms.MambaScanError as e:
            assert e.status == 5         # MS_ERR_TIMEOUT
            break
    else:
        assert False, "no wait ran out"
    assert torch.equal(ms.ssd_packed_fwd(*a.values(), cu, max_seqlen=1100, **kw), want)
    ms.ssd_check()


def test_norm_bwd_calls_in_a_row_with_one_workspace(ms):
    """The sum over the slabs starts beside the kernel that writes their shares, here over the shares of the call in
    front: every call gets its own."""
    g = rng(15)
    w = normal(g, 1530)
    calls = [(normal(g, 1500 + 40 * i, 1530), normal(g, 1500 + 40 * i, 1530)) for i in range(6)]
    alone = [ms.norm_bwd(dy, x, weight=w)["dweight"].clone() for x, dy in calls]
    ws = torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda")     # (NaN)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [ms.norm_bwd(dy, x, weight=w, workspace=ws)["dweight"] for x, dy in calls]
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, alone))


# ---- the convolution's largest channel counts ----------------------------------------------

@pytest.mark.parametrize("channels", [65535 * 64, 65535 * 64 + 1, (1 << 22) - 1, 1 << 22])
def test_conv_packed_most_channels(ms, channels):
    """One channel per thread where the count is no multiple of four: more blocks of channels than a grid has in y."""
    g = rng(16)
    x, weight, bias = normal(g, 2, channels), normal(g, channels, 2), normal(g, channels)
    state = normal(g, 1, 1, channels)
    cu, cu_t = offsets([2])
    want, new, mag = ref.conv(x, weight, cu, bias, True, state, None, [True], torch.zeros_like(x))
    got = ms.conv_packed_fwd(x, weight, cu_t, bias=bias, state=state, has_initial_state=torch.tensor([True], device="cuda"))
    close(got, want, conv_tol(mag, want, torch.float32, 2))
    assert torch.equal(state.to(F64), new)


@pytest.mark.parametrize("where", ["columns", "columns_and_steps", "rows", "one_row"])
def test_conv_packed_beside_its_input(ms, where):
    """x and y in one buffer without a shared element: columns of the same rows, rows in turn, one behind the other."""
    g = rng(17)
    buf = normal(g, 120, 100)
    x, out = {"columns": (buf[:60, :40], buf[:60, 40:80]), "columns_and_steps": (buf[::2, :40], buf[:60, 60:]),
              "rows": (buf[::2, :40], buf[1::2, :40]), "one_row": (buf[:1, :40], buf[:1, 40:80])}[where]
    weight = normal(g, 40, 4)
    cu, cu_t = offsets([len(x)])
    want, _, mag = ref.conv(x, weight, cu, None, True, None, None, None, torch.zeros(len(x), 40, device="cuda"))
    close(ms.conv_packed_fwd(x, weight, cu_t, out=out), want, conv_tol(mag, want, torch.float32, 4))
    with pytest.raises(ms.MambaScanError, match="overlap"):
        ms.conv_packed_fwd(x, weight, cu_t, out=buf[:len(x), 30:70])


@pytest.mark.parametrize("P,N,dtype", [(64, 128, torch.bfloat16), (7, 37, torch.float32), (48, 16, torch.float32)])
def test_ssd_state_update_in_place(ms, P, N, dtype):
    """y in the place of x, and of z."""
    g = rng(P)
    x, z = normal(g, 5, 2, P, dtype=dtype), normal(g, 5, 2, P, dtype=dtype)
    B, C, dt = normal(g, 5, 1, N, dtype=dtype), normal(g, 5, 1, N, dtype=dtype), normal(g, 5, 2, dtype=dtype)
    A, state = -torch.rand(2, device="cuda", generator=g), normal(g, 5, 2, P, N)
    want = ms.ssd_state_update(state.clone(), x, dt, A, B, C, z=z)
    for name in ("x", "z"):
        c = dict(x=x.clone(), z=z.clone())
        got = ms.ssd_state_update(state.clone(), c["x"], dt, A, B, C, z=c["z"], out=c[name])
        assert got is c[name] and torch.equal(got, want)
