"""GPU tests of calls of the serving operators and norms at their edges: NaN in the
decay, the schedules that large batches take, other streams, workspaces. Tolerances
as in test_serving_gpu.py."""
import pytest
import torch

from tests import serving_ref as ref
from tests.test_serving_gpu import F64, UB, close, i32, normal, offsets, rng, ssd_close, ssd_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ms():
    import selective_state_space_27_b200 as m
    return m


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
