"""GPU test of the ``stream`` argument of the scans, their backward and the decode steps: what a call allocates is memory
of that stream."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ms():
    import selective_state_space_27_b200 as m
    return m


def calls(ms):
    """name -> call of a stream; what it updates in place is made anew by each call and there before the call starts."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, device="cuda", generator=g).to(dtype)

    b, d, n, L, f32 = 2, 256, 16, 700, torch.float32
    u, delta, z, dy, lam = (normal(b, d, L) for _ in range(5))
    B, C = normal(b, n, L), normal(b, n, L)
    A, filt = -torch.rand(d, n, device="cuda", generator=g), normal(d, 4, dtype=f32)
    state, conv_state = normal(b, d, n, dtype=f32), normal(b, d, 4)
    xs, dts = normal(b, L, 4, 64), normal(b, L, 4)
    Bs, Cs, As = normal(b, L, 1, 128), normal(b, L, 1, 128), -torch.rand(4, device="cuda", generator=g)
    kept = []

    def fresh(t):
        kept.append(t.clone())
        torch.cuda.synchronize()
        return kept[-1]

    step = (u[:, :, 0].contiguous(), delta[:, :, 0].contiguous(), A, B[:, :, 0].contiguous(), C[:, :, 0].contiguous())
    return {
        "scan_fwd": lambda s: ms.scan_fwd(u, delta, A, B, C, z=z, stream=s),
        "scan_fwd_segments": lambda s: ms.scan_fwd(u, delta, A, B, C, force_segments=4, stream=s),
        "state_update": lambda s: ms.state_update(fresh(state), *step, stream=s),
        "conv_scan_fwd": lambda s: ms.conv_scan_fwd(u, filt, delta, A, B, C, stream=s),
        "conv_state_update": lambda s: ms.conv_state_update(fresh(state), fresh(conv_state), step[0], filt, *step[1:],
                                                            stream=s),
        "trap_scan_fwd": lambda s: ms.trap_scan_fwd(u, delta, lam, A, B, C, stream=s),
        "scan_bwd": lambda s: ms.scan_bwd(u, delta, A, B, C, dy, z=z, stream=s),
        "ssd_fwd": lambda s: ms.ssd_fwd(xs, dts, As, Bs, Cs, check=False, stream=s),
    }


def tensors(result):
    if isinstance(result, dict):
        result = tuple(result.values())
    return [t for t in (result if isinstance(result, tuple) else (result,)) if t is not None]


@pytest.mark.parametrize("name", ["scan_fwd", "scan_fwd_segments", "state_update", "conv_scan_fwd", "conv_state_update",
                                  "trap_scan_fwd", "scan_bwd", "ssd_fwd"])
def test_given_stream_owns_what_the_call_allocates(ms, name):
    """The outputs are not memory that the current stream has just given back, and dropped ones do not go to the current
    stream while the call still writes them."""
    call = calls(ms)[name]
    want = [t.clone() for t in tensors(call(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty_like(t) for t in want for _ in range(3)]
    freed = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in blocks]
    del blocks
    got = tensors(call(side))
    assert not any(lo <= t.data_ptr() < hi for t in got for lo, hi in freed)
    side.synchronize()
    # (the backward adds dA, dB, dC and the like up by atomics, in no fixed order: its row gradients are compared)
    assert len(got) == len(want) and all(t.isfinite().all() for t in got)
    rows = got[:3] if name == "scan_bwd" else got
    assert all(torch.equal(t, w) for t, w in zip(rows, want))
    for _ in range(3):
        places = {t.data_ptr() for t in tensors(call(side))}      # dropped at once
        mine = [torch.full_like(w, 3.0) for w in want]
        assert not places & {t.data_ptr() for t in mine}
        torch.cuda.synchronize()
        assert all((t == 3.0).all() for t in mine)
