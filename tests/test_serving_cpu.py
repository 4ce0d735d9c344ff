"""The serving operators without a GPU: the structs' layouts in the header, the
binding's mirrors and its packing agree; bad arguments are refused before any
CUDA call; calls with nothing to do return at once."""
import ctypes
import os
import subprocess

import pytest
import torch

import selective_state_space_27_b200 as ms
from selective_state_space_27_b200 import build as msbuild

msbuild.build()
from selective_state_space_27_b200 import serving   # noqa: E402  (needs the compiled tensor checks)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INCLUDE = os.path.join(ROOT, "include")
BASE = 1 << 20
STRUCTS = [("ms_conv_packed_args", ms.ConvPackedArgs, serving.CONV_PACKED),
           ("ms_conv1d_args", ms.Conv1dArgs, serving.CONV1D),
           ("ms_ssd_packed_args", ms.SsdPackedArgs, serving.SSD_PACKED),
           ("ms_ssd_update_args", ms.SsdUpdateArgs, serving.SSD_UPDATE),
           ("ms_norm_args", ms.NormArgs, None), ("ms_norm_bwd_args", ms.NormBwdArgs, None)]   # (packed in C++)


@pytest.fixture(scope="module")
def lib():
    msbuild.build()
    return ms.load_library()


@pytest.mark.parametrize("name,mirror,packing", STRUCTS)
def test_struct_layouts_agree(tmp_path, name, mirror, packing):
    fields = [f for f, _ in mirror._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mambascan.h"\nint main(void){\n' +
                   f'printf("%zu", sizeof({name}));\n' +
                   "".join(f'printf(" %zu", offsetof({name}, {f}));\n' for f in fields) + "return 0;}\n")
    subprocess.check_call(["gcc", "-std=c11", "-I", INCLUDE, str(src), "-o", str(tmp_path / "layout")])
    got = [int(v) for v in subprocess.check_output([str(tmp_path / "layout")], text=True).split()]
    assert got == [ctypes.sizeof(mirror)] + [getattr(mirror, f).offset for f in fields]
    if packing is None:
        return
    values = [float(i + 1) if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(mirror._fields_)]
    packed = mirror.from_buffer_copy(packing.pack(*values))
    assert packing.size == ctypes.sizeof(mirror) and [getattr(packed, f) for f in fields] == values


def _set(a, **kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def conv_args(**kw):
    a = ms.ConvPackedArgs()
    _set(a, tokens=100, channels=64, nseq=3, slots=5, in_dtype=ms.MS_BF16, x=BASE, x_token_stride=64, y=2 * BASE,
         y_token_stride=64, state=3 * BASE, state_slot_stride=192, state_row_stride=64, cu_seqlens=4 * BASE,
         state_indices=5 * BASE, has_initial_state=6 * BASE)
    return _set(a, **kw)


def conv_filter(**kw):
    return _set(_set(ms.Conv1dArgs(), weight=7 * BASE, bias=8 * BASE, width=4, silu=1), **kw)


@pytest.mark.parametrize("change,status", [
    (dict(in_dtype=7), 1), (dict(reserved=1), 1), (dict(tokens=-1), 1), (dict(tokens=1 << 31), 1),
    (dict(channels=0), 1), (dict(channels=(1 << 22) + 1), 1), (dict(nseq=-1), 1), (dict(slots=-1), 1),
    (dict(x=None), 1), (dict(y=None), 1), (dict(y_token_stride=63), 1), (dict(x_token_stride=-1), 1),
    (dict(state_row_stride=63), 1), (dict(state_slot_stride=128), 1), (dict(state=None), 1),
    (dict(state_indices=None, slots=2), 1),
    (dict(cu_seqlens=None), 1), (dict(cu_seqlens=None, nseq=100, slots=200), 1),
    (dict(cu_seqlens=None, nseq=100, has_initial_state=None, state=None, state_indices=None), 1),
    (dict(x=BASE + 1), 3), (dict(state=BASE * 3 + 1), 3), (dict(cu_seqlens=4 * BASE + 2), 3),
    (dict(state_indices=5 * BASE + 2), 3),
])
def test_conv_packed_refuses(lib, change, status):
    assert lib.mamba_conv_packed_fwd(ctypes.byref(conv_args(**change)), ctypes.byref(conv_filter()), None) == status


def test_conv_packed_refuses_in_place(lib):
    assert lib.mamba_conv_packed_fwd(ctypes.byref(conv_args(y=BASE)), ctypes.byref(conv_filter()), None) == 1
    assert b"in place" in lib.mamba_last_error()


@pytest.mark.parametrize("change,status", [(dict(weight=None), 1), (dict(width=0), 1), (dict(width=5), 2),
                                           (dict(silu=2), 1), (dict(weight=BASE + 2), 3)])
def test_conv_packed_refuses_filters(lib, change, status):
    assert lib.mamba_conv_packed_fwd(ctypes.byref(conv_args()), ctypes.byref(conv_filter(**change)), None) == status
    assert lib.mamba_conv_packed_fwd(None, ctypes.byref(conv_filter()), None) == 1
    assert lib.mamba_conv_packed_fwd(ctypes.byref(conv_args()), None, None) == 1


def ssd_args(**kw):
    a = ms.SsdPackedArgs()
    _set(a, tokens=100, nseq=3, nheads=4, ngroups=2, slots=5, in_dtype=ms.MS_BF16, dt_softplus=1, x=BASE,
         x_token_stride=256, dt=2 * BASE, dt_token_stride=4, B=3 * BASE, B_token_stride=256, C=4 * BASE,
         C_token_stride=256, y=5 * BASE, y_token_stride=256, A=6 * BASE, state=7 * BASE,
         state_slot_stride=4 * 64 * 128, cu_seqlens=8 * BASE, state_indices=9 * BASE, has_initial_state=10 * BASE)
    return _set(a, **kw)


SSD_REFUSED = [
    (dict(nheads=0), 1), (dict(ngroups=3), 1), (dict(reserved=1), 1), (dict(in_dtype=ms.MS_F32), 2),
    (dict(in_dtype=9), 1), (dict(tokens=-1), 1), (dict(max_seqlen=-1), 1), (dict(nheads=65536, ngroups=1), 2),
    (dict(nseq=1 << 28, slots=1 << 29), 2), (dict(nseq=-1), 1), (dict(x=None), 1), (dict(A=None), 1),
    (dict(cu_seqlens=None), 1), (dict(x_token_stride=248), 1), (dict(B_token_stride=128), 1),
    (dict(dt_token_stride=3), 1), (dict(z=BASE, z_token_stride=8), 1), (dict(state=None), 1),
    (dict(state_indices=None, slots=2), 1), (dict(state_slot_stride=64), 1),
    (dict(x_token_stride=260), 3), (dict(y=5 * BASE + 8), 3), (dict(C=4 * BASE + 8), 3), (dict(state=7 * BASE + 2), 3),
    (dict(dt=2 * BASE + 1), 3), (dict(A=6 * BASE + 2), 3), (dict(cu_seqlens=8 * BASE + 1), 3),
]


@pytest.mark.parametrize("change,status", SSD_REFUSED)
def test_ssd_packed_refuses(lib, change, status):
    a, n = ssd_args(**change), ctypes.c_size_t(7)
    assert lib.mamba_ssd_packed_workspace_size(ctypes.byref(a), ctypes.byref(n)) == status and n.value == 0
    assert lib.mamba_ssd_packed_fwd(ctypes.byref(a), 11 * BASE, 1 << 40, None) == status


def test_ssd_packed_needs_its_arguments(lib):
    n = ctypes.c_size_t(0)
    assert lib.mamba_ssd_packed_workspace_size(None, ctypes.byref(n)) == 1
    assert lib.mamba_ssd_packed_workspace_size(ctypes.byref(ssd_args()), None) == 1
    assert lib.mamba_ssd_packed_fwd(None, 11 * BASE, 256, None) == 1


def update_args(**kw):
    a = ms.SsdUpdateArgs()
    _set(a, batch=3, nheads=4, ngroups=2, headdim=64, dstate=128, slots=5, in_dtype=ms.MS_BF16, state=BASE,
         state_slot_stride=4 * 64 * 128, x=2 * BASE, x_batch_stride=256, dt=3 * BASE, dt_batch_stride=4, B=4 * BASE,
         B_batch_stride=256, C=5 * BASE, C_batch_stride=256, y=6 * BASE, y_batch_stride=256, A=7 * BASE,
         state_indices=8 * BASE)
    return _set(a, **kw)


@pytest.mark.parametrize("change,status", [
    (dict(in_dtype=5), 1), (dict(batch=-1), 1), (dict(nheads=0), 1), (dict(ngroups=3), 1), (dict(headdim=0), 1),
    (dict(dstate=0), 1), (dict(dstate=257, state_slot_stride=1 << 20), 2), (dict(batch=65536), 2),
    (dict(headdim=65536), 2), (dict(state=None), 1), (dict(x=None), 1), (dict(A=None), 1), (dict(B_batch_stride=-1), 1),
    (dict(y_batch_stride=255), 1), (dict(state_slot_stride=128), 1), (dict(state_indices=None, slots=2), 1),
    (dict(x=2 * BASE + 1), 3), (dict(state=BASE + 2), 3), (dict(state_indices=8 * BASE + 1), 3),
])
def test_ssd_update_refuses(lib, change, status):
    assert lib.mamba_ssd_state_update(ctypes.byref(update_args(**change)), None) == status
    assert lib.mamba_ssd_state_update(None, None) == 1


def norm_args(**kw):
    a = ms.NormArgs()
    _set(a, rows=10, dim=96, group_size=32, in_dtype=ms.MS_BF16, residual_dtype=ms.MS_F32, eps=1e-5,
         residual_scale=1.0, gate_first=1, x=BASE, x_row_stride=96, z=2 * BASE, z_row_stride=96, residual=3 * BASE,
         residual_row_stride=96, residual_out=4 * BASE, residual_out_row_stride=96, y=5 * BASE, y_row_stride=96,
         weight=6 * BASE)
    return _set(a, **kw)


def norm_grads(**kw):
    g = ms.NormBwdArgs()
    _set(g, dy=BASE, dy_row_stride=96, dresidual_out=2 * BASE, dresidual_out_row_stride=96, dx=3 * BASE,
         dx_row_stride=96, dz=4 * BASE, dz_row_stride=96, dresidual=5 * BASE, dresidual_row_stride=96,
         dweight=6 * BASE)
    return _set(g, **kw)


NORM_REFUSED = [
    (dict(in_dtype=4), 1), (dict(reserved=1), 1), (dict(rows=-1), 1), (dict(dim=0), 1), (dict(group_size=0), 1),
    (dict(group_size=36), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(gate_first=2), 1), (dict(residual_dtype=3), 1), (dict(in_dtype=ms.MS_F32, residual_dtype=ms.MS_BF16), 1),
    (dict(dim=1 << 31, group_size=1 << 31), 2), (dict(rows=1 << 30), 2), (dict(x_row_stride=-1), 1),
    (dict(x=BASE + 1), 3), (dict(residual_out=4 * BASE + 2), 3), (dict(weight=6 * BASE + 2), 3),
]


@pytest.mark.parametrize("change,status", NORM_REFUSED + [
    (dict(x=None), 1), (dict(y=None), 1), (dict(residual_out=None), 1), (dict(residual=None), 1),
    (dict(y_row_stride=95), 1), (dict(residual_out_row_stride=95), 1), (dict(y=5 * BASE + 1), 3)])
def test_norm_refuses(lib, change, status):
    assert lib.mamba_norm_fwd(ctypes.byref(norm_args(**change)), None) == status
    assert lib.mamba_norm_fwd(None, None) == 1


@pytest.mark.parametrize("change,status", NORM_REFUSED)
def test_norm_bwd_refuses_the_forward(lib, change, status):
    a, n = norm_args(**change), ctypes.c_size_t(7)
    assert lib.mamba_norm_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == status and n.value == 0
    assert lib.mamba_norm_bwd(ctypes.byref(a), ctypes.byref(norm_grads()), 7 * BASE, 1 << 40, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(dz=None), 1), (dict(dresidual=None), 1), (dict(dx_row_stride=95), 1),
    (dict(dy_row_stride=-1), 1), (dict(dx=3 * BASE + 1), 3), (dict(dresidual=5 * BASE + 2), 3),
    (dict(dweight=6 * BASE + 1), 3)])
def test_norm_bwd_refuses(lib, change, status):
    a = norm_args()
    assert lib.mamba_norm_bwd(ctypes.byref(a), ctypes.byref(norm_grads(**change)), 7 * BASE, 1 << 40, None) == status
    assert lib.mamba_norm_bwd(ctypes.byref(a), None, None, 0, None) == 1
    a = norm_args(residual=None, residual_out=None)
    assert lib.mamba_norm_bwd(ctypes.byref(a), ctypes.byref(norm_grads()), 7 * BASE, 1 << 40, None) == 1


def test_nothing_to_do(lib):
    """No sequences, requests or rows: MS_OK without a device."""
    a = conv_args(nseq=0, tokens=0, x=None, y=None)
    assert lib.mamba_conv_packed_fwd(ctypes.byref(a), ctypes.byref(conv_filter()), None) == 0
    assert lib.mamba_ssd_state_update(ctypes.byref(update_args(batch=0, x=None)), None) == 0
    assert lib.mamba_norm_fwd(ctypes.byref(norm_args(rows=0, x=None, y=None)), None) == 0
    n = ctypes.c_size_t(7)
    assert lib.mamba_norm_bwd_workspace_size(ctypes.byref(norm_args(rows=0)), ctypes.byref(n)) == 0 and n.value == 0
    assert lib.mamba_norm_bwd(ctypes.byref(norm_args(rows=0)), ctypes.byref(norm_grads(dweight=None)), None, 0,
                              None) == 0


def test_python_calls_refuse_host_tensors():
    f = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        ms.norm_fwd(f(2, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ms.norm_bwd(f(2, 8), f(2, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ms.conv_packed_update(f(2, 3, 8), f(2, 8), f(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        ms.ssd_state_update(f(2, 1, 4, 8), f(2, 1, 4), f(2, 1), f(1), f(2, 1, 8), f(2, 1, 8))
    with pytest.raises(AttributeError):
        ms.no_such_name


def test_tensor_checks():
    """The compiled checks: pointers, strides and refusals."""
    from selective_state_space_27_b200 import _binding as b
    f32, cpu = torch.float32, torch.device("cpu")
    x = torch.zeros(6, 4, 8)
    assert b.rows("x", x, f32, x.shape, cpu) == (x.data_ptr(), 32)
    y = torch.zeros(6, 50)[:, 10:42].unflatten(1, (4, 8))
    assert b.rows("y", y, f32, (6, 4, 8), cpu) == (y.data_ptr(), 50)
    assert b.rows("x", x[:1], f32, (1, 4, 8), cpu) == (x.data_ptr(), 32)
    assert b.rows("x", x[:0], f32, (0, 4, 8), cpu)[1] == 32
    assert b.rows("x", x[:1].expand(6, 4, 8), f32, (6, 4, 8), cpu) == (x.data_ptr(), 0)
    assert b.rows("none", None, f32, (1,), cpu) == (0, 0) and b.vector("none", None, 3, cpu, f32) == 0
    for bad in (x.transpose(1, 2).contiguous().transpose(1, 2), x[:, :, ::2], x.expand(6, 4, 8)[:, ::2]):
        with pytest.raises(ValueError, match="contiguous"):
            b.rows("x", bad, f32, bad.shape, cpu)
    with pytest.raises(TypeError, match="x must be torch.bfloat16, got torch.float32"):
        b.rows("x", x, torch.bfloat16, x.shape, cpu)
    with pytest.raises(ValueError, match="shape"):
        b.rows("x", x, f32, (6, 4, 9), cpu)
    with pytest.raises(ValueError, match="slots"):
        b.rows("x", x, f32, ("slots", 4, 8), cpu)
    with pytest.raises(ValueError, match="is on cpu"):
        b.rows("x", x, f32, x.shape, torch.device("cuda", 0))
    with pytest.raises(TypeError, match="tensor"):
        b.rows("x", [1.0], f32, (1,), cpu)
    v = torch.arange(5, dtype=torch.int32)
    assert b.vector("v", v, 5, cpu, torch.int32) == v.data_ptr()
    with pytest.raises(ValueError, match="shape"):
        b.vector("v", v, 4, cpu, torch.int32)
    with pytest.raises(ValueError, match="contiguous"):
        b.vector("v", torch.zeros(10)[::2], 5, cpu, f32)
    with pytest.raises(TypeError):
        b.vector("v", v, 5, cpu, f32)
    e = b.empty_like(y)
    assert e.shape == y.shape and e.dtype is f32 and e.is_contiguous()


def test_segments_have_places():
    """The map from places to (sequence, segment): sequence s starts at place
    cu[s] // Qs + s, so that no sequence's segments reach the next one's first
    place, for every ragged split tried."""
    import random
    r = random.Random(0)
    for _ in range(400):
        chunks = r.choice([2, 3, 4, 7, 16])
        size = chunks * 128
        lens = [r.choice([0, 0, 1, 127, 128, 129, size - 1, size, size + 1, r.randrange(5000)])
                for _ in range(r.choice([1, 2, 3, 31, 32, 33, 70]))]
        start, end_before = 0, -1
        total = sum(lens)
        for s, n in enumerate(lens):
            first = start // size + s
            assert first > end_before
            end_before = first + max(1, -(-n // size)) - 1
            start += n
        assert end_before < total // size + len(lens)
