"""Host-side checks of the gated delta rule's and the norms' C ABI (no GPU
needed, nothing launched): struct layouts, refusals, workspace sizes, and the
binding's own argument checks."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import selective_state_space_48_b200 as sss
from selective_state_space_48_b200 import builder as sbuild

FAKE = 0x10000
INV, UNS = sss.MSS_ERR_INVALID_ARG, sss.MSS_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    sbuild.build()
    return sss.load_library()


@pytest.mark.parametrize("header,name,mirror", [
    ("gated_delta.h", "mss_delta_args", sss.DeltaArgs),
    ("gated_delta.h", "mss_delta_update_args", sss.DeltaUpdateArgs),
    ("norm.h", "mss_gated_norm_args", sss.GatedNormArgs),
    ("norm.h", "mss_add_norm_args", sss.AddNormArgs)])
def test_struct_layout_matches_c(header, name, mirror):
    fields = [f[0] for f in mirror._fields_]
    src = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{header}"',
           "int main(void) {", f'printf("%zu\\n", sizeof({name}));']
    src += [f'printf("%zu\\n", offsetof({name}, {f}));' for f in fields] + ["return 0; }"]
    with tempfile.TemporaryDirectory() as tmp:
        c, exe = os.path.join(tmp, "l.c"), os.path.join(tmp, "l")
        open(c, "w").write("\n".join(src))
        subprocess.run(["gcc", "-I", sbuild.INCLUDE, c, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    assert [int(v) for v in out.split()] == \
        [ctypes.sizeof(mirror)] + [getattr(mirror, f).offset for f in fields]


def fill(a, kw):
    for k, v in kw.items():
        if isinstance(v, tuple):
            for i, x in enumerate(v):
                getattr(a, k)[i] = x
        else:
            setattr(a, k, v)
    return a


def delta_args(**kw):
    a = sss.DeltaArgs()
    B, L, H, P, G, N = 2, 100, 4, 64, 2, 64
    a.batch, a.seqlen, a.nheads, a.headdim, a.ngroups, a.dstate = B, L, H, P, G, N
    a.in_dtype = a.out_dtype = sss.MSS_BF16
    for n in ("q", "k", "v", "dt", "A", "beta", "y"):
        setattr(a, n, FAKE)
    for n, t in (("q", (L * G * N, G * N, N)), ("k", (L * G * N, G * N, N)),
                 ("v", (L * H * P, H * P, P)), ("y", (L * H * P, H * P, P)),
                 ("dt", (L * H, H, 1)), ("beta", (L * H, H, 1))):
        fill(a, {"stride_" + n: t})
    return fill(a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INV), (dict(seqlen=0), INV), (dict(nheads=0), INV), (dict(headdim=0), INV),
    (dict(dstate=0), INV), (dict(ngroups=3), INV), (dict(ngroups=0), INV),
    (dict(dstate=257), UNS), (dict(in_dtype=5), INV), (dict(out_dtype=-1), INV),
    (dict(q=0), INV), (dict(k=0), INV), (dict(v=0), INV), (dict(dt=0), INV), (dict(A=0), INV),
    (dict(beta=0), INV), (dict(y=0), INV), (dict(q=FAKE + 1), INV), (dict(A=FAKE + 2), INV),
    (dict(h0=FAKE + 2), INV), (dict(last_state=FAKE + 1), INV), (dict(dt_bias=FAKE + 3), INV),
    (dict(stride_q=(-1, 128, 64)), INV), (dict(stride_v=(1 << 50, 256, 64)), INV),
    (dict(stride_y=(25600, 255, 64)), INV), (dict(stride_y=(0, 256, 64)), INV),
    (dict(stride_y=(25600, 256, 63)), INV), (dict(num_seqs=2), INV),
    (dict(cu_seqlens=FAKE, num_seqs=2), INV),              # batch 2
    (dict(cu_seqlens=FAKE, num_seqs=0, batch=1), INV),
    (dict(cu_seqlens=FAKE + 2, num_seqs=2, batch=1), INV),
    (dict(plan=3), INV), (dict(plan=-1), INV), (dict(batch=1 << 31), UNS),
    (dict(seqlen=1 << 31), UNS), (dict(headdim=1 << 29, nheads=64, ngroups=1), UNS),
])
def test_delta_refusals(lib, kw, code):
    assert lib.gated_delta_fwd(ctypes.byref(delta_args(**kw)), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INV), (dict(ngroups=3), INV), (dict(dstate=300), UNS), (dict(state=0), INV),
    (dict(state=FAKE + 2), INV), (dict(v=0), INV), (dict(stride_y=(255, 64)), INV),
    (dict(stride_k=(-8, 64)), INV), (dict(in_dtype=9), INV)])
def test_update_refusals(lib, kw, code):
    a = sss.DeltaUpdateArgs()
    a.batch, a.nheads, a.headdim, a.ngroups, a.dstate = 2, 4, 64, 2, 64
    for n in ("state", "q", "k", "v", "dt", "A", "beta", "y"):
        setattr(a, n, FAKE)
    for n, t in (("q", (128, 64)), ("k", (128, 64)), ("v", (256, 64)), ("y", (256, 64)),
                 ("dt", (4, 1)), ("beta", (4, 1))):
        fill(a, {"stride_" + n: t})
    assert lib.gated_delta_update(ctypes.byref(fill(a, kw)), None) == code


def gated_args(**kw):
    a = sss.GatedNormArgs()
    a.rows, a.width, a.group_size, a.dtype, a.eps = 10, 128, 64, sss.MSS_BF16, 1e-5
    for n in ("x", "z", "weight", "y", "dy", "dx", "dz", "dweight"):
        setattr(a, n, FAKE)
    for n in ("x", "z", "y", "dy", "dx", "dz"):
        setattr(a, "stride_" + n, 128)
    return fill(a, kw)


@pytest.mark.parametrize("kw,fwd,bwd", [
    (dict(rows=0), INV, INV), (dict(width=0), INV, INV), (dict(group_size=0), INV, INV),
    (dict(group_size=60), INV, INV), (dict(dtype=3), INV, INV), (dict(eps=-1.0), INV, INV),
    (dict(eps=float("nan")), INV, INV), (dict(x=0), INV, INV), (dict(z=0), INV, INV),
    (dict(weight=0), INV, INV), (dict(weight=FAKE + 2), INV, INV), (dict(x=FAKE + 1), INV, INV),
    (dict(stride_x=-1), INV, INV), (dict(y=0), INV, None), (dict(stride_y=127), INV, None),
    (dict(dy=0), None, INV), (dict(dx=0), None, INV), (dict(stride_dz=100), None, INV),
    (dict(dweight=FAKE + 1), None, INV),
    (dict(width=16385 * 2, group_size=16385 * 2), UNS, UNS),
    (dict(width=65536, group_size=1), UNS, UNS), (dict(rows=1 << 40), UNS, UNS)])
def test_gated_norm_refusals(lib, kw, fwd, bwd):
    a = gated_args(**kw)
    if fwd is not None:
        assert lib.gated_rmsnorm_fwd(ctypes.byref(a), None) == fwd
    if bwd is not None:
        assert lib.gated_rmsnorm_bwd(ctypes.byref(a), None) == bwd


def add_args(**kw):
    a = sss.AddNormArgs()
    a.rows, a.width, a.dtype, a.res_dtype, a.eps = 10, 128, sss.MSS_BF16, sss.MSS_F32, 1e-5
    for n in ("x", "residual", "scale", "weight", "y", "residual_out", "dy", "dresidual_out", "dx",
              "dresidual", "dweight", "dscale"):
        setattr(a, n, FAKE)
    for n in ("x", "residual", "y", "residual_out", "dy", "dresidual_out", "dx", "dresidual"):
        setattr(a, "stride_" + n, 128)
    return fill(a, kw)


@pytest.mark.parametrize("kw,fwd,bwd", [
    (dict(rows=0), INV, INV), (dict(width=0), INV, INV), (dict(width=16385), UNS, UNS),
    (dict(dtype=sss.MSS_F32, res_dtype=sss.MSS_BF16), UNS, UNS), (dict(res_dtype=4), INV, INV),
    (dict(x=0), INV, INV), (dict(residual_out=0), INV, INV), (dict(scale=FAKE + 2), INV, INV),
    (dict(residual=FAKE + 2), INV, None), (dict(stride_residual=-4), INV, None),
    (dict(stride_residual_out=100), INV, None), (dict(y=FAKE + 1), INV, None),
    (dict(dresidual=FAKE + 2), None, INV), (dict(stride_dx=12), None, INV),
    (dict(dy=0), None, INV)])
def test_add_norm_refusals(lib, kw, fwd, bwd):
    a = add_args(**kw)
    if fwd is not None:
        assert lib.add_rmsnorm_fwd(ctypes.byref(a), None) == fwd
    if bwd is not None:
        assert lib.add_rmsnorm_bwd(ctypes.byref(a), None) == bwd


def test_null_arguments(lib):
    for f in (lib.gated_delta_fwd, lib.gated_delta_update, lib.gated_rmsnorm_fwd,
              lib.gated_rmsnorm_bwd, lib.add_rmsnorm_fwd, lib.add_rmsnorm_bwd):
        assert f(None, None) == INV
    n = ctypes.c_size_t(1)
    assert lib.mss_gated_rmsnorm_bwd_workspace_size(None, ctypes.byref(n)) == INV
    assert lib.mss_add_rmsnorm_bwd_workspace_size(ctypes.byref(add_args()), None) == INV
    # nothing to sum, nothing to hold (no device is asked for its size)
    assert lib.mss_gated_rmsnorm_bwd_workspace_size(
        ctypes.byref(gated_args(dweight=0)), ctypes.byref(n)) == sss.MSS_OK and n.value == 0
    assert lib.mss_add_rmsnorm_bwd_workspace_size(
        ctypes.byref(add_args(dweight=0, dscale=0)), ctypes.byref(n)) == sss.MSS_OK and n.value == 0


def test_binding_refuses_host_tensors_and_shapes():
    t = torch.zeros(2, 8, 4, 16)
    with pytest.raises(TypeError):
        sss.gated_delta_fwd(t, t, t, t[..., 0], torch.zeros(4), t[..., 0])
    with pytest.raises(ValueError):
        sss.gated_delta_fwd(t, t, t[0], t[..., 0], torch.zeros(4), t[..., 0])
    with pytest.raises(TypeError):
        sss.gated_delta_update(t, t[0], t[0], t[0], t[0, ..., 0], torch.zeros(4), t[0, ..., 0])
    with pytest.raises(TypeError):
        sss.gated_rmsnorm_fwd(t, t, torch.zeros(16))
    with pytest.raises(ValueError):
        sss.gated_rmsnorm_fwd(t, t, torch.zeros(16), group_size=5)
    with pytest.raises(ValueError):
        sss.gated_rmsnorm_fwd(t, t, torch.zeros(9))
    with pytest.raises(TypeError):
        sss.add_rmsnorm_fwd(t, t, torch.zeros(16))
    # leading dimensions that are not one run of rows
    with pytest.raises(ValueError):
        sss._rows_of("x", torch.zeros(4, 6, 16)[:, :3])
    assert sss._rows_of("x", torch.zeros(4, 6, 32)[..., :16]) == (24, 32)
    assert sss._rows_of("x", torch.zeros(1, 6, 1, 16)[:, ::2]) == (3, 32)


@pytest.mark.parametrize("n", ["q", "k", "v", "dt", "A", "beta"])
def test_delta_binding_refuses_what_is_no_tensor(n):
    """A missing tensor is a TypeError or ValueError that names the
    arguments, with a final state asked for or not."""
    d = dict(q=torch.zeros(1, 40, 1, 8), k=torch.zeros(1, 40, 1, 8), v=torch.zeros(1, 40, 1, 8),
             dt=torch.zeros(1, 40, 1), A=torch.zeros(1), beta=torch.zeros(1, 40, 1))
    for value in (None, 3.0):
        for last in (False, True):
            with pytest.raises((TypeError, ValueError)):
                sss.gated_delta_fwd(**dict(d, **{n: value}), return_last_state=last)


def test_delta_workspace_size_without_a_cut(lib):
    """0 for packed sequences, fp32 and the recurrent plan, whatever the
    device; refusals for sizes that a call refuses."""
    n = ctypes.c_size_t(9)
    size = lambda a: lib.mss_gated_delta_workspace_size(ctypes.byref(a), ctypes.byref(n))  # noqa: E731
    for kw in (dict(batch=1, cu_seqlens=FAKE, num_seqs=3), dict(in_dtype=sss.MSS_F32),
               dict(plan=sss.MSS_DELTA_RECURRENT), dict(dstate=200)):
        n.value = 9
        assert size(delta_args(**kw)) == sss.MSS_OK and n.value == 0
    assert size(delta_args(dstate=300)) == UNS
    assert size(delta_args(seqlen=0)) == INV
    assert lib.mss_gated_delta_workspace_size(None, ctypes.byref(n)) == INV


@pytest.mark.parametrize("cu", [[0, 40], 3, torch.tensor([0, 40]), torch.zeros(0, dtype=torch.int32),
                                torch.zeros(1, dtype=torch.int32)])
def test_offsets_that_are_none_are_refused_by_name(cu):
    d = dict(q=torch.zeros(1, 40, 1, 8), k=torch.zeros(1, 40, 1, 8), v=torch.zeros(1, 40, 1, 8),
             dt=torch.zeros(1, 40, 1), A=torch.zeros(1), beta=torch.zeros(1, 40, 1))
    for last in (False, True):
        with pytest.raises((TypeError, ValueError), match="cu_seqlens"):
            sss.gated_delta_fwd(**d, cu_seqlens=cu, return_last_state=last)
