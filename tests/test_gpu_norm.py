"""RMS norms before and after a block, forward and backward, against float64
(needs a GPU).

Tolerances, relative to the largest value: a sum over a row of D values (or
over R rows) is taken by threads and a tree, at most D/128 + 16 roundings deep
(rows: R / 16 + 64), each half a step of fp32; the rest of the formulas is
about 16 roundings, and the special functions are good to a few 1e-7 (8 half
steps).  An output of type t adds half a step of t.

The gradient through the norm is the difference of rstd dn and
rstd n mean(dn o n), each rounded to half a step of itself.  Where they
nearly cancel the difference keeps that absolute error, however small it is:
with one channel n^2 = a^2 / (a^2 + eps), so the difference is
eps / (a^2 + eps) of either term, 1e-5 and less.  Its error is therefore
measured against the larger of the value and of its first term (the second is
at most sqrt(D) mean |dn o n| <= max |dn| times a factor that the first term
of some channel reaches).
"""
import ctypes

import pytest
import torch

import selective_state_space_48_b200 as sss
from delta_checks import F64, gated_rmsnorm, rmsnorm, worst

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def tol(D, dtype=F32, rows=0):
    return (D / 128 + 16 + 16 + 8 + (rows / 16 + 64 if rows else 0)) * U + \
        (2.0 ** -8 if dtype == BF else 0.0)


def silu(z):
    return z / (1 + torch.exp(-z))


def silu_grad(z):
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def rnd(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


# rows, width, group
SHAPES = [(1, 1, 1), (3, 8, 8), (5, 64, 64), (17, 384, 64), (9, 7, 7), (33, 231, 77), (4, 128, 128),
          (130, 256, 256), (6, 600, 600), (300, 1155, 385), (7, 2048, 1024), (5, 2560, 2560),
          (64, 4096, 4096), (3, 5000, 5000), (2, 8192, 8192), (3, 9000, 9000), (2, 16384, 16384),
          (1000, 320, 16)]


@pytest.mark.parametrize("before", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", SHAPES)
def test_gated(shape, dtype, before):
    rows, width, group = shape
    for shared in (False, True):
        r = rnd(rows + width)
        x, z, dy = (r(rows, width).to(dtype) for _ in range(3))
        w = 1 + 0.1 * r(group if shared else width)
        kw = dict(eps=1e-5, group_size=group, norm_before_gate=before)
        y = sss.gated_rmsnorm_fwd(x, z, w, **kw)
        g = sss.gated_rmsnorm_bwd(x, z, w, dy, **kw)
        again = sss.gated_rmsnorm_bwd(x, z, w, dy, **kw)
        lx, lz, lw = (t.to(F64).requires_grad_() for t in (x, z, w))
        yr = gated_rmsnorm(lx, lz, lw, 1e-5, group, before)
        dx, dz, dw = torch.autograd.grad(yr, (lx, lz, lw), dy.to(F64))
        assert y.dtype == dtype and worst(y, yr) <= tol(group, dtype)
        # rstd dn times the factor that follows it into dx and dz
        gate, dgate = (f(lz.detach()) for f in (silu, silu_grad))
        a = (lx if before else lx * gate).detach().reshape(rows, -1, group)
        rstd = (a.pow(2).mean(-1, keepdim=True) + 1e-5).rsqrt().expand_as(a).reshape(rows, width)
        dn = rstd * dy.to(F64) * lw.detach().repeat(width // lw.numel())
        assert worst(g["dx"], dx, dn * gate) <= tol(group, dtype)
        assert worst(g["dz"], dz, None if before else dn * lx * dgate) <= tol(group, dtype)
        assert worst(g["dweight"], dw) <= tol(group, F32, rows * (width // group))
        assert all(torch.equal(g[n], again[n]) for n in g)


@pytest.mark.parametrize("dtype,res", [(F32, F32), (BF, F32), (BF, BF)])
@pytest.mark.parametrize("shape", [s[:2] for s in SHAPES])
def test_add(shape, dtype, res):
    rows, width = shape
    r = rnd(rows * 3 + width)
    x, dy = r(rows, width).to(dtype), r(rows, width).to(dtype)
    residual, dres = (4 * r(rows, width)).to(res), r(rows, width).to(res)
    w, scale = 1 + 0.1 * r(width), 0.5 + 0.1 * r(width)
    for scl, resid in ((scale, residual), (None, residual), (scale, None)):
        y, out = sss.add_rmsnorm_fwd(x, resid, w, scale=scl, residual_dtype=res)
        total = x.to(F64) * (1 if scl is None else scl.to(F64))
        total = total + (0 if resid is None else resid.to(F64))
        assert out.dtype == res and worst(out, total) <= 2 * U + (2.0 ** -8 if res == BF else 0)
        h, lw = out.to(F64).requires_grad_(), w.to(F64).requires_grad_()
        yr = rmsnorm(h, lw, 1e-5)
        assert worst(y, yr) <= tol(width, dtype)
        up = dres if resid is not None else None
        g = sss.add_rmsnorm_bwd(out, w, dy, dresidual_out=up, x=x, scale=scl)
        dh, dw = torch.autograd.grad(yr, (h, lw), dy.to(F64))
        dh = dh + (0 if up is None else up.to(F64))
        dn = (h.pow(2).mean(-1, keepdim=True) + 1e-5).rsqrt() * dy.to(F64) * lw
        s = 1 if scl is None else scl.to(F64)
        assert worst(g["dresidual"], dh, dn) <= tol(width, res)
        assert worst(g["dx"], dh * s, dn * s) <= tol(width, dtype)
        assert worst(g["dweight"], dw) <= tol(width, F32, rows)
        if scl is None:
            assert g["dscale"] is None
        else:
            assert worst(g["dscale"], (dh * x.to(F64)).sum(0), dn * x.to(F64)) <= \
                tol(width, F32, rows)


def test_gradients_against_differences():
    """dx, dz and dweight of the gated norm and dx, dscale of the other along
    random directions against central differences of the CUDA forward in
    fp32: at step h the difference is off by h^2 of the third derivative and
    by the forward's rounding over h."""
    r = rnd(5)
    x, z, w, dy = r(6, 96), r(6, 96), 1 + 0.1 * r(96), r(6, 96)
    h = 2.0 ** -7  # h^2 = 6e-5; rounding 2^-22 * sqrt(576) / h = 7e-4
    for before in (False, True):
        kw = dict(group_size=32, norm_before_gate=before)
        f = lambda x, z, w: float((sss.gated_rmsnorm_fwd(x, z, w, **kw).double() * dy).sum())  # noqa: E731
        g = sss.gated_rmsnorm_bwd(x, z, w, dy, **kw)
        for i, n in enumerate(("dx", "dz", "dweight")):
            args = [x, z, w]
            d = r(*args[i].shape)
            lo, hi = list(args), list(args)
            lo[i], hi[i] = args[i] - h * d, args[i] + h * d
            want = (f(*hi) - f(*lo)) / (2 * h)
            size = float((g[n].abs() * d.abs()).sum())
            assert abs(want - float((g[n] * d).sum())) <= 2e-3 * size
    scale, res = 0.5 + 0.1 * r(96), r(6, 96)
    f = lambda x, s: float((sss.add_rmsnorm_fwd(x, res, w, scale=s)[0].double() * dy).sum())  # noqa: E731
    _, out = sss.add_rmsnorm_fwd(x, res, w, scale=scale)
    g = sss.add_rmsnorm_bwd(out, w, dy, x=x, scale=scale)
    for n, d, pair in (("dx", r(6, 96), lambda s, d: (x + s * d, scale)),
                       ("dscale", r(96), lambda s, d: (x, scale + s * d))):
        want = (f(*pair(h, d)) - f(*pair(-h, d))) / (2 * h)
        assert abs(want - float((g[n] * d).sum())) <= 2e-3 * float((g[n].abs() * d.abs()).sum())


def test_views_and_in_place():
    """Halves of a projection, 3-d inputs, the residual updated in place."""
    r = rnd(9)
    both = r(4, 10, 512).to(BF)
    x, z = both.chunk(2, -1)
    w = 1 + 0.1 * r(256)
    y = sss.gated_rmsnorm_fwd(x, z, w, group_size=64)
    assert torch.equal(y, sss.gated_rmsnorm_fwd(x.contiguous(), z.contiguous(), w, group_size=64))
    odd = r(7, 300)[:, 1:256]
    w1 = 1 + 0.1 * r(255)
    assert torch.equal(sss.gated_rmsnorm_fwd(odd, odd, w1),
                       sss.gated_rmsnorm_fwd(odd.contiguous(), odd.contiguous(), w1))
    res = r(4, 10, 256)
    want_y, want = sss.add_rmsnorm_fwd(x, res, w)
    y, out = sss.add_rmsnorm_fwd(x, res, w, residual_out=res)
    assert out is res and torch.equal(res, want) and torch.equal(y, want_y)


def test_zero_rows_and_non_finite_rows_stay_apart():
    """A row of zeros gives zeros; a row with an infinity or NaN spoils only
    itself (and, in the backward, the sums over rows)."""
    r = rnd(3)
    x, z, w, dy = r(6, 64), r(6, 64), 1 + 0.1 * r(64), r(6, 64)
    clean = sss.gated_rmsnorm_fwd(x, z, w)
    x[1] = 0
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    y = sss.gated_rmsnorm_fwd(x, z, w)
    g = sss.gated_rmsnorm_bwd(x, z, w, dy, need_dweight=False)
    assert g["dweight"] is None
    assert (y[1] == 0).all()
    for i in (0, 2, 5):
        assert torch.equal(y[i], clean[i]) and torch.isfinite(g["dx"][i]).all()
    assert torch.isnan(y[4]).all()
    big = torch.full((2, 64), 100.0, device="cuda")
    assert torch.isfinite(sss.gated_rmsnorm_bwd(r(2, 64), -big, w, r(2, 64))["dz"]).all()


def test_autograd_layer():
    """add norm -> gated norm through the autograd wrappers, shared inputs
    and a broadcast residual, against float64."""
    r = rnd(11)
    x, res = r(5, 1, 128), r(1, 1, 128)
    w1, w2, scale = 1 + 0.1 * r(128), 1 + 0.1 * r(32), 0.5 + 0.1 * r(128)
    leaves = [t.clone().requires_grad_() for t in (x, res, w1, w2, scale)]
    def run(x, res, w1, w2, scale, own):
        res = res.expand(5, 3, 128)
        xe = x.expand(5, 3, 128)
        if own:
            y, out = sss.add_rmsnorm_fn(xe, res, w1, scale=scale)
            o = sss.gated_rmsnorm_fn(y, out, w2, group_size=32)
        else:
            out = res + scale * xe
            y = rmsnorm(out, w1, 1e-5)
            o = gated_rmsnorm(y, out, w2, 1e-5, 32, False)
        return (o * torch.arange(1, 385, device="cuda").view(3, 128) / 384).sum() + (out ** 2).sum()
    got = torch.autograd.grad(run(*leaves, True), leaves)
    ref = [t.detach().to(F64).requires_grad_() for t in leaves]
    want = torch.autograd.grad(run(*ref, False), ref)
    for a, b in zip(got, want):
        assert worst(a, b) <= 4 * tol(128, F32, 15)


def test_fn_with_unused_outputs():
    r = rnd(2)
    x, res, w = r(4, 64).to(BF).requires_grad_(), r(4, 64).requires_grad_(), 1 + 0.1 * r(64)
    y, out = sss.add_rmsnorm_fn(x, res, w)
    dx, dres = torch.autograd.grad(out.sum(), (x, res))
    assert (dres == 1).all() and (dx == 1).all()
    y, out = sss.add_rmsnorm_fn(x, res, w)
    torch.autograd.grad(y.float().sum(), (x, res))


def test_graph_capture_and_other_stream():
    r = rnd(4)
    x, z, w, dy = r(40, 256).to(BF), r(40, 256).to(BF), 1 + 0.1 * r(256), r(40, 256).to(BF)
    want = sss.gated_rmsnorm_bwd(x, z, w, dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sss.gated_rmsnorm_bwd(x, z, w, dy, stream=side)
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(sss.gated_rmsnorm_bwd(x, z, w, dy))
        graphs.append(graph)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("width", [16, 128, 512, 640])
def test_no_epsilon(width):
    """eps 0 and a number of rows that fills no block: the places behind the
    last row add nothing to the sums over rows."""
    r = rnd(width)
    x, z, w, dy = r(5, width), r(5, width), 1 + 0.1 * r(width), r(5, width)
    g = sss.gated_rmsnorm_bwd(x, z, w, dy, eps=0.0)
    lx, lz, lw = (t.to(F64).requires_grad_() for t in (x, z, w))
    dw, = torch.autograd.grad(gated_rmsnorm(lx, lz, lw, 0.0, width, False), lw, dy.to(F64))
    assert worst(g["dweight"], dw) <= tol(width, F32, 5)
    g = sss.add_rmsnorm_bwd(x, w, dy, eps=0.0)
    lx = x.to(F64).requires_grad_()
    dw, = torch.autograd.grad(rmsnorm(lx, lw, 0.0), lw, dy.to(F64))
    assert worst(g["dweight"], dw) <= tol(width, F32, 5)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("width,group", [(320, 16), (1155, 385), (4096, 4096), (16384, 16384)])
def test_gradient_in_place_of_its_upstream(width, group, dtype):
    """dx, or dz, in the memory of dy, through the C entry point."""
    r = rnd(width + group)
    x, z, dy = (r(600, width).to(dtype) for _ in range(3))
    w = 1 + 0.1 * r(width)
    want = sss.gated_rmsnorm_bwd(x, z, w, dy, group_size=group)
    lib = sss.load_library()
    for place in ("dx", "dz"):
        a = sss.GatedNormArgs()
        a.rows, a.width, a.group_size, a.eps = 600, width, group, 1e-5
        a.dtype = sss.MSS_F32 if dtype == F32 else sss.MSS_BF16
        up, other, dw = dy.clone(), torch.empty_like(dy), torch.empty_like(w)
        a.x, a.z, a.weight, a.dy = x.data_ptr(), z.data_ptr(), w.data_ptr(), up.data_ptr()
        a.dx, a.dz = (t.data_ptr() for t in ((up, other) if place == "dx" else (other, up)))
        a.dweight = dw.data_ptr()
        for n in ("x", "z", "dy", "dx", "dz"):
            setattr(a, "stride_" + n, width)
        need = ctypes.c_size_t(0)
        assert lib.mss_gated_rmsnorm_bwd_workspace_size(ctypes.byref(a), ctypes.byref(need)) == 0
        ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
        a.workspace, a.workspace_bytes = ws.data_ptr(), need.value
        stream = torch.cuda.current_stream().cuda_stream
        assert lib.gated_rmsnorm_bwd(ctypes.byref(a), stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(up, want[place]) and torch.equal(dw, want["dweight"])
        assert torch.equal(other, want["dz" if place == "dx" else "dx"])


def test_parameters_as_weights():
    r = rnd(8)
    x, z = r(3, 64).requires_grad_(), r(3, 64)
    w, s = (torch.nn.Parameter(1 + 0.1 * r(64)) for _ in range(2))
    y, out = sss.add_rmsnorm_fn(x, z, w, scale=s)
    o = sss.gated_rmsnorm_fn(y, out, w)
    dx, dw, ds = torch.autograd.grad(o.sum(), (x, w, s))
    lx, lw, ls = (t.detach().to(F64).requires_grad_() for t in (x, w, s))
    total = lx * ls + z
    want = gated_rmsnorm(rmsnorm(total, lw, 1e-5), total, lw, 1e-5, 64, False).sum()
    for a, b in zip((dx, dw, ds), torch.autograd.grad(want, (lx, lw, ls))):
        assert worst(a, b) <= 4 * tol(64, F32, 3)


@pytest.mark.parametrize("upstream", ["constant", "differentiable"])
@pytest.mark.parametrize("op", ["gated", "add", "scan"])
def test_second_derivatives_are_refused(op, upstream):
    """create_graph gives the first derivative; differentiating that raises,
    beside a path that has a second one and whatever the upstream gradient."""
    r = rnd(3)
    x, z, w = r(4, 64).requires_grad_(), r(4, 64), torch.ones(64, device="cuda")
    if op == "scan":
        y = sss.selective_scan_fn(x[None], z[None], -torch.ones(4, 8, device="cuda"),
                                  r(1, 8, 64), r(1, 8, 64))[0]
    else:
        y = sss.gated_rmsnorm_fn(x, z, w) if op == "gated" else sss.add_rmsnorm_fn(x, z, w)[0]
    loss = (y * x if upstream == "differentiable" else y).sum() + (x ** 3).sum()
    first, = torch.autograd.grad(loss, x, create_graph=True)
    plain, = torch.autograd.grad((y * x.detach() if upstream == "differentiable" else y).sum(), x,
                                 retain_graph=True)
    extra = y if upstream == "differentiable" else torch.zeros_like(x)
    # three fp32 terms, added in either order: two roundings of a partial sum on
    # each side, and up to four of the product 3 x^2, half a step of the terms'
    # sizes each (the terms may cancel)
    sizes = plain.abs() + extra.abs() + 3 * x ** 2
    assert ((first - (plain + extra + 3 * x ** 2)).abs() <= 8 * U * sizes).all()
    with pytest.raises(RuntimeError, match="differentiated again"):
        torch.autograd.grad(first.sum(), x)
