"""Gated delta rule against the recurrence in float64 (needs a GPU).

Tolerances, relative to the largest value.  Recurrent kernel: a step rounds
sums of up to dstate products and a few factors, at most (dstate + 16) half
steps of fp32 (2^-24); the transition never grows an error, and the steps'
errors have either sign, so they add up like the square root of the steps.
Chunked kernel: an operand that is the sum of two bf16 values is off by at
most 2^-18, and the product of the two low parts that is left out is below
2^-18, so a product is off by at most 2^-17 of its terms' size; a value
passes five such products in a chunk, and chunks add like the square root of
their number.  A bf16 output is off by another half step:
bf16 has 8 bits, so half a step is at most
2^-8 of the value.
"""
import ctypes
import math

import pytest
import torch

import selective_state_space_48_b200 as sss
from delta_checks import delta_inputs, gated_delta, gated_rmsnorm, worst

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
PLANS = {"recurrent": sss.MSS_DELTA_RECURRENT, "chunked": sss.MSS_DELTA_CHUNKED,
         "auto": sss.MSS_DELTA_AUTO}


def tolerance(N, L, out_dtype=F32, chunked=False):
    tol = (N + 16) * 2.0 ** -24 * math.sqrt(L)
    if chunked:
        tol += 5 * 2.0 ** -17 * math.sqrt(-(-L // 64))
    return tol + (2.0 ** -8 if out_dtype == BF else 0.0)


def check(d, plan="auto", out_dtype=F32, **kw):
    N, L = d["q"].shape[-1], d["q"].shape[1]
    y, last = sss.gated_delta_fwd(**d, return_last_state=True, out_dtype=out_dtype,
                                  plan=PLANS[plan], check_status=True, **kw)
    yr, lr = gated_delta(**d, **{n: v for n, v in kw.items() if n not in ("y", "last_state")})
    chunked = plan != "recurrent" and d["q"].dtype == BF
    if kw.get("cu_seqlens") is not None:
        inside = ~torch.isnan(yr)
        assert worst(y[inside], yr[inside]) <= tolerance(N, L, out_dtype, chunked)
    else:
        assert worst(y, yr) <= tolerance(N, L, out_dtype, chunked)
    assert worst(last, lr) <= tolerance(N, L, F32, chunked)
    return y, last


# batch, L, heads, headdim, groups, dstate
SIZES = [(1, 1, 1, 1, 1, 1), (2, 7, 3, 5, 1, 3), (1, 64, 2, 16, 2, 16), (2, 65, 4, 33, 2, 31),
         (1, 130, 6, 128, 3, 128), (3, 100, 2, 80, 1, 72), (1, 40, 2, 20, 2, 200),
         (1, 33, 1, 130, 1, 256)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("size", SIZES)
def test_recurrent(size, dtype):
    check(delta_inputs(*size, dtype, h0=size[1] != 64), "recurrent")


CHUNKED_SIZES = [(1, 64, 1, 128, 1, 128), (1, 1, 1, 128, 1, 128), (2, 63, 2, 64, 1, 64),
                 (1, 128, 2, 128, 1, 128), (1, 129, 4, 128, 2, 128), (2, 65, 3, 8, 3, 8),
                 (1, 200, 2, 24, 1, 40), (1, 333, 2, 136, 1, 96), (1, 70, 1, 264, 1, 72),
                 (3, 513, 4, 128, 4, 128), (1, 1025, 2, 120, 2, 128)]


@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("size", CHUNKED_SIZES)
def test_chunked(size, out_dtype):
    check(delta_inputs(*size, BF, seed=size[1], h0=size[1] % 2 == 1), "chunked", out_dtype)


def test_chunked_gates():
    """softplus and sigmoid off; strengths up to 2; hard decays (a block of
    32 steps that loses more than 2^64) beside none at all."""
    d = delta_inputs(1, 150, 4, 64, 2, 64, BF, h0=True, signed=True)
    d["dt_bias"] = None
    d["dt"] = (d["dt"].float().abs() * 0.05).to(BF)
    d["beta"] = (2 * torch.sigmoid(d["beta"].float())).to(BF)
    check(d, "chunked", dt_softplus=False, beta_sigmoid=False, scale=0.7)
    d["A"] = torch.tensor([0.0, -1.0, -300.0, -40.0], device="cuda")
    d["beta"] = (d["beta"].float() / 2).to(BF)
    check(d, "chunked", dt_softplus=False, beta_sigmoid=False)


def test_chunked_repeated_keys():
    """Every key the same, full strength, no decay: A is all ones below the
    diagonal, the state holds the last value only."""
    d = delta_inputs(1, 200, 2, 64, 1, 64, BF)
    d["k"] = torch.zeros_like(d["k"])
    d["k"][..., 3] = 1
    d["A"] = torch.zeros(2, device="cuda")
    d["beta"] = torch.ones_like(d["beta"])
    y, last = check(d, "chunked", beta_sigmoid=False)
    assert worst(last[0, :, :, 3], d["v"][0, -1].double()) <= tolerance(64, 200, F32, True)


def test_nothing_leaks_from_behind_a_sequence():
    """Values behind a sequence's end, NaN among them, do not reach it."""
    cu = torch.tensor([0, 70, 100], dtype=torch.int32, device="cuda")
    d = delta_inputs(1, 140, 2, 64, 1, 64, BF)
    want, wl = sss.gated_delta_fwd(**d, cu_seqlens=cu, return_last_state=True, plan=2)
    for n in ("q", "k", "v", "dt", "beta"):
        d[n][:, 100:] = float("nan")
    got, gl = sss.gated_delta_fwd(**d, cu_seqlens=cu, return_last_state=True, plan=2)
    assert torch.equal(got[:, :100], want[:, :100]) and torch.equal(gl, wl)
    for n in ("q", "k", "v", "dt", "beta"):
        d[n][:, 70:100] = float("nan")
    got, gl = sss.gated_delta_fwd(**d, cu_seqlens=cu, return_last_state=True, plan=2)
    assert torch.equal(got[:, :70], want[:, :70]) and torch.equal(gl[0], wl[0])


def test_chunked_refusals():
    d = delta_inputs(1, 70, 2, 64, 1, 64, F32)
    for bad in (d, delta_inputs(1, 70, 2, 64, 1, 60, BF), delta_inputs(1, 70, 2, 60, 1, 64, BF),
                delta_inputs(1, 70, 2, 64, 1, 136, BF)):
        with pytest.raises(sss.MssError) as e:
            sss.gated_delta_fwd(**bad, plan=sss.MSS_DELTA_CHUNKED)
        assert e.value.code == sss.MSS_ERR_UNSUPPORTED


@pytest.mark.parametrize("out_dtype", [F32, BF])
def test_recurrent_output_types(out_dtype):
    check(delta_inputs(2, 50, 4, 48, 2, 40, F32), "recurrent", out_dtype)
    check(delta_inputs(2, 50, 4, 48, 2, 40, BF), "recurrent", out_dtype)


def test_plain_gates_and_scale():
    """softplus and sigmoid off, no bias, another scale, strength above 1."""
    d = delta_inputs(2, 70, 4, 32, 2, 32, F32, h0=True)
    d["dt"] = d["dt"].abs() * 0.05
    d["beta"] = 2 * torch.sigmoid(d["beta"])
    d["dt_bias"] = None
    check(d, "recurrent", dt_softplus=False, beta_sigmoid=False, scale=0.7)


@pytest.mark.parametrize("batch,H,P,G,N,dtype", [
    (1, 2, 128, 1, 128, BF), (5, 9, 77, 3, 70, F32), (3, 4, 64, 4, 64, F32), (64, 4, 128, 2, 128, BF),
    (2, 3, 1, 1, 1, F32), (2, 2, 40, 2, 256, BF)])
def test_update(batch, H, P, G, N, dtype):
    d = delta_inputs(batch, 3, H, P, G, N, dtype, h0=True)
    state = d.pop("h0").clone()
    want = state.clone()
    for t in range(3):
        one = {n: (d[n][:, t] if n in ("q", "k", "v", "dt", "beta") else d[n]) for n in d}
        y = sss.gated_delta_update(state, **one)
        yr, want = gated_delta(**{n: (d[n][:, t:t + 1] if one[n] is not d[n] else d[n]) for n in d},
                               h0=want)
        assert worst(y, yr[:, 0]) <= tolerance(N, t + 1)
        assert worst(state, want) <= tolerance(N, t + 1)


def test_update_continues_a_prompt():
    """A prompt, then single tokens, equals the longer prompt."""
    d = delta_inputs(2, 140, 4, 64, 2, 64, BF)
    y, state = sss.gated_delta_fwd(**{n: (t[:, :137] if n in ("q", "k", "v", "dt", "beta") else t)
                                      for n, t in d.items()}, return_last_state=True)
    rows = [sss.gated_delta_update(state, **{n: (t[:, i] if n in ("q", "k", "v", "dt", "beta") else t)
                                             for n, t in d.items() if n != "h0"})
            for i in range(137, 140)]
    yr, lr = gated_delta(**d)
    tol = tolerance(64, 140, F32, True)
    assert worst(torch.cat([y, torch.stack(rows, 1)], 1), yr) <= tol
    assert worst(state, lr) <= tol


@pytest.mark.parametrize("plan,dtype", [("recurrent", F32), ("recurrent", BF), ("chunked", BF)])
def test_packed(plan, dtype):
    """Ragged sequences with an empty and a one-token one, and rows behind
    the last: those stay as they were."""
    cu = torch.tensor([0, 70, 70, 71, 135, 263, 290], dtype=torch.int32, device="cuda")
    d = delta_inputs(1, 300, 4, 64, 2, 64, dtype, h0=True, seqs=6)
    y = torch.full((1, 300, 4, 64), 7.0, device="cuda")
    check(d, plan, cu_seqlens=cu, y=y)
    assert (y[0, 290:] == 7.0).all()
    d["h0"] = None
    check(d, plan, cu_seqlens=cu)


def test_packed_offsets_outside_the_row_are_clamped():
    cu = torch.tensor([-5, 20, 10, 2000], dtype=torch.int32, device="cuda")
    d = delta_inputs(1, 40, 2, 16, 1, 16, F32, h0=True, seqs=3)
    y, last = sss.gated_delta_fwd(**d, cu_seqlens=cu, return_last_state=True)
    assert torch.isfinite(last).all()
    assert torch.equal(last[1], d["h0"][1])  # [20, 10) is empty


def test_views_of_a_projection():
    """q, k, v as slices of one wide tensor, dt and beta transposed, y a
    slice: same bits as dense copies."""
    d = delta_inputs(2, 40, 4, 24, 2, 20, F32)
    wide = torch.cat([d["q"].flatten(2), d["k"].flatten(2), d["v"].flatten(2)], -1)
    q, k, v = wide.split([40, 40, 96], -1)
    views = dict(d, q=q.unflatten(2, (2, 20)), k=k.unflatten(2, (2, 20)), v=v.unflatten(2, (4, 24)),
                 dt=d["dt"].transpose(1, 2).contiguous().transpose(1, 2),
                 beta=d["beta"].transpose(0, 1).contiguous().transpose(0, 1))
    want = sss.gated_delta_fwd(**d)
    buf = torch.zeros(2, 40, 4, 30, device="cuda")
    got = sss.gated_delta_fwd(**views, y=buf[..., :24])
    assert torch.equal(got, want)
    assert (buf[..., 24:] == 0).all()


def test_state_in_place_other_stream_and_graph():
    d = delta_inputs(2, 80, 4, 64, 2, 64, BF, h0=True)
    want_y, want = sss.gated_delta_fwd(**d, return_last_state=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    state = d["h0"].clone()
    side.wait_stream(torch.cuda.current_stream())
    y, _ = sss.gated_delta_fwd(**dict(d, h0=state), last_state=state, return_last_state=True,
                               stream=side)
    side.synchronize()
    assert torch.equal(state, want) and torch.equal(y, want_y)
    state = d["h0"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = sss.gated_delta_fwd(**dict(d, h0=state), last_state=state, return_last_state=True)
    state.copy_(d["h0"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(state, want) and torch.equal(y, want_y)


def projection(batch, L, H, P, G, N, seed=0):
    """q, k, v as slices of one wide bf16 projection, and the same dense."""
    d = delta_inputs(batch, L, H, P, G, N, BF, seed=seed, h0=True)
    parts = [d[n].flatten(2) for n in ("q", "k", "v")]
    wide = torch.cat([parts[0], torch.zeros_like(parts[0][..., :8]), *parts[1:]], -1)
    q, _, k, v = wide.split([G * N, 8, G * N, H * P], -1)
    views = dict(d, q=q.unflatten(2, (G, N)), k=k.unflatten(2, (G, N)), v=v.unflatten(2, (H, P)))
    return d, views


@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_chunked_views_of_a_projection(out_dtype, shift):
    """Strided q, k, v and a strided y, whose rows start on 16 bytes (they
    leave through tensor maps in bf16) or do not: the bits of dense copies,
    and nothing written beside y."""
    d, views = projection(2, 150, 4, 64, 2, 64)
    want, wl = sss.gated_delta_fwd(**d, return_last_state=True, out_dtype=out_dtype, plan=2)
    buf = torch.full((2, 150, 4, 80), 7.0, device="cuda", dtype=out_dtype)
    y = buf[..., shift:shift + 64]
    got, gl = sss.gated_delta_fwd(**views, return_last_state=True, y=y, plan=2)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    assert (buf[..., :shift] == 7).all() and (buf[..., shift + 64:] == 7).all()


@pytest.mark.parametrize("headdim", [64, 72, 136, 192])
def test_chunked_packed_bf16_rows(headdim):
    """Rows behind the last sequence stay as they were, bf16 y included, for
    widths that fill their 64-wide and 128-wide tiles or do not."""
    cu = torch.tensor([0, 64, 64, 65, 200, 328, 330], dtype=torch.int32, device="cuda")
    d = delta_inputs(1, 340, 2, headdim, 1, 64, BF, h0=True, seqs=6)
    y = torch.full((1, 340, 2, headdim), 7.0, device="cuda", dtype=BF)
    check(d, "chunked", BF, cu_seqlens=cu, y=y)
    assert (y[0, 330:] == 7.0).all()


@pytest.mark.parametrize("seqs", [7, 890, 1000])
def test_chunked_many_sequences(seqs):
    """Sequences are taken longest first up to a number of them and in their
    own order beyond: every one is done, equal lengths among them."""
    lens = torch.tensor([(i * 7) % 5 for i in range(seqs)])
    lens[seqs // 2] = 130
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]).to(torch.int32).cuda()
    d = delta_inputs(1, int(cu[-1]), 2, 64, 1, 64, BF, h0=True, seqs=seqs)
    y, last = sss.gated_delta_fwd(**d, cu_seqlens=cu, return_last_state=True, plan=2)
    yr, lr = sss.gated_delta_fwd(**d, cu_seqlens=cu, return_last_state=True, plan=1)
    assert worst(y, yr) <= tolerance(64, 130, F32, True) + tolerance(64, 130)
    assert worst(last, lr) <= tolerance(64, 130, F32, True) + tolerance(64, 130)


@pytest.mark.parametrize("n", ["q", "k", "v", "dt", "beta"])
def test_non_finite_steps_stay_in_their_head_and_chunk(n):
    """A NaN in a step of a head reaches that head's rows from the start of
    its 64-step chunk on (chunked) or from its step on (recurrent), and
    nothing else."""
    d = delta_inputs(2, 200, 4, 64, 4, 64, BF)
    want = {p: sss.gated_delta_fwd(**d, plan=p) for p in (1, 2)}
    d[n][1, 100, 2] = float("nan")
    for plan, first in ((1, 100), (2, 64)):
        y = sss.gated_delta_fwd(**d, plan=plan)
        assert torch.isnan(y[1, 100, 2]).any()
        same = torch.ones(2, 200, 4, dtype=torch.bool, device="cuda")
        same[1, first:, 2] = False
        assert torch.equal(y[same], want[plan][same])


def test_plan_follows_the_length():
    for L, plan in ((31, 1), (32, 2)):
        d = delta_inputs(2, L, 2, 64, 1, 64, BF)
        assert torch.equal(sss.gated_delta_fwd(**d), sss.gated_delta_fwd(**d, plan=plan))
    d = delta_inputs(1, 64, 2, 64, 1, 64, BF, seqs=4)
    cu = torch.tensor([0, 61, 62, 63, 64], dtype=torch.int32, device="cuda")  # 16 on average
    kw = dict(cu_seqlens=cu)
    assert torch.equal(sss.gated_delta_fwd(**d, **kw), sss.gated_delta_fwd(**d, plan=1, **kw))


@pytest.mark.parametrize("plan", [1, 2])
def test_two_calls_at_once_and_two_graphs(plan):
    """Calls on two streams at the same time, then two graphs of the same
    tensors, replayed twice: the bits of a call alone."""
    d = [delta_inputs(4, 150, 8, 64, 2, 64, BF, seed=s, h0=True) for s in (1, 2)]
    want = [sss.gated_delta_fwd(**x, return_last_state=True, plan=plan) for x in d]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in d]
    for _ in range(5):
        got = [sss.gated_delta_fwd(**x, return_last_state=True, plan=plan, stream=s)
               for x, s in zip(d, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    graphs, outs = [], []
    for x in d:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(sss.gated_delta_fwd(**x, return_last_state=True, plan=plan))
        graphs.append(graph)
    for graph in graphs * 2:
        graph.replay()
    torch.cuda.synchronize()
    for g, w in zip(outs, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_layer():
    """The operators as a layer uses them: the norm with the residual sum, a
    projection whose slices go into the delta rule in place, the gated norm
    per head; a prompt, then single tokens from its state.  Every stage is
    compared with float64 of what entered it."""
    B, L, H, P, G, N, D = 2, 70, 4, 64, 2, 64, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    widths = [G * N, G * N, H * P, H * P, H, H]
    w_in = (rnd(D, sum(widths)) / 16).to(BF)
    w1, w2, scale = 1 + 0.1 * rnd(D), 1 + 0.1 * rnd(P), 0.5 + 0.1 * rnd(D)
    A, bias = -1 - 15 * torch.rand(H, generator=g, device="cuda"), rnd(H) - 4
    state = torch.zeros(B, H, P, N, device="cuda")
    want_state = state.double()
    unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).to(BF)  # noqa: E731
    for steps in (L, 1, 1):
        x, res = rnd(B, steps, D).to(BF), rnd(B, steps, D)
        h, total = sss.add_rmsnorm_fwd(x, res, w1, scale=scale)
        want = x.double() * scale + res
        assert worst(total, want) <= 2.0 ** -23
        want = total.double() / torch.sqrt(total.double().pow(2).mean(-1, keepdim=True) + 1e-5)
        assert worst(h, want * w1) <= 2.0 ** -8 + 64 * 2.0 ** -24
        wide = h @ w_in
        wide[..., :2 * G * N] = unit(wide[..., :2 * G * N].unflatten(-1, (-1, N))).flatten(-2)
        q, k, v, z, dt, beta = wide.split(widths, -1)
        q, k, v = (q.unflatten(-1, (G, N)), k.unflatten(-1, (G, N)), v.unflatten(-1, (H, P)))
        if steps > 1:
            y, _ = sss.gated_delta_fwd(q, k, v, dt, A, beta, bias, h0=state, last_state=state,
                                       return_last_state=True, out_dtype=BF, check_status=True)
        else:
            y = sss.gated_delta_update(state, q[:, 0], k[:, 0], v[:, 0], dt[:, 0], A, beta[:, 0],
                                       bias, out_dtype=BF)[:, None]
        yr, want_state = gated_delta(q, k, v, dt, A, beta, bias, h0=want_state)
        assert worst(y, yr) <= tolerance(N, L + 2, BF, True)
        assert worst(state, want_state) <= tolerance(N, L + 2, F32, True)
        o = sss.gated_rmsnorm_fwd(y.flatten(-2), z, w2, group_size=P)
        want = gated_rmsnorm(y.flatten(-2).double(), z.double(), w2.double(), 1e-5, P, False)
        assert worst(o, want) <= 2.0 ** -8 + 64 * 2.0 ** -24


def call(a):
    """The call of filled arguments, without the binding's own workspace."""
    stream = torch.cuda.current_stream().cuda_stream
    return sss.load_library().gated_delta_fwd(ctypes.byref(a), stream)


def workspace_bytes(a):
    n = ctypes.c_size_t(0)
    assert sss.load_library().mss_gated_delta_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("size,h0", [
    ((1, 1500, 1, 128, 1, 128), True), ((2, 1001, 3, 136, 1, 96), False),
    ((1, 2048, 2, 64, 1, 64), True), ((1, 1217, 4, 72, 2, 40), True),
    ((1, 1100, 1, 264, 1, 8), False), ((2, 2001, 3, 136, 1, 96), True),
    ((1, 1700, 1, 264, 1, 8), True)])
def test_segments(size, h0, out_dtype):
    """Long sequences of few heads are cut into segments that run beside each
    other: the float64 recurrence's values, every time the same bits.  (The
    transition of a segment is a chunked state of its own, so a start off by
    twice a chunked state's error joins the segment's.)"""
    B, L, H, P, G, N = size
    d = delta_inputs(*size, BF, seed=L, h0=h0)
    y = torch.empty(B, L, H, P, device="cuda", dtype=out_dtype)
    last = torch.empty(B, H, P, N, device="cuda")
    got, gl = sss.gated_delta_fwd(**d, return_last_state=True, y=y, check_status=True)
    yr, lr = gated_delta(**d)
    extra = 3 * tolerance(N, L, F32, True)
    assert worst(got, yr) <= extra + (2.0 ** -8 if out_dtype == BF else 0)
    assert worst(gl, lr) <= extra
    for _ in range(3):
        again, al = sss.gated_delta_fwd(**d, return_last_state=True, out_dtype=out_dtype)
        assert torch.equal(again, got) and torch.equal(al, gl)
    # whole sequences, without a workspace
    whole = sss.make_gated_delta_args(**d, y=torch.empty_like(y), last_state=last)
    assert call(whole) == sss.MSS_OK
    torch.cuda.synchronize()
    assert worst(gl, last.double()) <= extra


def test_segments_follow_the_sizes():
    """Long sequences of few heads ask for a workspace; short ones, those that
    fill the machine, packed ones and the recurrent plan do not."""
    def size(B, L, H, dtype=BF, **kw):
        d = delta_inputs(B, L, H, 64, 1, 64, dtype)
        return workspace_bytes(sss.make_gated_delta_args(**d, **kw))
    assert size(1, 1500, 1) > 0 and size(2, 2001, 3) > 0 and size(1, 1217, 4) > 0
    cu = torch.tensor([0, 2000], dtype=torch.int32, device="cuda")
    assert size(1, 500, 1) == size(1, 2000, 160) == size(1, 2000, 2, cu_seqlens=cu) == 0
    assert size(1, 2000, 2, plan=1) == size(1, 2000, 2, F32) == 0


def test_segments_in_place_and_workspace_errors():
    d = delta_inputs(1, 1500, 2, 64, 1, 64, BF, h0=True)
    want, wl = sss.gated_delta_fwd(**d, return_last_state=True)
    state = d["h0"].clone()
    got, _ = sss.gated_delta_fwd(**dict(d, h0=state), last_state=state, return_last_state=True)
    assert torch.equal(got, want) and torch.equal(state, wl)
    y = torch.full_like(want, 7.0)
    a = sss.make_gated_delta_args(**d, y=y)
    n = workspace_bytes(a)
    ws = torch.full((n + 64,), 171, dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = ws.data_ptr(), n - 1
    assert call(a) == sss.MSS_ERR_WORKSPACE
    a.workspace, a.workspace_bytes = ws.data_ptr() + 8, n
    assert call(a) == sss.MSS_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (y == 7).all()
    a.workspace = ws.data_ptr()
    assert call(a) == sss.MSS_OK
    torch.cuda.synchronize()
    assert torch.equal(y, want) and (ws[n:] == 171).all()


def test_segments_on_another_stream_and_in_graphs():
    d = [delta_inputs(1, 1300, 2, 64, 1, 64, BF, seed=s, h0=True) for s in (1, 2)]
    want = [sss.gated_delta_fwd(**x, return_last_state=True) for x in d]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in d]
    for _ in range(5):
        got = [sss.gated_delta_fwd(**x, return_last_state=True, stream=s)
               for x, s in zip(d, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    graphs, outs = [], []
    for x in d:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(sss.gated_delta_fwd(**x, return_last_state=True))
        graphs.append(graph)
    for graph in graphs * 2:
        graph.replay()
    torch.cuda.synchronize()
    for g, w in zip(outs, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


# batch, L, heads, headdim, groups, dstate that no tensor map takes as they lie
ODD_SIZES = [(2, 130, 3, 33, 1, 31), (1, 64, 2, 20, 2, 20), (3, 300, 4, 77, 2, 70),
             (1, 1500, 1, 100, 1, 36), (1, 1700, 2, 129, 1, 127), (2, 200, 2, 1, 1, 1)]


@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("size", ODD_SIZES)
def test_copied_sizes(size, out_dtype):
    """Odd sizes in bf16 are copied into rows that the chunked evaluation
    takes, states of odd rows among them."""
    d = delta_inputs(*size, BF, seed=size[1], h0=size[0] != 2)
    N, L = size[5], size[1]
    assert workspace_bytes(sss.make_gated_delta_args(**d, y=torch.empty_like(d["v"]))) > 0
    y, last = sss.gated_delta_fwd(**d, return_last_state=True, out_dtype=out_dtype,
                                  check_status=True)
    yr, lr = gated_delta(**d)
    tol = 3 * tolerance(N, L, F32, True)  # (as for segments)
    assert worst(y, yr) <= tol + (2.0 ** -8 if out_dtype == BF else 0.0)
    assert worst(last, lr) <= tol
    again, al = sss.gated_delta_fwd(**d, return_last_state=True, out_dtype=out_dtype)
    assert torch.equal(again, y) and torch.equal(al, last)


def test_copied_packed_rows_and_views():
    """Packed odd sizes with rows behind the last sequence; q, k, v as odd
    slices of one projection, y a slice at an odd place."""
    cu = torch.tensor([0, 70, 70, 71, 200, 328], dtype=torch.int32, device="cuda")
    d = delta_inputs(1, 340, 2, 45, 1, 50, BF, h0=True, seqs=5)
    for n in ("q", "k", "v", "dt", "beta"):
        d[n][:, 328:] = float("nan")
    y = torch.full((1, 340, 2, 45), 7.0, device="cuda", dtype=BF)
    y, last = sss.gated_delta_fwd(**d, cu_seqlens=cu, return_last_state=True, y=y)
    yr, lr = gated_delta(**d, cu_seqlens=cu)
    assert worst(y[0, :328], yr[0, :328]) <= tolerance(50, 130, BF, True)
    assert worst(last, lr) <= tolerance(50, 130, F32, True)
    assert (y[0, 328:] == 7).all()
    d = delta_inputs(2, 150, 4, 30, 2, 25, BF, h0=True)
    want, wl = sss.gated_delta_fwd(**d, return_last_state=True, out_dtype=BF)
    wide = torch.cat([d[n].flatten(2) for n in ("q", "k", "v")], -1)
    q, k, v = wide.split([50, 50, 120], -1)
    views = dict(d, q=q.unflatten(2, (2, 25)), k=k.unflatten(2, (2, 25)), v=v.unflatten(2, (4, 30)))
    buf = torch.full((2, 150, 4, 33), 7.0, device="cuda", dtype=BF)
    got, gl = sss.gated_delta_fwd(**views, return_last_state=True, y=buf[..., 1:31])
    assert torch.equal(got, want) and torch.equal(gl, wl)
    assert (buf[..., :1] == 7).all() and (buf[..., 31:] == 7).all()
    # rows of y on 16 bytes, their width not: nothing written beside it
    for width in (30, 25):
        buf = torch.full((2, 150, 4, 40), 7.0, device="cuda", dtype=BF)
        got, _ = sss.gated_delta_fwd(**dict(d, v=d["v"][..., :width], h0=None),
                                     return_last_state=True, y=buf[..., :width])
        want, _ = sss.gated_delta_fwd(**dict(d, v=d["v"][..., :width], h0=None),
                                      return_last_state=True, out_dtype=BF)
        assert torch.equal(got, want) and (buf[..., width:] == 7).all()


def test_copies_keep_inside_their_workspace():
    d = delta_inputs(1, 100, 2, 33, 1, 31, BF)
    want = sss.gated_delta_fwd(**d)
    y = torch.full_like(want, 7.0)
    a = sss.make_gated_delta_args(**d, y=y)
    n = workspace_bytes(a)
    ws = torch.full((n + 64,), 171, dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = ws.data_ptr(), n - 1
    assert call(a) == sss.MSS_ERR_WORKSPACE
    a.workspace_bytes = n
    assert call(a) == sss.MSS_OK
    torch.cuda.synchronize()
    assert torch.equal(y, want) and (ws[n:] == 171).all()


def test_even_sizes_at_odd_places():
    """Sizes that the chunked evaluation takes, in views and states whose
    addresses or strides it does not: the same values."""
    d = delta_inputs(1, 1500, 1, 64, 1, 64, BF, h0=True)
    want, wl = sss.gated_delta_fwd(**d, return_last_state=True)
    tol = 6 * tolerance(64, 1500, F32, True)  # (two evaluations)
    shifted = dict(d)
    for n in ("q", "k", "v"):
        buf = torch.zeros(d[n].numel() + 3, device="cuda", dtype=BF)
        buf[3:] = d[n].flatten()
        shifted[n] = buf[3:].view_as(d[n])
    state = torch.zeros(64 * 64 + 1, device="cuda")
    state[1:] = d["h0"].flatten()
    state = state[1:].view_as(d["h0"])
    wide = torch.zeros(1, 1500, 1, 67, device="cuda", dtype=BF)
    wide[..., 1:65] = d["v"]
    for odd in (shifted, dict(d, h0=state), dict(d, v=wide[..., 1:65]),
                dict(d, k=d["k"].expand(1, 1500, 1, 64), v=wide[..., 1:65], h0=state)):
        y, last = sss.gated_delta_fwd(**odd, return_last_state=True)
        assert worst(y, want.double()) <= tol and worst(last, wl.double()) <= tol
    y, _ = sss.gated_delta_fwd(**dict(d, h0=state), last_state=state, return_last_state=True)
    assert worst(y, want.double()) <= tol and worst(state, wl.double()) <= tol


def resets(L, every, size):
    """Steps of weak decays (a factor of 0.95 to 1) with a hard one, whose
    log2 is -size, now and then: dt for A = -1 without softplus, and where the
    hard ones are."""
    g = torch.Generator(device="cuda").manual_seed(L)
    dt = 0.05 * torch.rand(L, generator=g, device="cuda")
    at = torch.arange(every // 2, L, every, device="cuda")
    dt[at] = size * math.log(2)
    return dt.to(BF), at.tolist()


@pytest.mark.parametrize("size", [46.0, 461.0, 2300.0, 2.3e5, 2.3e6, 1e9, 1e38, math.inf])
@pytest.mark.parametrize("plan,L,every", [("recurrent", 128, 41), ("chunked", 128, 41),
                                          ("chunked", 192, 7), ("auto", 1536, 111)])
def test_weak_decays_after_a_hard_one(plan, L, every, size):
    """A step that wipes the state (its decay is 0 in fp32 from log2 -150 on)
    takes nothing from the precision of the decays after it, nor does one that
    leaves next to nothing.  Every stretch between two of them and every head
    is measured by its own largest value.  A running sum of log2 decays is off
    by at most 2^-24 of the weak part and of what the sum's low word leaves,
    2^-47 of 64 * 300: inside the (dstate + 16) half steps of fp32 that the
    tolerance counts.  (auto: segments, as for those.)"""
    d = delta_inputs(1, L, 2, 64, 1, 64, BF, h0=True)
    dt, at = resets(L, every, size)
    d["dt"] = dt[None, :, None].expand(1, L, 2)
    d["A"], d["dt_bias"] = torch.tensor([-1.0, -0.75], device="cuda"), None
    y, last = sss.gated_delta_fwd(**d, dt_softplus=False, plan=PLANS[plan],
                                  return_last_state=True, check_status=True)
    yr, lr = gated_delta(**d, dt_softplus=False)
    tol = (3 if plan == "auto" else 1) * tolerance(64, L, F32, plan != "recurrent")
    for h in range(2):
        for lo, hi in zip([0] + at, at + [L]):
            assert worst(y[0, lo:hi, h], yr[0, lo:hi, h]) <= tol, (h, lo)
        assert worst(last[0, h], lr[0, h]) <= tol


@pytest.mark.parametrize("chunks", [0, 1, 2, 3, 4])
def test_tails_with_every_sm_busy(chunks):
    """Last chunks of every length behind 0 to 4 whole ones, NaN behind each
    sequence, more blocks than SMs and a copy beside them that keeps the memory
    busy: what the tail clears of K and V is that chunk's own, so the bits are
    those of the same rows with zeros behind them, in every run."""
    tails = [1, 2, 15, 16, 17, 31, 32, 33, 48, 49, 62, 63]
    lens = [64 * chunks + t for t in tails for _ in range(2)]
    starts, at = [], 0
    for n in lens:  # (in whole rows of 8 steps, some behind each)
        starts += [at, at + n]
        at += n + 8
    cu = torch.tensor(starts + [at], dtype=torch.int32, device="cuda")
    seqs = len(cu) - 1  # every other one is the rows behind a sequence
    d = delta_inputs(1, at, 32, 128, 8, 128, BF, seed=chunks, h0=True, seqs=seqs)
    keep = torch.zeros(at, dtype=torch.bool, device="cuda")
    for lo, hi in zip(starts[::2], starts[1::2]):
        keep[lo:hi] = True
    def run(fill):
        for n in ("q", "k", "v", "dt", "beta"):
            d[n][:, ~keep] = fill
        return sss.gated_delta_fwd(**d, cu_seqlens=cu, return_last_state=True, plan=2,
                                   check_status=True)
    want, wl = run(0.0)
    big, other = torch.empty(2, 1 << 27, device="cuda"), torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(other):
            for _ in range(4):
                big[1].copy_(big[0])
        y, last = run(float("nan"))
        assert torch.equal(y[:, keep], want[:, keep])
        assert torch.equal(last[::2], wl[::2])
    other.synchronize()


def test_packed_calls_one_behind_the_other():
    """Ragged packs of more blocks than SMs, hundreds of calls that nothing
    waits between: none of their waits runs out, and the last call's bits are
    the first's."""
    cu = torch.tensor([0, 700, 700, 1362, 1363, 1500, 1890, 1999, 2600, 2663, 2999],
                      dtype=torch.int32, device="cuda")
    d = delta_inputs(1, 3002, 32, 128, 16, 128, BF, h0=True, seqs=10)
    y = torch.zeros(1, 3002, 32, 128, device="cuda", dtype=BF)
    last = torch.empty(10, 32, 128, 128, device="cuda")
    kw = dict(cu_seqlens=cu, return_last_state=True, plan=2)
    want, wl = (t.clone() for t in sss.gated_delta_fwd(**d, **kw, y=y, last_state=last,
                                                       check_status=True))
    for _ in range(600):
        sss.gated_delta_fwd(**d, **kw, y=y, last_state=last)
    assert sss.gated_delta_status() == sss.MSS_OK
    assert torch.equal(y, want) and torch.equal(last, wl)


@pytest.mark.parametrize("size,cu,out_dtype", [
    ((1, 192, 2, 128, 1, 128), None, BF), ((4, 130, 32, 128, 8, 128), None, F32),
    ((1, 2048, 1, 64, 1, 64), None, BF), ((1, 300, 4, 100, 2, 60), None, BF),
    ((1, 264, 8, 64, 2, 64), [0, 70, 70, 71, 200, 264], BF)])
def test_a_wait_that_runs_out_is_reported(size, cu, out_dtype):
    """Waits of a microsecond (a chunk's inverse alone takes several) end the
    call with a status, once, whatever it computes: whole sequences, segments,
    copies, packed ones.  The calls after it are as before."""
    seqs = None if cu is None else len(cu) - 1
    cu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    d = delta_inputs(*size, BF, h0=True, seqs=seqs)
    kw = dict(cu_seqlens=cu, out_dtype=out_dtype, return_last_state=True)
    want, wl = sss.gated_delta_fwd(**d, **kw, check_status=True)
    y = torch.empty_like(want)
    a = sss.make_gated_delta_args(**d, y=y, cu_seqlens=cu, spin_timeout_ns=1)
    ws = torch.empty(max(workspace_bytes(a), 16), dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
    for _ in range(3):
        assert call(a) == sss.MSS_OK
        assert sss.gated_delta_status() == sss.MSS_ERR_TIMEOUT
        assert sss.gated_delta_status() == sss.MSS_OK
    got, gl = sss.gated_delta_fwd(**d, **kw, check_status=True)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    a.spin_timeout_ns = 10 ** 18  # (above what the kernel counts to)
    assert call(a) == sss.MSS_OK
    assert sss.gated_delta_status() == sss.MSS_OK
    assert torch.equal(y, want)


@pytest.mark.parametrize("size", ODD_SIZES + [(2, 100, 2, 57, 1, 121)])
def test_copies_read_nothing_behind_their_rows(size):
    """A workspace full of NaN gives the bits of one full of zeros, and the
    copies' rows end in zeros."""
    B, L, H, P, G, N = size
    d = delta_inputs(*size, BF, h0=True)
    y, last = torch.empty_like(d["v"]), torch.empty(B, H, P, N, device="cuda")
    a = sss.make_gated_delta_args(**d, y=y, last_state=last)
    n = workspace_bytes(a)
    got = []
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        a.workspace, a.workspace_bytes = ws.data_ptr(), n
        assert call(a) == sss.MSS_OK
        assert sss.gated_delta_status() == sss.MSS_OK
        got.append((y.clone(), last.clone()))
        width, pitch = (N, -(-N // 8) * 8)
        rows = ws[:2 * B * L * G * pitch].view(BF).view(-1, pitch)
        assert torch.equal(rows[:, :width], d["q"].reshape(-1, N))
        assert (rows[:, width:] == 0).all()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def delayed(stream, ms=20):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(ms * 2e6))


def stream_calls():
    """Calls of every operator (taking a stream) with the bytes of what each
    allocates."""
    d = delta_inputs(2, 100, 4, 64, 2, 64, BF, h0=True)
    seg = delta_inputs(1, 1500, 2, 64, 1, 64, BF)
    ws = workspace_bytes(sss.make_gated_delta_args(**seg))
    one = {n: (t[:, 0] if n in ("q", "k", "v", "dt", "beta") else t)
           for n, t in d.items() if n != "h0"}
    x, z = torch.randn(2, 64, 512, device="cuda")
    w = torch.ones(512, device="cuda")
    y = torch.empty(1, 1500, 2, 64, device="cuda")
    size = 4 * x.numel()

    def update(s):
        with torch.cuda.stream(s or torch.cuda.current_stream()):
            state = d["h0"].clone()  # (in that stream's order)
        return sss.gated_delta_update(state, **one, stream=s)

    return {
        "fwd": (lambda s: sss.gated_delta_fwd(**d, stream=s), 4 * d["v"].numel()),
        "fwd state": (lambda s: sss.gated_delta_fwd(**d, return_last_state=True, stream=s)[1],
                      4 * d["h0"].numel()),
        "workspace": (lambda s: sss.gated_delta_fwd(**seg, y=y, stream=s), ws),
        "update": (update, 4 * one["v"].numel()),
        "gated": (lambda s: sss.gated_rmsnorm_fwd(x, z, w, stream=s), size),
        "gated bwd": (lambda s: sss.gated_rmsnorm_bwd(x, z, w, z, stream=s)["dz"], size),
        "add": (lambda s: sss.add_rmsnorm_fwd(x, z, w, stream=s)[0], size),
        "add bwd": (lambda s: sss.add_rmsnorm_bwd(x, w, z, stream=s)["dx"], size),
    }


@pytest.mark.parametrize("name", ["fwd", "fwd state", "workspace", "update", "gated", "gated bwd",
                                  "add", "add bwd"])
def test_streams_do_not_share_memory(name):
    """A call on a stream of its own allocates nothing that the current
    stream has freed and still uses, and what it still writes is not handed to
    the current stream when it is dropped."""
    call, nbytes = stream_calls()[name]
    want = call(None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of that size, freed while the current stream has yet to read them
    held = [torch.full((nbytes // 4,), 5.0, device="cuda") for _ in range(8)]
    delayed(torch.cuda.current_stream())
    sums = [t.sum(dtype=torch.float64) for t in held]
    del held
    out = call(side)
    torch.cuda.synchronize()
    assert [float(v) for v in sums] == [5.0 * (nbytes // 4)] * 8
    assert torch.equal(out, want)
    del out
    # dropped while that stream has yet to write it
    delayed(side)
    call(side)
    held = [torch.full((nbytes // 4,), 5.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert all(bool((t == 5).all()) for t in held)


@pytest.mark.parametrize("n", ["q", "k", "v", "dt", "A", "beta", "dt_bias", "h0"])
def test_inputs_that_require_gradients_are_refused(n):
    """The delta rule is forward only: no call returns values without the
    graph that a gradient would need.  Under no_grad, and detached, it runs."""
    d = delta_inputs(1, 70, 2, 64, 1, 64, F32, h0=True)
    want = sss.gated_delta_fwd(**d)
    d[n] = d[n].clone().requires_grad_()
    one = {m: (t[:, 0] if m in ("q", "k", "v", "dt", "beta") else t) for m, t in d.items()}
    state = one.pop("h0")
    with pytest.raises(RuntimeError, match="forward only"):
        sss.gated_delta_fwd(**d)
    with pytest.raises(RuntimeError, match="forward only"):
        sss.gated_delta_update(state, **one)
    with torch.no_grad():
        assert torch.equal(sss.gated_delta_fwd(**d), want)
        assert torch.isfinite(sss.gated_delta_update(state, **one)).all()


@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("plan", ["recurrent", "chunked"])
def test_one_chunk_of_unit_keys_keeps_fp32(plan, out_dtype):
    """64 different unit vectors as keys, the queries the same ones, no decay:
    column t of the state is b_t v_t and y_t = scale b_t v_t, one term each, so
    every value can be held to fp32 by itself.  In half steps (2^-24) of the
    value: b about 10 (the argument's and the sum's rounding, an exponential
    good to 3, a quotient good to 4), b v 1, and two products' sums of three
    pieces, each a truncation (2) of a whole: 24; y: six more, and two for the
    scale: 38.  (b v in two bf16 pieces would be up to 64 off, b as well.)"""
    P = 128
    d = delta_inputs(1, 64, 2, P, 1, 64, BF, seed=11)
    d["q"] = d["k"] = torch.eye(64, device="cuda", dtype=BF).view(1, 64, 1, 64)
    d["A"] = torch.zeros(2, device="cuda")
    y, last = sss.gated_delta_fwd(**d, scale=0.1, return_last_state=True, out_dtype=out_dtype,
                                  plan=PLANS[plan], check_status=True)
    u = torch.sigmoid(d["beta"].double())[..., None] * d["v"].double()  # (1, 64, 2, P)
    want = u[0].permute(1, 2, 0)  # heads, rows, columns
    assert ((last[0] - want).abs() <= 24 * 2.0 ** -24 * want.abs()).all()
    half = 38 * 2.0 ** -24 + (2.0 ** -8 if out_dtype == BF else 0)
    scaled = float(torch.tensor(0.1)) * u
    assert ((y.double() - scaled).abs() <= half * scaled.abs()).all()


def test_a_forked_stream_in_a_captured_graph():
    """A graph whose captured stream forks into another, on which the calls
    run (with a workspace, and with gradients' partial sums), replayed: the
    bits of calls alone."""
    d = delta_inputs(1, 1500, 2, 64, 1, 64, BF, h0=True)
    x, z = torch.randn(2, 64, 512, device="cuda")
    w = torch.ones(512, device="cuda")
    want = sss.gated_delta_fwd(**d, return_last_state=True)
    grads = sss.gated_rmsnorm_bwd(x, z, w, z)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = sss.gated_delta_fwd(**d, return_last_state=True, stream=side)
        g = sss.gated_rmsnorm_bwd(x, z, w, z, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in (*got, *g.values()):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(g[n], grads[n]) for n in grads)
    assert sss.gated_delta_status() == sss.MSS_OK
