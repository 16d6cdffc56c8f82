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
import math

import pytest
import torch

import selective_state_space_48_b200 as sss
from delta_checks import delta_inputs, gated_delta, worst

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
