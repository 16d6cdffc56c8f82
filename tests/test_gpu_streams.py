"""Calls of the scans on a stream of their own, beside another that uses the
same allocator (needs a GPU)."""
import pytest
import torch

import selective_state_space_48_b200 as sss

pytestmark = pytest.mark.gpu


def scan_inputs(batch=2, dim=64, L=300, N=16):
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(u=rnd(batch, dim, L), delta=rnd(batch, dim, L), A=-torch.exp(rnd(dim, N)),
                B=rnd(batch, N, L), C=rnd(batch, N, L)), rnd


def stream_calls():
    """Each operator's call, taking a stream, with the bytes of what it
    allocates and returns."""
    d, rnd = scan_inputs()
    size = 4 * d["u"].numel()
    dy, state = rnd(*d["u"].shape), rnd(2, 64, 16)
    bf = lambda *s: rnd(*s).to(torch.bfloat16)  # noqa: E731
    ssd = dict(x=bf(1, 256, 4, 64), dt=bf(1, 256, 4), A=-torch.rand(4, device="cuda"),
               B=bf(1, 256, 1, 128), C=bf(1, 256, 1, 128))

    def update(s):
        with torch.cuda.stream(s or torch.cuda.current_stream()):
            st = state.clone()  # (in that stream's order)
        return sss.selective_state_update(st, dy[..., 0].contiguous(), dy[..., 1].contiguous(),
                                          d["A"], d["B"][..., 0].contiguous(),
                                          d["C"][..., 0].contiguous(), stream=s)

    return {
        "scan": (lambda s: sss.selective_scan_fwd(**d, stream=s), size),
        "scan state": (lambda s: sss.selective_scan_fwd(**d, return_last_state=True, stream=s)[1],
                       4 * state.numel()),
        "scan bwd": (lambda s: sss.selective_scan_bwd(**d, dy=dy, stream=s)["du"], size),
        "ssd": (lambda s: sss.ssd_fwd(**ssd, stream=s), 4 * ssd["x"].numel()),
        "update": (update, 4 * 2 * 64),
    }


@pytest.mark.parametrize("name", ["scan", "scan state", "scan bwd", "ssd", "update"])
def test_streams_do_not_share_memory(name):
    """A call on a stream of its own allocates nothing that the current
    stream has freed and still uses, and what it still writes is not handed to
    the current stream when it is dropped."""
    call, nbytes = stream_calls()[name]
    want = call(None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((nbytes // 4,), 5.0, device="cuda") for _ in range(12)]
    torch.cuda._sleep(int(4e7))
    sums = [t.sum(dtype=torch.float64) for t in held]
    del held
    if name == "update":  # (its own small inputs are made on that stream too)
        with torch.cuda.stream(side):
            out = call(side)
    else:
        out = call(side)
    torch.cuda.synchronize()
    assert [float(v) for v in sums] == [5.0 * (nbytes // 4)] * 12
    assert torch.equal(out, want)
    del out
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(4e7))
    call(side)
    held = [torch.full((nbytes // 4,), 5.0, device="cuda") for _ in range(12)]
    torch.cuda.synchronize()
    assert all(bool((t == 5).all()) for t in held)


def test_a_stream_of_another_device_is_refused():
    d, _ = scan_inputs()

    class Elsewhere:
        device = torch.device("cuda", 7)

    with pytest.raises(ValueError):
        sss.selective_scan_fwd(**d, stream=Elsewhere())
