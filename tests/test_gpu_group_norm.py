"""GPU parity of the group norm with 64 bits, within ssm_ref.norm's bound."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def draw(rows, channels, size, seed, gate, shared, bias, fp32):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, channels, generator=g) * torch.exp(torch.randn(rows, 1, generator=g)) + 0.3).to(BF)
    z = torch.randn(rows, channels, generator=g).to(BF) if gate != "none" else None
    n = size if shared else channels
    w = (1 + 0.2 * torch.randn(n, generator=g)).to(torch.float32 if fp32 else BF)
    b = (0.2 * torch.randn(n, generator=g)).to(torch.float32 if fp32 else BF) if bias else None
    return x, z, w, b


def run(rows, channels, size, seed=0, gate="last", kind="rms", activation="silu", shared=False, bias=False, fp32=False,
        eps=1e-5, weight=True, edit=None, place=lambda t: t.to(DEV), out=None):
    x, z, w, b = draw(rows, channels, size, seed, gate, shared, bias, fp32)
    if not weight:
        w = None
    if edit:
        edit(x, z)
    want, tol = R.norm(x, size, w, b, z, eps, kind, activation, gate == "first")
    put = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    gx, gz = place(x), None if z is None else place(z)
    o = {None: None, "x": gx, "z": gz, "new": place(torch.zeros_like(x))}[out]
    got = S.sconv_group_norm(gx, size, weight=put(w), bias=put(b), z=gz, eps=eps, norm=kind, activation=activation,
                             gate_first=gate == "first", out=o)
    assert o is None or got is o
    R.check(got, want, tol, f"norm {rows} x {channels} by {size}")


@pytest.mark.parametrize("size", [1, 2, 7, 8, 16, 24, 64, 80, 100, 128, 129, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096,
                                  5000, 8192, 8200, 16384, 16392, 40001])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_sizes(size, kind):
    run(5, size * (3 if size < 4096 else 1), size, seed=size, kind=kind)


@pytest.mark.parametrize("gate", ["first", "last", "none"])
@pytest.mark.parametrize("activation", ["silu", "sigmoid", None])
@pytest.mark.parametrize("shared,bias,fp32", [(True, False, False), (False, True, False), (True, True, True), (False, False, True)])
def test_options(gate, activation, shared, bias, fp32):
    run(9, 512, 128, seed=3, gate=gate, activation=activation, shared=shared, bias=bias, fp32=fp32)
    run(3, 150, 50, seed=4, gate=gate, activation=activation, shared=shared, bias=bias, fp32=fp32, kind="layer")


@pytest.mark.parametrize("rows", [1, 2, 3, 31, 64, 1000])
def test_rows(rows):
    run(rows, 384, 96, seed=rows)
    run(rows, 3, 1, seed=rows)


def test_without_weights_and_with_eps():
    run(7, 256, 64, weight=False)
    run(7, 256, 64, weight=False, bias=True)
    run(7, 256, 64, eps=0.0)
    run(7, 256, 64, eps=10.0)


def test_rows_of_zeros_and_of_one_value():
    def edit(x, z):
        x[0] = 0
        x[1] = 2.5
        x[2] = 0
        x[2, 5] = 1e4
        x[3] *= 1e-12
        x[4] *= 1e15
    for kind in ("rms", "layer"):
        run(6, 256, 128, kind=kind, edit=edit)


def test_nan_and_inf_stay_in_their_group():
    x, z, w, b = draw(4, 256, 64, 1, "last", False, False, False)
    want, tol = R.norm(x, 64, w, b, z, 1e-5, "rms", "silu", False)
    x[1, 70] = float("nan")
    x[2, 3] = float("inf")
    got = S.sconv_group_norm(x.to(DEV), 64, weight=w.to(DEV), z=z.to(DEV), activation="silu").cpu()
    ok = torch.ones(4, 256, dtype=torch.bool)
    ok[1, 64:128] = False
    ok[2, :64] = False
    R.check(got[ok], want[ok], tol[ok], "norm")
    assert torch.isnan(got[1, 64:128]).all()


@pytest.mark.parametrize("where", ["x", "z", "new"])
@pytest.mark.parametrize("channels,size", [(512, 128), (8192, 8192), (300, 75)])
def test_in_place(where, channels, size):
    run(11, channels, size, out=where)


@pytest.mark.parametrize("which", ["pitched", "offset", "transposed", "one_row"])
@pytest.mark.parametrize("channels,size", [(512, 128), (200, 50)])
def test_layouts(which, channels, size):
    def place(t):
        if which == "transposed":
            return t.t().contiguous().t().to(DEV)
        extra, off = (8, 8) if which == "pitched" else (5, 3)
        w = torch.full((t.shape[0], t.shape[1] + extra), 7.0, dtype=t.dtype, device=DEV)[:, off:off + t.shape[1]]
        return w.copy_(t)
    run(1 if which == "one_row" else 6, channels, size, place=place, out="new")


def test_heads():
    """(rows, heads, head_dim), as views too, is (rows, channels) by head_dim."""
    x, z, w, _ = draw(10, 6 * 64, 64, 5, "last", True, False, False)
    x, z, w = x.to(DEV), z.to(DEV), w.to(DEV)
    want = S.sconv_group_norm(x, 64, weight=w, z=z, activation="silu")
    got = S.sconv_group_norm(x.view(10, 6, 64), weight=w, z=z.view(10, 6, 64), activation="silu")
    assert torch.equal(got.view(10, -1), want)
    odd = x.view(10, 6, 64).transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(S.sconv_group_norm(odd, weight=w, z=z.view(10, 6, 64), activation="silu").reshape(10, -1), want)


def test_graph_replays_match_eager():
    x, z, w, _ = (t.to(DEV) if t is not None else None for t in draw(50, 1024, 128, 6, "first", False, False, False))
    out = torch.zeros_like(x)
    call = lambda o: S.sconv_group_norm(x, 128, weight=w, z=z, activation="silu", gate_first=True, out=o)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for _ in range(3):
        x.mul_(1.5)
        graph.replay()
        want = call(None)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_empty():
    x = torch.zeros(0, 64, dtype=BF, device=DEV)
    assert S.sconv_group_norm(x, 32).shape == (0, 64)
    x = torch.zeros(3, 0, dtype=BF, device=DEV)
    assert S.sconv_group_norm(x).shape == (3, 0)


def test_rows_past_32_bits():
    """More than 2^32 bytes of rows."""
    rows, c = (1 << 31) // 4096 + 5, 4096
    x = torch.zeros(rows, c, dtype=BF, device=DEV)
    x[-1] = torch.randn(c, device=DEV).to(BF)
    out = S.sconv_group_norm(x, 1024)
    want, tol = R.norm(x[-1:].cpu(), 1024, None, None, None, 1e-5, "rms", None, False)
    R.check(out[-1:], want, tol, "norm")
    assert not out[:-1].any()
