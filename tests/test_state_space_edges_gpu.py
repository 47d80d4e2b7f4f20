"""GPU tests of the state space operators where they can go wrong: nothing to
do, values that are not numbers, and sizes that take the forms which the shapes
of ``test_state_space_gpu.py`` leave out.  Inputs, checks and tolerances are
that file's where a test does not state its own."""
import pytest
import torch

import onnx_lstm_gru_gb300 as rk
from test_state_space_gpu import (  # noqa: F401  (layer: the fixture)
    DTYPES, F64, check, conv_inputs, conv_want, layer, past_zero, poison, scan_inputs, scan_want)

pytestmark = pytest.mark.gpu

SCAN_GRADS = ("dX", "dDelta", "dA", "dB", "dC", "dD", "d_delta_bias", "d_initial_state", "dZ")


def check_all(got, want, name=""):
    """``check`` where the definition is finite; NaN and infinities exactly where it has them."""
    g, w = got.double().cpu(), want.to(F64)
    assert g.shape == w.shape, name
    assert torch.equal(g.isnan(), w.isnan()), f"{name}: {int(g.isnan().sum())} NaN, {int(w.isnan().sum())} by definition"
    assert torch.equal(g[w.isinf()], w[w.isinf()]), f"{name}: infinities"
    on = w.isfinite()
    check(torch.where(on.to(got.device), got, torch.zeros_like(got)), torch.where(on, w, torch.zeros_like(w)), name)


# ---- nothing to do -----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("channels", [1, 5, 20, 33, 64])
@pytest.mark.parametrize("width", [1, 4, 8])
def test_conv_no_steps_any_channels(layer, channels, width, dtype):
    """The state after no steps is the state before them, of channels that
    16-byte pieces divide or not; and nothing else is written."""
    p = rk.ConvProblem(0, 3, channels, width, dtype)
    t, _ = conv_inputs(p, channels + width)
    size = 3 * (width - 1) * channels
    room = torch.full((size + 64,), 7.0, dtype=rk.torch_dtype(dtype), device="cuda")
    final = room[32:32 + size].view(3, width - 1, channels)
    assert torch.equal(layer.conv(p, **t, final_state=final)["final_state"], t["initial_state"])
    assert bool((room[:32] == 7).all()) and bool((room[32 + size:] == 7).all())
    del t["initial_state"]
    assert not layer.conv(p, **t, final_state=final)["final_state"].any()
    state = final.fill_(3.0)
    assert bool((layer.conv(p, **t, initial_state=state, final_state=state)["final_state"] == 3).all())


# ---- values that are not numbers --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seq,batch,channels,state,groups,lens", [
    (1, 3, 40, 16, 2, [1, 0, 1]), (1, 2, 40, 5, 1, None), (21, 3, 40, 16, 2, [21, 5, 0]), (13, 2, 24, 5, 1, None),
    (16, 2, 24, 64, 1, [16, 9]), (203, 3, 40, 16, 2, [203, 13, 0]), (203, 2, 24, 7, 1, [100, 61]),
    (67, 1, 24, 100, 1, None)])
def test_scan_nan_rate(layer, seq, batch, channels, state, groups, lens, dtype):
    """A rate that is no number makes none of its channel's state, and of
    nothing else: not of a sequence without steps, and not of the gradient that
    reaches the last step, which no decay has touched."""
    p = rk.ScanProblem(seq, batch, channels, state, groups, dtype)
    t, g = scan_inputs(p, seq + state, True, lens)
    t["A"][3, 2] = float("nan")
    if lens:
        poison(p, t, ("X", "Delta", "B", "C", "Z"), lens)
        poison(p, g, ("dY",), lens)
    want = scan_want(p, t, g)
    assert bool(want["Y"].isnan().any()) and not bool(want["Y"].isnan().all())
    for k, v in {**layer.scan(p, **t), **layer.scan_grad(p, **t, **g, want=SCAN_GRADS)}.items():
        check_all(v, want[k], k)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("seq,batch,channels,lens", [(21, 3, 24, [21, 5, 0]), (7, 2, 10, [0, 2]), (40, 1, 16, None),
                                                     (90, 2, 16, [90, 64])])
def test_conv_special_weights(layer, seq, batch, channels, lens, act, dtype):
    """Weights that are infinite or no numbers meet the steps that there are,
    not the zeros past a row's length or on both sides of a chunk."""
    for width in (1, 3, 4, 8):
        p = rk.ConvProblem(seq, batch, channels, width, dtype, 1, act)
        t, g = conv_inputs(p, seq, True, lens)
        t["W"][5, 0], t["W"][7, width // 2] = float("inf"), float("nan")
        t["W"][9, width - 1] = -float("inf")
        t["B"][2] = float("nan")
        if lens:
            poison(p, t, ("X",), lens)
            poison(p, g, ("dY",), lens)
        want = conv_want(p, t, g)
        got = {**layer.conv(p, **t), **layer.conv_grad(p, **t, **g, want=("dX", "dW", "dB", "d_initial_state"))}
        for k, v in got.items():
            check_all(v, want[k], f"{k} width={width}")
        if lens:
            past_zero(p, got, ("Y", "dX"), lens)


# ---- accuracy of float32 outputs ------------------------------------------------------------------------

def relative(got, want, bound):
    off = ((got.double().cpu() - want) / want).abs()
    assert float(off.max()) <= bound, f"off by {float(off.max()):.3g} at {int(off.argmax())}"


def test_silu_and_gates_far_below_zero(layer):
    """x sigmoid(x) and its slope keep their relative accuracy where they are
    tiny.  The exponential is off by 2^-22 and three roundings of 2^-24, 1 + e by
    2^-24, the reciprocal by 2^-23, the product by 2^-24: under 3 * 2^-22.  The
    slope, sigmoid(x) (1 + x (1 - sigmoid(x))), is taken below -3, where its
    second factor is at least 1.8: three roundings more and at most twice the
    sigmoid's error, 2^-20."""
    x = torch.linspace(-85.0, -3.0, 4096, device="cuda")
    z = x.double().cpu()
    s = torch.sigmoid(z)
    silu, slope = z * s, s * (1 + z * (1 - s))
    p = rk.ConvProblem(1, 1, 4096, 1)
    one, rows = torch.ones(4096, 1, device="cuda"), x.view(1, 1, -1)
    relative(layer.conv(p, X=rows, W=one)["Y"].view(-1), silu, 3 * 2.0 ** -22)
    relative(layer.conv_grad(p, X=rows, W=one, dY=torch.ones_like(rows))["dX"].view(-1), slope, 2.0 ** -20)
    for steps in (1, 5):  # D u alone behind the gate
        q = rk.ScanProblem(steps, 1, 4096, 4)
        Z, B = x.expand(steps, 1, 4096).contiguous(), torch.zeros(steps, 1, 4, device="cuda")
        o, D = torch.ones_like(Z), torch.ones(4096, device="cuda")
        args = dict(X=o, Delta=o, A=-torch.ones(4096, 4, device="cuda"), B=B, C=B, D=D, Z=Z)
        got = {**layer.scan(q, **args), **layer.scan_grad(q, **args, dY=o, want=("dZ", "dX"))}
        for i in range(steps):
            relative(got["Y"][i, 0], silu, 3 * 2.0 ** -22)
            relative(got["dZ"][i, 0], slope, 2.0 ** -20)
            relative(got["dX"][i, 0], silu, 2.0 ** -20)


def test_silu_and_gates_at_the_ends(layer):
    """What is beyond float32: 0 far below, x far above; an infinity above and
    a NaN stay what they are."""
    x = torch.tensor([-1e30, -200.0, -89.0, 0.0, 89.0, 200.0, 1e30, float("inf"), float("nan")], device="cuda")
    want = torch.tensor([0.0, 0.0, 0.0, 0.0, 89.0, 200.0, 1e30, float("inf"), float("nan")], device="cuda")
    rows, o, B = x.view(1, 1, -1), torch.ones(1, 1, 9, device="cuda"), torch.zeros(1, 1, 4, device="cuda")
    for y in (layer.conv(rk.ConvProblem(1, 1, 9, 1), X=rows, W=torch.ones(9, 1, device="cuda"))["Y"],
              layer.scan(rk.ScanProblem(1, 1, 9, 4), X=o, Delta=o, A=-torch.ones(9, 4, device="cuda"), B=B, C=B,
                         D=torch.ones(9, device="cuda"), Z=rows)["Y"]):
        assert torch.equal(y.view(-1).isnan(), want.isnan())
        assert torch.equal(y.view(-1)[:-1], want[:-1]), y


# ---- calls ----------------------------------------------------------------------------------------------

def test_inputs_are_not_made_up(layer):
    """A wanted name is an output or a tensor that was passed; memory made for
    anything else would be read as an operand."""
    p = rk.ScanProblem(4, 2, 16, 16)
    t, g = scan_inputs(p, 1, state=False, extras=False)
    before = layer.launches()
    for name in ("Z", "D", "delta_bias", "sequence_lens", "initial_state"):
        with pytest.raises(ValueError, match=name):
            layer.scan(p, **t, want=("Y", name))
    for name in ("Z", "d_final_state"):
        with pytest.raises(ValueError, match=name):
            layer.scan_grad(p, **t, **g, want=("dX", name))
    with pytest.raises(ValueError, match="initial_state"):
        layer.conv(rk.ConvProblem(4, 2, 16), t["X"], W=torch.zeros(16, 4, device="cuda"), want=("initial_state",))
    with pytest.raises(ValueError, match="Scale"):
        layer.norm(rk.NormProblem(4, 16), torch.zeros(4, 16, device="cuda"), want=("Y", "Scale"))
    assert layer.launches() == before
    got = layer.scan(p, **t, want=("Y", "X", "A"))
    assert got["X"] is t["X"] and got["A"] is t["A"]
    assert layer.scan_grad(p, **t, **g, want=SCAN_GRADS[:-1]).keys() == set(SCAN_GRADS[:-1])


@pytest.mark.parametrize("cols,counts", [(64, (2, 1, 2)), (8192, (2, 1, 2)), (8200, (3, 1, 2))])
def test_launches_are_counted(layer, cols, counts):
    """All gradients, the rows' alone, the weights' alone: dX of rows too wide
    for registers is a launch of its own."""
    p = rk.NormProblem(40, cols)
    X, dY = torch.randn(40, cols, device="cuda"), torch.randn(40, cols, device="cuda")
    f = layer.norm(p, X)
    for want, n in zip((("dX", "dScale", "dB"), ("dX",), ("dB",)), counts):
        before = layer.launches()
        layer.norm_grad(p, X, dY=dY, Mean=f["Mean"], InvStdDev=f["InvStdDev"], want=want)
        assert layer.launches() - before == n, want
