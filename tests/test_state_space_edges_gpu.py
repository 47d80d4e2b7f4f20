"""GPU tests of the state space operators where they can go wrong: nothing to
do, values that are not numbers, and sizes that take the forms which the shapes
of ``test_state_space_gpu.py`` leave out.  Inputs, checks and tolerances are
that file's where a test does not state its own."""
import pytest
import torch

import onnx_lstm_gru_gb300 as rk
import state_space_reference as ref
from onnx_lstm_gru_gb300 import state_space as ss
from test_state_space_gpu import (  # noqa: F401  (layer: the fixture)
    DTYPES, F64, UNIT, Inputs, check, conv_inputs, conv_want, layer, past_zero, poison, scan_inputs, scan_want)

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


# ---- states that grow --------------------------------------------------------------------------------------

def growing(S, batch, C, K, tiny, seed=5):
    """Zeros through steps of e^20 until the last two steps' inputs; or a state
    of 1e-30 that grows by e^120 within a chunk.  The gradients' way back alike."""
    i = Inputs(seed, "f32")
    t = dict(X=torch.zeros(S, batch, C, device="cuda"), Delta=torch.zeros(S, batch, C, device="cuda"),
             B=i.normal(S, batch, K), C=i.normal(S, batch, K), A=torch.full((C, K), 2.0, device="cuda"))
    g = dict(dY=torch.zeros(S, batch, C, device="cuda"))
    if tiny:
        t["Delta"][S // 3 - 3:S // 3 + 3] = 10.0
        t["initial_state"] = i.normal(batch, C, K) * 1e-30
        g["d_final_state"] = i.normal(batch, C, K) * 1e-30
    else:
        t["Delta"] += 10.0
        t["X"][-2:] = i.normal(2, batch, C)
        t["initial_state"] = torch.zeros(batch, C, K, device="cuda")
        g["dY"][:2] = i.normal(2, batch, C)
    return t, g


@pytest.mark.parametrize("tiny", [False, True])
@pytest.mark.parametrize("batch,state", [(1, 16), (3, 5)])
def test_scan_growing_over_chunks(layer, batch, state, tiny):
    """Chunks that run side by side give what the steps give, although the
    product of a chunk's factors passes float32's range."""
    p = rk.ScanProblem(200, batch, 24, state, softplus=False)
    assert rk.rk_scan_scratch_length(p.to_c()) > 0  # chunks
    t, _ = growing(200, batch, 24, state, tiny)
    t["A"][1] = -2.0  # and a channel that forgets beside them
    want = scan_want(p, t)
    assert float(want["final_state"].abs().max()) > 1e2
    for k, v in layer.scan(p, **t).items():
        check_all(v, want[k], k)


@pytest.mark.parametrize("tiny", [False, True])
@pytest.mark.parametrize("seq,batch,state", [(200, 1, 16), (203, 3, 5), (20, 2, 16), (17, 1, 64)])
def test_scan_grad_growing(layer, seq, batch, state, tiny):
    """The way back alike, in chunks and without them, where the state at a
    step is found from what entered the chunk."""
    p = rk.ScanProblem(seq, batch, 24, state, softplus=False)
    t, g = growing(seq, batch, 24, state, tiny)
    t["A"][1] = -2.0
    want = scan_want(p, t, g)
    names = tuple(n for n in SCAN_GRADS if n != "dZ")
    for k, v in layer.scan_grad(p, **t, **g, want=names).items():
        check_all(v, want[k], k)


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


# ---- forms that larger or other sizes take ------------------------------------------------------------------
#
# float32 bounds here are the operators' own, u the unit roundoff 2^-24:
# a sum of n terms in a tree of depth at most t is off by t u times the sum of
# their magnitudes.

U = 2.0 ** -24


def within(got, want, bound, name=""):
    """|got - want| <= bound, element by element, plus the rounding to got's type."""
    off = (got.double() - want).abs().cpu()
    limit = (bound + UNIT[got.dtype] * want.abs()).cpu() + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    assert bool((off <= limit).all()), f"{name}: off by {float((off / limit.clamp_min(1e-300)).max()):.3g} times the bound"


# Rows at a time start at 6080 rows of up to 256 columns, 3040 of up to 512, 1520 of up to 1024, 608 of up to 2048 and
# 152 of up to 4096; the last group of rows is whole, or short by one to three.  Odd widths are read element by element.
@pytest.mark.parametrize("rows,cols", [(1519, 1000), (1520, 1024), (1523, 1000), (1521, 999), (6083, 96), (6081, 33),
                                       (3043, 400), (613, 2000), (155, 4000), (157, 3001), (153, 4096), (4999, 1017)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_many_rows(layer, rows, cols, dtype):
    """Sums of up to 8 terms per thread, 5 exchanges and up to 16 warps: depth
    under 32.  The mean is off by that of the mean magnitude, the differences
    from it by as much, the deviation's square by twice 32 u; y, at most 6 here
    but for the weights, by less than 200 u times its terms' sizes."""
    i = Inputs(rows + cols, dtype)
    X, S, B = i.rows(rows, cols, mean=0.5), i.normal(cols, mean=1.0, scale=0.2), i.normal(cols)
    p = rk.NormProblem(rows, cols, dtype, epsilon=1e-3)
    guard = torch.full((rows + 4, cols), 7.0, dtype=X.dtype, device="cuda")
    got = layer.norm(p, X, Scale=S, B=B, Y=guard[2:-2])
    x, s, b = X.double(), S.double(), B.double()
    want = ref.norm(x, s, b, 1e-3)
    size = ((x.abs() + x.abs().mean(1, keepdim=True)) * want["InvStdDev"][:, None]) * s.abs() + b.abs()
    within(got["Y"], want["Y"], 200 * U * size, "Y")
    within(got["Mean"], want["Mean"], 64 * U * x.abs().mean(1), "Mean")
    within(got["InvStdDev"], want["InvStdDev"], 128 * U * want["InvStdDev"], "InvStdDev")
    assert bool((guard[:2] == 7).all()) and bool((guard[-2:] == 7).all())
    near = layer.norm(p, X, Scale=S, B=B)
    assert all(torch.equal(near[k], got[k]) for k in near)


def conv_definition(p, t, g):
    """The 64-bit definition over whole tensors, [batch, seq, channels]: sums of shifted rows, masked by length; and the
    sums of magnitudes that dX, dW and dB add up."""
    w, S = p.width, p.seq
    h = {k: v.double() if v.is_floating_point() else v for k, v in {**t, **g}.items()}
    lens = h["sequence_lens"].clamp(0, S).long() if "sequence_lens" in h else torch.full((p.batch,), S, device="cuda")
    on = (torch.arange(S, device="cuda") < lens[:, None])[..., None]
    X, dY = h["X"].where(on, torch.zeros((), dtype=F64, device="cuda")), h["dY"].where(on, torch.zeros((), dtype=F64, device="cuda"))
    x = torch.cat([h["initial_state"], X], 1)  # row s + w - 1 is step s
    pre = h["B"] + sum(h["W"][:, j] * x[:, j:j + S] for j in range(w))
    sig = torch.sigmoid(pre)
    dp = dY * sig * (1 + pre * (1 - sig)) if p.activation == "silu" else dY
    dx, size = torch.zeros_like(x), torch.zeros_like(x)
    for j in range(w):
        dx[:, j:j + S] += h["W"][:, j] * dp
        size[:, j:j + S] += (h["W"][:, j] * dY).abs() * (1 + pre.abs())
    n = torch.arange(p.batch, device="cuda")[:, None]
    last = lens[:, None] + torch.arange(w - 1, device="cuda")
    dx[n, last] += h["d_final_state"]
    size[n, last] += h["d_final_state"].abs()
    dW = torch.stack([(dp * x[:, j:j + S]).sum((0, 1)) for j in range(w)], 1)
    dWs = torch.stack([(dY * x[:, j:j + S]).abs().mul(1 + pre.abs()).sum((0, 1)) for j in range(w)], 1)
    y = pre * sig if p.activation == "silu" else pre
    out = dict(Y=y * on, final_state=x[n, last], dX=dx[:, w - 1:] * on, dW=dW, dB=dp.sum((0, 1)),
               d_initial_state=dx[:, :w - 1])
    ysize = h["B"].abs() + sum((h["W"][:, j] * x[:, j:j + S]).abs() for j in range(w))
    return out, dict(Y=ysize, final_state=0 * out["final_state"], dX=size[:, w - 1:], dW=dWs,
                     dB=(dY.abs() * (1 + pre.abs())).sum((0, 1)), d_initial_state=size[:, :w - 1])


# Chunks of the gradient are 12, 20, 44 and 64 steps here (they grow with seq * batch * channels), with groups of four
# steps inside a chunk for every width; lengths end in, at the end of and before a chunk.
@pytest.mark.parametrize("seq,batch,channels", [(700, 4, 512), (1207, 4, 400), (2600, 4, 500), (3001, 3, 1030)])
@pytest.mark.parametrize("width", [1, 2, 3, 4, 5, 6, 7, 8])
def test_conv_grad_long_chunks(layer, seq, batch, channels, width):
    """At most width products per sum for dX, with the pre-activation's slope
    off by under 32 u (1 + |p|); sums for dW and dB over at most 64 steps of a
    thread, 4 chunks of a block and the slices, in eight parts: depth under 512."""
    for dtype, act, ragged in (("f32", "silu", True), ("bf16", "none", False)):
        p = rk.ConvProblem(seq, batch, channels, width, dtype, 1, act)
        lens = [seq, 64, 65, 1][:batch] if ragged else None
        t, g = conv_inputs(p, seq + width, True, lens)
        if lens:
            poison(p, t, ("X",), lens)
            poison(p, g, ("dY",), lens)
        names = ("dX", "dW", "dB", "d_initial_state")
        got = {**layer.conv(p, **t), **layer.conv_grad(p, **t, **g, want=names)}
        want, size = conv_definition(p, t, g)
        for k, v in got.items():
            within(v, want[k], (512 if k in ("dW", "dB") else 64) * U * size[k], f"{k} {dtype}")
        if lens:
            past_zero(p, got, ("Y", "dX"), lens)
        again = layer.conv_grad(p, **t, **g, want=names)
        assert all(torch.equal(got[k], again[k]) for k in names)


# One token: 1, 2, 4, 8, 16 and 32 threads per channel, read in pieces of four (whole multiples of four, dense) and
# element by element; sequences in groups of four, the last one short.
@pytest.mark.parametrize("state", [1, 3, 4, 7, 8, 13, 16, 20, 31, 32, 50, 64, 100, 128])
@pytest.mark.parametrize("dtype", DTYPES)
def test_single_tokens(layer, state, dtype):
    for batch, channels, groups, wide, lens in ((1, 40, 1, False, None), (7, 66, 2, False, [1, 0, 1, 1, 0, 1, 9]),
                                                (5, 33, 3, True, None), (9, 130, 1, False, None)):
        p = rk.ScanProblem(1, batch, channels, state, groups, dtype)
        t, _ = scan_inputs(p, state + batch, True, lens, wide)
        if lens:
            poison(p, t, ("X", "Delta", "B", "C", "Z"), lens)
        want = scan_want(p, t)
        got = layer.scan(p, **t)
        for k, v in got.items():
            check(v, want[k], f"{k} {batch} x {channels}")
        once = layer.scan(p, **t, final_state=t["initial_state"])  # updated in place
        assert torch.equal(once["final_state"], got["final_state"]) and torch.equal(once["Y"], got["Y"])


# The gradient's sums of dB and dC are limited to 2^26 floats of partial sums; beyond it a block runs several channel
# tiles in turn.  (tiles, tiles per block) here: (9, 2) with a last block of one tile and a last tile of six channels,
# and (9, 2) over chunks of one long sequence; in both, halves of the channels stay below the limit.
@pytest.mark.parametrize("seq,batch,lens", [(12, 2500, True), (29300, 1, False), (9800, 3, True)])
def test_scan_grad_several_tiles_per_block(layer, seq, batch, lens):
    C, K = 70, 128
    p = rk.ScanProblem(seq, batch, C, K, layout=1)
    half = rk.ScanProblem(seq, batch, C // 2, K, layout=1)
    row = batch * seq * 2 * K
    assert 9 * row > 64 << 20 and 5 * row < 64 << 20
    lens = [seq - n % seq if n % 5 else 0 for n in range(batch)] if lens and batch > 3 else [seq, 1003, 0] if lens else None
    t, g = scan_inputs(p, seq, True, lens)
    if lens:
        poison(p, t, ("X", "Delta", "B", "C", "Z"), lens)
        poison(p, g, ("dY",), lens)
    got = layer.scan_grad(p, **t, **g, want=SCAN_GRADS)
    assert all(torch.equal(v, got[k]) for k, v in layer.scan_grad(p, **t, **g, want=SCAN_GRADS).items())
    # the halves of the channels, each below the limit: rows and states side by side, dB and dC their sum
    by_channel = {k: -1 for k in ("X", "Delta", "Z", "dY", "dX", "dDelta", "dZ")}
    by_channel.update({k: 0 for k in ("A", "D", "delta_bias", "dA", "dD", "d_delta_bias")})
    by_channel.update({k: 1 for k in ("initial_state", "d_final_state", "d_initial_state")})

    def part(x, a):
        return {k: v.narrow(by_channel[k], a, C // 2).contiguous() if k in by_channel else v for k, v in x.items()}
    parts = [layer.scan_grad(half, **part({**t, **g}, a), want=SCAN_GRADS) for a in (0, C // 2)]
    for k in SCAN_GRADS:
        a, b = parts[0][k].double(), parts[1][k].double()
        want = a + b if k in ("dB", "dC") else torch.cat([a, b], by_channel[k])
        top = float(want.abs().max())
        # both are float32 results of the same steps, cut into chunks in different places: the bound of ``check``, twice
        assert float((got[k].double() - want).abs().max()) <= 2e-4 * top, k
    if lens:
        past_zero(p, got, ("dX", "dDelta", "dZ", "dB", "dC"), lens)
    if batch > 3:  # against the definition: a few sequences alone (dA, dD and d_delta_bias are sums over all)
        some = [0, 1, 4, 5, 2499]
        few = rk.ScanProblem(seq, len(some), C, K, layout=1)
        t2 = {k: v if k in ("A", "D", "delta_bias") else v[some] for k, v in t.items()}
        want = scan_want(few, t2, {k: v[some] for k, v in g.items()})
        for k in ("dX", "dDelta", "dZ", "dB", "dC", "d_initial_state"):
            check(got[k][some], want[k], k)


# ---- the C entries with the handle's own scratch ---------------------------------------------------------------

def c_operands(op, problem, tensors):
    """The operand list of dense tensors."""
    ops = getattr(ss, f"rk_{op}_operands")()
    rows = ss._OPERANDS[op][0]
    for n, v in tensors.items():
        setattr(ops, n, ss.rk_rows(v.data_ptr(), 0, v.numel(), 0, 0) if n in rows else
                rk.rk_tensor(v.data_ptr(), 0, v.numel()))
    return ops


def c_call(handle, op, problem, tensors, outputs):
    out = {n: torch.full(problem.shapes()[n], float("nan"), device="cuda",
                         dtype=torch.float32 if problem._operands()[n][1] == "f" else rk.torch_dtype(problem.dtype))
           for n in outputs}
    st = getattr(rk, f"rk_{op}_encode")(handle, problem.to_c(), c_operands(op, problem, {**tensors, **out}), None,
                                        torch.cuda.current_stream().cuda_stream)
    return st, out


def test_scratch_of_the_handle(layer):
    """Grown from call to call, and used again by smaller ones; refused while
    a graph is captured, which would keep its address."""
    handle = rk.rk_create(0)
    calls = []
    for op, p in (("scan", rk.ScanProblem(100, 1, 24, 16)), ("scan_grad", rk.ScanProblem(300, 2, 72, 16)),
                  ("scan", rk.ScanProblem(64, 2, 24, 5)), ("conv_grad", rk.ConvProblem(90, 2, 40)),
                  ("norm_grad", rk.NormProblem(300, 260)), ("scan_grad", rk.ScanProblem(900, 3, 130, 16))):
        if op.startswith("scan"):
            t, g = scan_inputs(p, 3)
            outputs = ("Y", "final_state") if op == "scan" else SCAN_GRADS
        elif op == "conv_grad":
            t, g = conv_inputs(p, 3)
            outputs = ("dX", "dW", "dB", "d_initial_state")
        else:
            i = Inputs(3, "f32")
            t = dict(X=i.normal(300, 260), dY=i.normal(300, 260), Mean=i.normal(300), InvStdDev=i.normal(300).abs())
            g, outputs = {}, ("dX", "dScale", "dB")
        if op == "scan":
            g = {}
        calls.append((op, p, {**t, **g}, outputs))
    for op, p, t, outputs in calls:
        want = getattr(layer, op)(p, **t, want=outputs)
        st, got = c_call(handle, op, p, t, outputs)
        assert st == rk.RK_OK, rk.rk_last_error(handle)
        torch.cuda.synchronize()
        for k in outputs:
            assert torch.equal(got[k], want[k]), (op, k)
    op, p, t, outputs = calls[0]
    x = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    before = rk.rk_launch_count(handle)
    with torch.cuda.graph(graph):
        x += 1
        st, _ = c_call(handle, op, p, t, outputs)
        message = rk.rk_last_error(handle)
    assert st == rk.RK_ERR_UNSUPPORTED and "scratch: place it" in message
    assert rk.rk_launch_count(handle) == before
    graph.replay()
    st, got = c_call(handle, op, p, t, outputs)  # and the handle goes on
    assert st == rk.RK_OK
    torch.cuda.synchronize()
    want = getattr(layer, op)(p, **t, want=outputs)
    assert all(torch.equal(got[k], want[k]) for k in outputs) and bool((x == 1).all())
    rk.rk_destroy(handle)
