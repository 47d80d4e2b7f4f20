"""GPU tests of the state space operators against their 64-bit definitions.

Tolerance, per element of an output with largest magnitude m: u |r| + 1e-4 m.
u is the unit roundoff of the output's type (half its epsilon: float32 2^-24,
Half 2^-11, bfloat16 2^-8): every output is rounded once.  1e-4 covers float32 arithmetic:
a state or gradient is the result of at most 300 steps here, each with an
exponential of relative error 2^-22 and three roundings of 2^-24, 300 * 1.75 *
2^-22 = 1.3e-4 if all of them were the largest possible and of one sign; half
of that is far above what rounding errors of both signs reach.  Half outputs
below its smallest normal number are rounded to multiples of 2^-24.
Past a row's length outputs are exactly 0, and everything is bit-identical
between runs.
"""
import numpy as np
import pytest
import torch

import onnx_lstm_gru_gb300 as rk
import state_space_reference as ref

pytestmark = pytest.mark.gpu

F64 = torch.float64
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
DTYPES = ["f32", "f16", "bf16"]


@pytest.fixture(scope="module")
def layer():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    rk.build()
    rk.load()
    lay = rk.StateSpaceLayer()
    yield lay
    torch.cuda.synchronize()
    lay.close()


class Inputs:
    """Seeded inputs in a problem's types; wide: rows as slices of wider ones, with NaN around them."""

    def __init__(self, seed, dtype, wide=False):
        self.rng = np.random.default_rng(seed)
        self.t = rk.torch_dtype(dtype)
        self.wide = wide

    def normal(self, *shape, scale=1.0, mean=0.0, dtype=None):
        x = torch.from_numpy(self.rng.normal(mean, scale, shape))
        return x.to(dtype or self.t).cuda()

    def rows(self, *shape, **kw):
        x = self.normal(*shape, **kw)
        if not self.wide:
            return x
        wide = torch.full(shape[:-1] + (shape[-1] + 8 + int(self.rng.integers(0, 2)),), float("nan"), dtype=x.dtype,
                          device="cuda")
        at = int(self.rng.integers(0, 9))
        wide[..., at:at + shape[-1]] = x
        return wide[..., at:at + shape[-1]]


def check(got, want, name="", arithmetic=1e-4):
    want = want.to(F64)
    g = got.double().cpu()
    assert g.shape == want.shape, name
    if not want.numel():
        return
    top = float(want.abs().max())
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    bound = UNIT[got.dtype] * want.abs() + arithmetic * top + tiny
    off = (g - want).abs()
    assert bool((off <= bound).all()), f"{name}: off by {float((off - bound).max()):.3g} beyond the bound, largest {top:.3g}"


def host(t):
    return {k: (v.double().cpu() if v.is_floating_point() else v.cpu()) for k, v in t.items() if v is not None}


def bits(out):
    return {k: v.contiguous().cpu().view(torch.uint8) for k, v in out.items()}


def same_bits(a, b):
    a, b = bits(a), bits(b)
    assert a.keys() == b.keys()
    for k in a:
        assert torch.equal(a[k], b[k]), k


# ---- layer normalisation -------------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (3, 7), (5, 128), (33, 512), (64, 1024), (7, 1000), (9, 2050), (2, 4096), (3, 5003), (2, 8200),
               (2, 16400), (2, 40000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm(layer, rows, cols, dtype):
    for wide in (False, True):
        i = Inputs(rows * cols, dtype, wide)
        X, S, B = i.rows(rows, cols, mean=0.5), i.normal(cols, mean=1.0, scale=0.2), i.normal(cols)
        p = rk.NormProblem(rows, cols, dtype, epsilon=1e-3)
        got = layer.norm(p, X, Scale=S, B=B)
        h = host(dict(X=X, S=S, B=B))
        want = ref.norm(h["X"], h["S"], h["B"], 1e-3)
        for k in want:
            check(got[k], want[k], f"{k} wide={wide}")
        same_bits(got, layer.norm(p, X, Scale=S, B=B))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(1500, 96), (700, 1024), (257, 777)])
def test_norm_grad(layer, rows, cols, dtype):
    for wide in (False, True):
        i = Inputs(rows + cols, dtype, wide)
        X, dY, S = i.rows(rows, cols, mean=0.5), i.rows(rows, cols), i.normal(cols, mean=1.0, scale=0.2)
        f = ref.norm(X.double().cpu(), epsilon=1e-3)
        mean, inv = f["Mean"].float().cuda(), f["InvStdDev"].float().cuda()
        p = rk.NormProblem(rows, cols, dtype, epsilon=1e-3)
        args = dict(Scale=S, Mean=mean, InvStdDev=inv, dY=dY)
        got = layer.norm_grad(p, X, **args)
        h = host(dict(X=X, **args))
        want = ref.norm_grad(h["X"], h["dY"], h["Mean"], h["InvStdDev"], h["Scale"])
        for k in want:
            check(got[k], want[k], f"{k} wide={wide}")
        same_bits(got, layer.norm_grad(p, X, **args))


# many rows, read in pieces and element by element: whole turns of all blocks, one row less and more
@pytest.mark.parametrize("rows,cols", [(455, 130), (457, 130), (913, 264), (3649, 264), (2433, 1031), (7296, 777),
                                       (7297, 777), (29185, 33)])
def test_norm_grad_many_rows(layer, rows, cols):
    for dtype in ("f32", "bf16"):
        i = Inputs(rows + cols, dtype)
        X, dY, S = i.rows(rows, cols), i.rows(rows, cols), i.normal(cols, mean=1.0, scale=0.2)
        f = ref.norm(X.double().cpu(), epsilon=1e-3)
        args = dict(Scale=S, Mean=f["Mean"].float().cuda(), InvStdDev=f["InvStdDev"].float().cuda(), dY=dY)
        got = layer.norm_grad(rk.NormProblem(rows, cols, dtype, epsilon=1e-3), X, **args)
        h = host(dict(X=X, **args))
        want = ref.norm_grad(h["X"], h["dY"], h["Mean"], h["InvStdDev"], h["Scale"])
        for k in want:
            check(got[k], want[k], k)


def test_norm_without_weights(layer):
    i = Inputs(1, "f32")
    X, dY = i.normal(6, 50), i.normal(6, 50)
    p = rk.NormProblem(6, 50)
    got = layer.norm(p, X)
    want = ref.norm(X.double().cpu())
    check(got["Y"], want["Y"])
    g = layer.norm_grad(p, X, Mean=got["Mean"], InvStdDev=got["InvStdDev"], dY=dY)
    w = ref.norm_grad(X.double().cpu(), dY.double().cpu(), want["Mean"], want["InvStdDev"])
    for k in w:
        check(g[k], w[k], k)
    assert layer.norm_grad(p, X, Mean=got["Mean"], InvStdDev=got["InvStdDev"], dY=dY, want=("dX",)).keys() == {"dX"}


def test_norm_no_rows(layer):
    p = rk.NormProblem(0, 40, "f16")
    e = torch.empty(0, 40, dtype=torch.float16, device="cuda")
    stat = torch.empty(0, device="cuda")
    assert layer.norm(p, e)["Y"].shape == (0, 40)
    g = layer.norm_grad(p, e, Mean=stat, InvStdDev=stat, dY=e)
    assert not g["dScale"].any() and not g["dB"].any()


def test_norm_special_rows(layer):
    """A constant row is its bias; a mean far above the spread costs no more
    than the rounding of the inputs' differences; a NaN stays in its row."""
    cols = 640
    i = Inputs(3, "f32")
    X = i.normal(4, cols)
    X[0] = 3.25
    X[1] += 4096.0
    X[2, 17] = float("nan")
    B = i.normal(cols)
    got = layer.norm(rk.NormProblem(4, cols), X, B=B)
    want = ref.norm(X.double().cpu(), B=B.double().cpu())
    assert torch.equal(got["Y"][0], B)
    for r in (0, 1, 3):
        check(got["Y"][r], want["Y"][r], str(r), arithmetic=4096 * 2.0 ** -23)
    assert bool(got["Y"][2].isnan().all())


# ---- causal convolution ----------------------------------------------------------------------------

def conv_inputs(p, seed, state=True, lens=None, wide=False):
    i = Inputs(seed, p.dtype, wide)
    sh = p.shapes()
    t = dict(X=i.rows(*sh["X"]), W=i.normal(*sh["W"], scale=0.5), B=i.normal(*sh["B"], scale=0.3))
    if state:
        t["initial_state"] = i.normal(*sh["initial_state"])
    if lens is not None:
        t["sequence_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    g = dict(dY=i.rows(*sh["dY"]))
    if state:
        g["d_final_state"] = i.normal(*sh["final_state"])
    return t, g


def batch_first(p, t, names):
    return {k: (v.transpose(0, 1) if k in names and p.layout == 0 and v.dim() == 3 else v) for k, v in t.items()}


def conv_want(p, t, g=None):
    h = host(batch_first(p, {**t, **(g or {})}, ("X", "dY")))
    lens = h.pop("sequence_lens", None)
    out = ref.conv(lens=lens, silu=p.activation == "silu", **h)
    return batch_first(p, out, ("Y", "dX"))


def poison(p, t, names, lens):
    """NaN past every row's length."""
    for k in names:
        if k in t:
            x = t[k] if p.layout == 1 else t[k].transpose(0, 1)
            for n, L in enumerate(lens):
                x[n, min(max(L, 0), p.seq):] = float("nan")


def past_zero(p, out, names, lens):
    for k in names:
        if k in out:
            x = out[k] if p.layout == 1 else out[k].transpose(0, 1)
            for n, L in enumerate(lens):
                assert not x[n, min(max(L, 0), p.seq):].any(), k


CONV = [  # seq, batch, channels, width, layout, lens
    (1, 1, 1, 4, 0, None), (1, 5, 64, 4, 1, None), (2, 3, 40, 4, 0, [2, 0, 1]), (3, 2, 7, 8, 1, [3, 2]),
    (17, 3, 64, 4, 0, [17, 1, 0]), (33, 2, 200, 3, 1, None), (70, 4, 36, 5, 0, [70, 33, -2, 99]),
    (100, 2, 65, 8, 1, [100, 64]), (64, 2, 24, 1, 0, [64, 5]), (50, 2, 264, 2, 1, [16, 32]), (40, 1, 16, 6, 0, None),
    (35, 2, 16, 7, 1, None),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seq,batch,channels,width,layout,lens", CONV)
def test_conv(layer, seq, batch, channels, width, layout, lens, dtype):
    for wide, state, act in ((False, True, "silu"), (True, False, "none"), (True, True, "silu")):
        p = rk.ConvProblem(seq, batch, channels, width, dtype, layout, act)
        t, g = conv_inputs(p, seq + channels, state, lens, wide)
        if lens:
            poison(p, t, ("X",), lens)
            poison(p, g, ("dY",), lens)
        got = layer.conv(p, **t)
        grads = ("dX", "dW", "dB") + (("d_initial_state",) if state else ())
        back = layer.conv_grad(p, **t, **g, want=grads)
        want = conv_want(p, t, g)
        for k, v in {**got, **back}.items():
            check(v, want[k], f"{k} wide={wide} state={state}")
        if lens:
            past_zero(p, {**got, **back}, ("Y", "dX"), lens)
        same_bits(got, layer.conv(p, **t))
        same_bits(back, layer.conv_grad(p, **t, **g, want=grads))


@pytest.mark.parametrize("dtype", DTYPES)
def test_transposed_views(layer, dtype):
    """Operands stored in the other layout's order."""
    for layout in (0, 1):
        p = rk.ConvProblem(19, 3, 40, 4, dtype, layout)
        t, g = conv_inputs(p, 2)
        q = rk.ScanProblem(19, 3, 40, 16, 2, dtype, layout)
        u, d = scan_inputs(q, 2)

        def turned(x):
            return {k: (v.transpose(0, 1).contiguous().transpose(0, 1) if k in ROWS and v.dim() == 3 else v)
                    for k, v in x.items()}
        same_bits(layer.conv(p, **turned(t)), layer.conv(p, **t))
        same_bits(layer.conv_grad(p, **turned({**t, **g})), layer.conv_grad(p, **t, **g))
        same_bits(layer.scan(q, **turned(u)), layer.scan(q, **u))
        outs = turned({k: torch.empty(q.shapes()[k], dtype=rk.torch_dtype(dtype), device="cuda") for k in ("dX", "dB", "dZ")})
        same_bits(layer.scan_grad(q, **turned({**u, **d}), **outs, want=("dX", "dB", "dZ")),
                  layer.scan_grad(q, **u, **d, want=("dX", "dB", "dZ")))


@pytest.mark.parametrize("dtype", DTYPES)
def test_conv_in_pieces(layer, dtype):
    """A prompt, then single tokens on a state updated in place, give the bits
    of the whole sequence."""
    N, C, w = 3, 72, 4
    whole = rk.ConvProblem(25, N, C, w, dtype, layout=1)
    t, _ = conv_inputs(whole, 5, state=False)
    want = layer.conv(whole, **t)
    x = t.pop("X")
    got = layer.conv(rk.ConvProblem(18, N, C, w, dtype, layout=1), X=x[:, :18], **t)
    state, parts = got["final_state"], [got["Y"]]
    for s in range(18, 25):
        o = layer.conv(rk.ConvProblem(1, N, C, w, dtype, layout=1), X=x[:, s:s + 1], initial_state=state,
                       final_state=state, **t)
        parts.append(o["Y"])
    same_bits(dict(Y=torch.cat(parts, 1), final_state=state), want)


def test_conv_state_in_place_over_chunks(layer):
    """The state's row is read by the first steps and written by the same call."""
    p = rk.ConvProblem(200, 2, 48, 4, "f32", layout=0)
    t, _ = conv_inputs(p, 9)
    want = layer.conv(p, **t)
    state = t["initial_state"]
    got = layer.conv(p, **t, final_state=state)
    same_bits(got, want)


def test_conv_no_steps(layer):
    p = rk.ConvProblem(0, 2, 16, 4, "f16")
    t, g = conv_inputs(p, 1)
    assert torch.equal(layer.conv(p, **t)["final_state"], t["initial_state"])
    back = layer.conv_grad(p, **t, **g, want=("dX", "dW", "dB", "d_initial_state"))
    assert torch.equal(back["d_initial_state"], g["d_final_state"]) and not back["dW"].any() and not back["dB"].any()
    none = rk.ConvProblem(4, 0, 16, 4, "f16")
    t, g = conv_inputs(none, 1)
    assert layer.conv(none, **t)["Y"].numel() == 0
    assert not layer.conv_grad(none, **t, **g)["dW"].any()


# ---- selective scan ------------------------------------------------------------------------------------

def scan_inputs(p, seed, state=True, lens=None, wide=False, extras=True):
    i = Inputs(seed, p.dtype, wide)
    sh = p.shapes()
    t = dict(X=i.rows(*sh["X"]), Delta=i.rows(*sh["Delta"], scale=0.5, mean=0.0 if p.softplus else 0.5),
             B=i.rows(*sh["B"]), C=i.rows(*sh["C"]))
    t["A"] = -torch.from_numpy(i.rng.uniform(0.1, 8.0, sh["A"])).float().cuda()
    if extras:
        t.update(D=i.normal(*sh["D"], dtype=torch.float32), Z=i.rows(*sh["Z"]),
                 delta_bias=i.normal(*sh["delta_bias"], scale=0.5, mean=-2.0 if p.softplus else 0.0,
                                     dtype=torch.float32))
    if not p.softplus:
        t["Delta"] = t["Delta"].abs()
        t.pop("delta_bias", None)
    if state:
        t["initial_state"] = i.normal(*sh["initial_state"], dtype=torch.float32)
    if lens is not None:
        t["sequence_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    g = dict(dY=i.rows(*sh["dY"]))
    if state:
        g["d_final_state"] = i.normal(*sh["final_state"], dtype=torch.float32)
    return t, g


ROWS = ("X", "Delta", "Z", "Y", "dY", "dX", "dDelta", "dZ", "B", "C", "dB", "dC")


def scan_want(p, t, g=None):
    h = host(batch_first(p, {**t, **(g or {})}, ROWS))
    lens = h.pop("sequence_lens", None)
    return batch_first(p, ref.scan(lens=lens, softplus=p.softplus, groups=p.groups, **h), ROWS)


SCAN = [  # seq, batch, channels, state, groups, layout, lens
    (1, 1, 1, 1, 1, 0, None), (1, 3, 40, 16, 1, 0, [1, 0, 1]), (3, 2, 24, 5, 2, 1, [3, 1]), (4, 2, 8, 128, 1, 0, None),
    (5, 2, 16, 4, 1, 1, None), (9, 3, 24, 3, 3, 0, [9, 0, 1]), (17, 2, 72, 8, 2, 1, [17, 16]),
    (16, 2, 130, 16, 1, 0, None), (40, 3, 136, 16, 2, 1, [40, 33, 5]), (33, 2, 100, 24, 4, 0, [33, 17]),
    (21, 2, 48, 32, 1, 1, None), (19, 2, 40, 64, 2, 0, [19, 18]), (18, 1, 24, 128, 1, 1, None),
    (20, 1, 17, 100, 1, 0, None), (150, 2, 40, 16, 1, 0, [150, 70]), (300, 1, 72, 7, 1, 1, None),
    (260, 3, 33, 20, 3, 0, [260, -1, 400]), (200, 2, 16, 64, 1, 1, [200, 3]),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seq,batch,channels,state,groups,layout,lens", SCAN)
def test_scan(layer, seq, batch, channels, state, groups, layout, lens, dtype):
    for wide, carried, extras, softplus in ((False, True, True, True), (True, False, False, False),
                                            (True, True, True, True)):
        p = rk.ScanProblem(seq, batch, channels, state, groups, dtype, layout, softplus)
        t, g = scan_inputs(p, seq + channels, carried, lens, wide, extras)
        if lens:
            poison(p, t, ("X", "Delta", "B", "C", "Z"), lens)
            poison(p, g, ("dY",), lens)
        got = layer.scan(p, **t)
        grads = ("dX", "dDelta", "dA", "dB", "dC", "dD", "d_delta_bias") + (("d_initial_state",) if carried else ()) \
            + (("dZ",) if extras else ())
        back = layer.scan_grad(p, **t, **g, want=grads)
        want = scan_want(p, t, g)
        for k, v in {**got, **back}.items():
            check(v, want[k], f"{k} wide={wide} carried={carried}")
        if lens:
            past_zero(p, {**got, **back}, ("Y", "dX", "dDelta", "dZ", "dB", "dC"), lens)
        same_bits(got, layer.scan(p, **t))
        same_bits(back, layer.scan_grad(p, **t, **g, want=grads))


# lengths on both sides of where sequences are cut into chunks, chunks of every remainder, lengths that end inside,
# at the end and before a chunk
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("seq,batch,channels,state", [(23, 2, 40, 16), (24, 2, 40, 16), (39, 3, 33, 16),
                                                      (40, 3, 33, 16), (41, 1, 130, 4), (43, 2, 24, 64),
                                                      (50, 2, 17, 100), (203, 2, 70, 16), (209, 3, 20, 24)])
def test_scan_around_chunks(layer, seq, batch, channels, state, ragged):
    lens = [[seq - 1, 8, 0][n % 3] for n in range(batch)] if ragged else None
    for dtype, layout in (("f32", 0), ("bf16", 1)):
        p = rk.ScanProblem(seq, batch, channels, state, 1, dtype, layout)
        t, g = scan_inputs(p, seq * state, True, lens)
        if lens:
            poison(p, t, ("X", "Delta", "B", "C", "Z"), lens)
            poison(p, g, ("dY",), lens)
        got = layer.scan(p, **t)
        back = layer.scan_grad(p, **t, **g, want=("dX", "dDelta", "dA", "dB", "dC", "dD", "d_delta_bias",
                                                  "d_initial_state", "dZ"))
        want = scan_want(p, t, g)
        for k, v in {**got, **back}.items():
            check(v, want[k], k)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scan_in_pieces(layer, dtype):
    """A prompt, then single tokens on a state updated in place."""
    N, C, K = 2, 72, 16
    whole = rk.ScanProblem(23, N, C, K, dtype=dtype, layout=1)
    t, _ = scan_inputs(whole, 3, state=False)
    want = scan_want(whole, t)
    rows = {k: t.pop(k) for k in ("X", "Delta", "B", "C", "Z")}

    def piece(a, b, **kw):
        return layer.scan(rk.ScanProblem(b - a, N, C, K, dtype=dtype, layout=1),
                          **{k: v[:, a:b] for k, v in rows.items()}, **t, **kw)
    first = piece(0, 18)
    state, parts = first["final_state"], [first["Y"]]
    for s in range(18, 23):
        parts.append(piece(s, s + 1, initial_state=state, final_state=state)["Y"])
    check(torch.cat(parts, 1), want["Y"], "Y")
    check(state, want["final_state"], "final_state")


def test_scan_state_in_place_over_chunks(layer):
    p = rk.ScanProblem(700, 2, 48, 16, layout=0)
    assert rk.rk_scan_scratch_length(p.to_c()) > 0
    t, _ = scan_inputs(p, 9)
    want = layer.scan(p, **t)
    got = layer.scan(p, **t, final_state=t["initial_state"])
    same_bits(got, want)


def test_scan_decays_to_nothing_and_stands_still(layer):
    """Step sizes that underflow leave the state, ones that overflow the decay
    forget it; neither gives a NaN, in either direction."""
    p = rk.ScanProblem(40, 1, 32, 16)
    t, g = scan_inputs(p, 4)
    t["Delta"][:, :, :16] = -200.0
    t["Delta"][:, :, 16:] = 300.0
    t["delta_bias"].zero_()
    got = layer.scan(p, **t)
    back = layer.scan_grad(p, **t, **g, want=("dX", "dDelta", "dA", "dB", "dC", "dD", "d_delta_bias", "dZ",
                                              "d_initial_state"))
    want = scan_want(p, t, g)
    for k, v in {**got, **back}.items():
        check(v, want[k], k)


def test_scan_no_steps(layer):
    p = rk.ScanProblem(0, 2, 8, 4)
    t, g = scan_inputs(p, 1)
    assert torch.equal(layer.scan(p, **t)["final_state"], t["initial_state"])
    back = layer.scan_grad(p, **t, **g, want=("dX", "dA", "dD", "d_delta_bias", "d_initial_state"))
    assert torch.equal(back["d_initial_state"], g["d_final_state"])
    assert not back["dA"].any() and not back["dD"].any() and not back["d_delta_bias"].any()
    none = rk.ScanProblem(6, 0, 8, 4)
    t, g = scan_inputs(none, 1)
    assert layer.scan(none, **t)["Y"].numel() == 0
    assert not layer.scan_grad(none, **t, **g)["dA"].any()


def test_scan_single_outputs(layer):
    """Any output may be left out."""
    p = rk.ScanProblem(300, 1, 40, 16)
    t, g = scan_inputs(p, 2)
    full = layer.scan(p, **t)
    same_bits(layer.scan(p, **t, want=("final_state",)), dict(final_state=full["final_state"]))
    same_bits(layer.scan(p, **t, want=("Y",)), dict(Y=full["Y"]))
    names = ("dX", "dDelta", "dA", "dB", "dC", "dD", "d_delta_bias", "dZ", "d_initial_state")
    back = layer.scan_grad(p, **t, **g, want=names)
    for n in names:
        same_bits(layer.scan_grad(p, **t, **g, want=(n,)), {n: back[n]})


# ---- streams, graphs, large offsets ---------------------------------------------------------------------

def test_side_stream(layer):
    """A call on a stream of its own, its inputs dropped at once and their
    memory asked for again on the current stream."""
    p = rk.ScanProblem(300, 1, 256, 16)
    t, _ = scan_inputs(p, 7)
    want = layer.scan(p, **t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    copies = {k: v.clone() for k, v in t.items()}
    torch.cuda.synchronize()
    got = layer.scan(p, **copies, stream=side)
    shapes = {k: v.shape for k, v in copies.items()}
    del copies
    for s in shapes.values():
        torch.full(s, float("nan"), device="cuda")
    torch.cuda.current_stream().wait_stream(side)
    same_bits(got, want)


def test_captured_into_a_graph(layer):
    p, q = rk.ScanProblem(300, 1, 64, 16), rk.NormProblem(40, 64)
    t, g = scan_inputs(p, 8)
    x = torch.randn(40, 64, device="cuda")

    def run():
        o = layer.norm(q, x)
        return {**layer.scan(p, **t), **layer.scan_grad(p, **t, **g),
                **layer.norm_grad(q, x, Mean=o["Mean"], InvStdDev=o["InvStdDev"], dY=o["Y"], want=("dScale",))}
    want = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        for v in got.values():
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        same_bits(got, want)


def test_offsets_past_32_bits(layer):
    """Rows 2^30 elements apart: the third starts past 2^31."""
    gap = 2 ** 30
    C = 40
    buf = torch.zeros(2 * gap + 4096, dtype=torch.bfloat16, device="cuda")

    def far(at, inner):
        return torch.as_strided(buf, (3, 1, inner), (gap, gap, 1), at)
    i = Inputs(1, "bf16")
    X, Y, B, Cm = far(0, C), far(64, C), far(128, 16), far(192, 16)
    X.copy_(i.normal(3, 1, C)), B.copy_(i.normal(3, 1, 16)), Cm.copy_(i.normal(3, 1, 16))
    near = {k: v.contiguous() for k, v in dict(X=X, B=B, C=Cm).items()}
    p = rk.ScanProblem(3, 1, C, 16, dtype="bf16")
    args = dict(Delta=i.normal(3, 1, C), A=-torch.rand(C, 16, device="cuda"))
    same_bits(layer.scan(p, X=X, B=B, C=Cm, Y=Y, **args), layer.scan(p, **near, **args))
    q = rk.ConvProblem(3, 1, C, 4, "bf16")
    W = i.normal(C, 4)
    same_bits(layer.conv(q, X=X, W=W, Y=Y), layer.conv(q, X=near["X"], W=W))
    same_bits(layer.conv_grad(q, X=X, W=W, dY=Y, dX=far(256, C)),
              layer.conv_grad(q, X=near["X"], W=W, dY=Y.contiguous()))
    n = rk.NormProblem(3, C, "bf16")
    same_bits(layer.norm(n, X=X[:, 0], Y=Y[:, 0]), layer.norm(n, X=near["X"][:, 0]))


def test_binding_refusals(layer):
    p = rk.NormProblem(4, 8)
    x = torch.zeros(4, 8, device="cuda")
    before = layer.launches()
    with pytest.raises(TypeError):
        layer.norm(p, x.half())
    with pytest.raises(TypeError):
        layer.conv(p, x)
    with pytest.raises(ValueError):
        layer.norm(p, x[:3])
    with pytest.raises(ValueError):
        layer.norm(p, x.cpu())
    with pytest.raises(ValueError):
        layer.norm(p, x, Scale=torch.zeros(8))
    with pytest.raises(ValueError):
        layer.norm(p, x, Scale=torch.zeros(16, device="cuda")[::2])
    with pytest.raises(ValueError):
        layer.norm_grad(p, x, dY=x)
    with pytest.raises(KeyError):
        layer.norm(p, x, Q=x)
    with pytest.raises(KeyError):
        layer.norm(p, x, want=("Q",))
    with pytest.raises(rk.RkError) as e:
        layer.scan(rk.ScanProblem(4, 1, 8, 200), *[torch.zeros(4, 1, 8, device="cuda")],
                   Delta=torch.zeros(4, 1, 8, device="cuda"), A=torch.zeros(8, 200, device="cuda"),
                   B=torch.zeros(4, 1, 200, device="cuda"), C=torch.zeros(4, 1, 200, device="cuda"))
    assert e.value.code == rk.RK_ERR_UNSUPPORTED and "SelectiveScan: state" in e.value.message
    assert layer.launches() == before


# ---- all of them together ----------------------------------------------------------------------------------

def test_example_layer(layer):
    """The example: a layer that is trained through every gradient learns its
    task (to remember inputs; its target has variance 1, which is the loss of
    not learning), and gives token by token what it gives for the whole
    sequence.  The two runs differ in the order of float32 sums of a few
    hundred terms of size 1: 2^-24 * 300 * 10."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "state_space_layer.py")
    spec = importlib.util.spec_from_file_location("state_space_layer_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    first, last, off = example.main(steps=250)
    assert last < 0.5 * first and last < 0.5
    assert off < 2e-4
