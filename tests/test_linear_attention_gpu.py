"""GPU tests of the linear attention operators against their 64-bit definitions.

Tolerance, per element of an output with largest magnitude m: u |r| + 1e-4 m.
u is the unit roundoff of the output's type (half its epsilon: float32 2^-24,
Half 2^-11, bfloat16 2^-8): every output is rounded once.  1e-4 covers float32
arithmetic: an output is a sum over at most 300 steps and 128 elements here,
38400 products whose magnitudes add up to about sqrt(38400) = 196 times the
sum's own size, each off by at most 2^-21 (a decay 2^-22, three roundings of
2^-24 and a sum's): 196 * 2^-21 = 0.94e-4 if all errors were the largest
possible and of one sign.  A head of queries or keys is a sum of at most 256
squares, far below that; its angles are off by 2^-23 at most.  Half outputs
below its smallest normal number are rounded to multiples of 2^-24.
Past a row's length outputs are exactly 0, and everything is bit-identical
between runs.
"""
import numpy as np
import pytest
import torch

import linear_attention_reference as ref
import onnx_lstm_gru_gb300 as rk

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


def check(got, want, name="", arithmetic=1e-4, absolute=0.0):
    want = want.to(F64)
    g = got.double().cpu()
    assert g.shape == want.shape, name
    if not want.numel():
        return
    assert torch.equal(torch.isnan(g), torch.isnan(want)), f"{name}: NaN elsewhere"
    fine = torch.isfinite(want)
    assert torch.equal(g[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{name}: infinite elsewhere"
    g, want = g[fine], want[fine]
    if not want.numel():
        return
    top = float(want.abs().max())
    # below its smallest normal number a type has multiples of one step (half of it is lost), or 0 in its place
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -126
    bound = UNIT[got.dtype] * want.abs() + arithmetic * top + tiny + absolute
    off = (g - want).abs()
    assert bool((off <= bound).all()), f"{name}: off by {float((off - bound).max()):.3g} beyond the bound, largest {top:.3g}"


def bits(out):
    return {k: v.contiguous().cpu().view(torch.uint8) for k, v in out.items()}


def same_bits(a, b):
    a, b = bits(a), bits(b)
    assert a.keys() == b.keys()
    for k in a:
        assert torch.equal(a[k], b[k]), k


class Inputs:
    """Seeded inputs; rows in either layout, and wide: as slices of wider ones with NaN around them."""

    def __init__(self, seed, dtype, layout=0, wide=False):
        self.rng = np.random.default_rng(seed)
        self.t = rk.torch_dtype(dtype)
        self.layout, self.wide = layout, wide

    def normal(self, *shape, scale=1.0, mean=0.0, dtype=None):
        return torch.from_numpy(self.rng.normal(mean, scale, shape)).to(dtype or self.t).cuda()

    def rows(self, S, N, width, **kw):
        shape = (S, N, width) if self.layout == 0 else (N, S, width)
        x = self.normal(*shape, **kw)
        if not self.wide:
            return x
        at = int(self.rng.integers(0, 9))
        wide = torch.full(shape[:-1] + (width + 8 + int(self.rng.integers(0, 2)),), float("nan"), dtype=x.dtype,
                          device="cuda")
        wide[..., at:at + width] = x
        return wide[..., at:at + width]


def batch_first(x, layout):
    x = x.double().cpu() if x.is_floating_point() else x.cpu()
    return x.transpose(0, 1) if layout == 0 else x


def dead_steps_are_zero(x, layout, lens):
    x = x.cpu().transpose(0, 1) if layout == 0 else x.cpu()
    for n, L in enumerate(lens):
        assert not x[n, max(L, 0):].float().abs().any()


# ---- queries and keys ------------------------------------------------------------------------------

#       S, N, heads, key_heads, size, rotary, interleaved, norm
QK_SHAPES = [
    (1, 1, 1, 1, 1, 0, False, "rms"), (1, 3, 2, 1, 2, 2, True, "l2"), (5, 2, 4, 2, 8, 8, False, "rms"),
    (3, 4, 16, 4, 128, 128, False, "rms"), (3, 4, 16, 4, 128, 128, True, "rms"), (7, 2, 3, 3, 64, 32, False, "none"),
    (9, 3, 6, 3, 90, 34, True, "l2"), (9, 3, 6, 3, 90, 34, False, "rms"), (4, 2, 5, 1, 72, 72, False, "rms"),
    (4, 2, 2, 2, 256, 256, False, "l2"), (2, 3, 3, 2, 255, 130, True, "rms"), (2, 2, 9, 3, 48, 0, False, "rms"),
    (2, 2, 40, 8, 16, 16, True, "rms"), (6, 3, 2, 7, 12, 4, False, "rms"), (2, 1, 3, 1, 24, 16, False, "rms"),
    (2, 1, 3, 1, 4, 4, False, "none"), (130, 40, 4, 4, 32, 32, False, "rms"),
]


def qk_case(shape, dtype, layout, wide, seed, positions=None, ragged=True):
    S, N, H, KH, d, r, il, norm = shape
    i = Inputs(seed, dtype, layout, wide)
    p = rk.QkProblem(seq=S, batch=N, heads=H, key_heads=KH, size=d, rotary=r, interleaved=il, norm=norm, epsilon=1e-3,
                     dtype=dtype, layout=layout)
    t = dict(Q=i.rows(S, N, H * d), K=i.rows(S, N, KH * d), QScale=i.normal(d, mean=1.0, scale=0.3),
             KScale=i.normal(d, mean=1.0, scale=0.3))
    if r:
        t["Frequencies"] = torch.exp(torch.linspace(0, -9, r // 2)).cuda()
    lens = [int(x) for x in i.rng.integers(0, S + 1, N)]
    if ragged:
        t["sequence_lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    if positions is not None:
        t["positions"] = positions((S, N) if layout == 0 else (N, S), i.rng)
    return i, p, t, lens if ragged else None


def qk_reference(p, t, lens, side, dY=None):
    b = {k: batch_first(t[k], p.layout) for k in ("Q", "K", "positions") if t.get(k) is not None}
    f = {k: t[k].double().cpu() for k in ("QScale", "KScale", "Frequencies") if t.get(k) is not None}
    return ref.qk(b[side], p.heads if side == "Q" else p._key_heads, f.get(side + "Scale"), f.get("Frequencies"),
                  b.get("positions"), lens, p.rotary, p.interleaved, p.norm, p.epsilon, dY)


def cancelled(p, t, lens, side, dY):
    """dX = inv g - x inv^3 sum(g x) / m is a difference of two terms, of which
    the second is no larger than sqrt(size) times the first's largest
    (Cauchy-Schwarz: |x| inv is at most sqrt(m), |g| at most sqrt(size) of its
    largest).  A head of one element, or of one large one, leaves far less than
    the terms have, and of those each is off by its own float32 roundings, at
    most eight of 2^-24."""
    if p.norm == "none":
        return 0.0
    b = batch_first(t[side], p.layout).unflatten(-1, (-1, p.size))
    b = torch.where(ref._live(lens, *b.shape[:2])[..., None, None], b, torch.zeros((), dtype=F64))
    m = p.size if p.norm == "rms" else 1
    inv = ((b * b).sum(-1) / m + p.epsilon) ** -0.5
    w = t[side + "Scale"].abs().max().item() if t.get(side + "Scale") is not None else 1.0
    live = torch.where(ref._live(lens, *b.shape[:2])[..., None], dY, torch.zeros((), dtype=F64))
    # a turned pair's elements are at most sqrt(2) of its largest
    return 8 * 2.0 ** -24 * p.size ** 0.5 * 2 ** 0.5 * w * float(inv.max()) * float(live.abs().max())


def near(shape, rng):
    return torch.from_numpy(rng.integers(-50, 5000, shape).astype(np.int32)).cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", QK_SHAPES)
def test_qk(layer, shape, dtype):
    for layout, wide, positions in ((0, False, None), (1, False, near), (0, True, near), (1, True, None)):
        i, p, t, lens = qk_case(shape, dtype, layout, wide, sum(shape[:6]), positions, ragged=layout == 1)
        got = layer.qk(p, **t)
        for side in "QK":
            check(batch_first(got["Y" + side], layout).to(got["YQ"].dtype), qk_reference(p, t, lens, side),
                  f"Y{side} {layout} {wide}")
            if lens:
                dead_steps_are_zero(got["Y" + side], layout, lens)
        same_bits(got, layer.qk(p, **t))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", QK_SHAPES)
def test_qk_grad(layer, shape, dtype):
    for layout, wide, positions in ((0, False, None), (1, False, near), (0, True, near), (1, True, None)):
        i, p, t, lens = qk_case(shape, dtype, layout, wide, 7 + sum(shape[:6]), positions, ragged=layout == 1)
        S, N, H, KH, d = shape[:5]
        t.update(dYQ=i.rows(S, N, H * d), dYK=i.rows(S, N, KH * d))
        got = layer.qk_grad(p, **t)
        for side in "QK":
            dY = batch_first(t["dY" + side], layout)
            dX, dScale = qk_reference(p, t, lens, side, dY)
            check(batch_first(got["d" + side], layout).to(got["dQ"].dtype), dX, f"d{side} {layout} {wide}",
                  absolute=cancelled(p, t, lens, side, dY))
            check(got[f"d{side}Scale"], dScale, f"d{side}Scale {layout} {wide}")
            if lens:
                dead_steps_are_zero(got["d" + side], layout, lens)
        same_bits(got, layer.qk_grad(p, **t))


def test_qk_without_scales(layer):
    i, p, t, lens = qk_case((5, 3, 4, 2, 32, 16, False, "rms"), "f32", 0, False, 3)
    t["QScale"] = t["KScale"] = None
    got = layer.qk(p, **t)
    check(batch_first(got["YQ"], 0).float(), qk_reference(p, t, lens, "Q"))
    t.update(dYQ=i.rows(5, 3, 128), dYK=i.rows(5, 3, 64))
    got = layer.qk_grad(p, **t)
    dX, dScale = qk_reference(p, t, lens, "K", batch_first(t["dYK"], 0))
    check(batch_first(got["dK"], 0).float(), dX)
    check(got["dKScale"], dScale)
    assert layer.qk_grad(p, want=("dK",), **t).keys() == {"dK"}
    assert layer.qk(p, want=("YQ",), **t_of_qk(t)).keys() == {"YQ"}


def t_of_qk(t):
    return {k: v for k, v in t.items() if not k.startswith("dY")}


@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_far_positions(layer, interleaved):
    """Angles of positions up to 2^31 are as exact as those of near ones:
    frequency and turn are products of whole numbers that wrap at a turn, off
    by the frequency's 2^-53 times the position, 2^-22 of a radian times the
    frequency at most."""
    def far(shape, rng):
        x = rng.integers(-2 ** 31, 2 ** 31, shape)
        return torch.from_numpy(x.astype(np.int32)).cuda()
    i, p, t, lens = qk_case((17, 3, 2, 2, 64, 64, interleaved, "none"), "f32", 0, False, 5, far, ragged=False)
    t["Frequencies"] = torch.cat([torch.tensor([1.0, 3.0, 0.7, -0.3, 100.0, 0.0]), torch.exp(torch.linspace(0, -12, 26))]).cuda()
    got = layer.qk(p, **t)
    for side in "QK":
        check(batch_first(got["Y" + side], 0).float(), qk_reference(p, t, None, side))


def test_qk_frequencies_that_are_no_numbers(layer):
    """Their pairs are NaN, the others not; past the rows' ends all is 0."""
    i, p, t, lens = qk_case((4, 2, 2, 1, 16, 8, False, "rms"), "f32", 0, False, 5)
    t["Frequencies"] = torch.tensor([1.0, float("nan"), float("inf"), 0.5]).cuda()
    t["sequence_lens"] = torch.tensor([4, 2], dtype=torch.int32).cuda()
    y = batch_first(layer.qk(p, **t)["YQ"], 0).reshape(2, 4, 2, 16)
    bad = torch.zeros(16, dtype=torch.bool)
    bad[[1, 2, 5, 6]] = True
    assert torch.equal(torch.isnan(y[0]), bad.expand(4, 2, 16))
    assert not y[1, 2:].any()


def test_qk_no_rows(layer):
    for S, N in ((0, 3), (3, 0)):
        p = rk.QkProblem(seq=S, batch=N, heads=2, size=16, rotary=8, dtype="bf16")
        x = torch.zeros(S, N, 32, dtype=torch.bfloat16, device="cuda")
        f = torch.ones(4, device="cuda")
        assert layer.qk(p, x, K=x, Frequencies=f)["YQ"].shape == (S, N, 32)
        g = layer.qk_grad(p, x, K=x, dYQ=x, dYK=x, Frequencies=f)
        assert not g["dQScale"].any() and not g["dKScale"].any()


def test_qk_large_values_do_not_overflow(layer):
    """Heads of about 1e-12 with no epsilon have an inverse whose cube is beyond float32's range."""
    p = rk.QkProblem(seq=2, batch=2, heads=2, size=8, norm="l2", epsilon=0.0)
    i = Inputs(3, "f32")
    t = dict(Q=i.rows(2, 2, 16, scale=1e-14), K=i.rows(2, 2, 16, scale=1e15), dYQ=i.rows(2, 2, 16, scale=1e-10),
             dYK=i.rows(2, 2, 16))
    got = layer.qk_grad(p, **t)
    for side in "QK":
        dX, _ = qk_reference(p, t, None, side, batch_first(t["dY" + side], 0))
        check(batch_first(got["d" + side], 0).float(), dX)


#       heads of pieces of two elements and of one, of several units a lane; many turns a warp
QK_MORE = [
    (3, 2, 3, 2, 256, 252, False, "rms"), (3, 2, 3, 2, 254, 254, True, "rms"), (2, 2, 2, 2, 130, 64, True, "l2"),
    (2, 2, 3, 1, 100, 50, False, "l2"), (3, 3, 5, 2, 255, 100, False, "rms"), (30, 64, 40, 8, 16, 16, True, "rms"),
    (40, 64, 3, 9, 62, 62, False, "rms"), (300, 20, 2, 1, 33, 30, True, "l2"),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", QK_MORE)
def test_qk_pieces_and_turns(layer, shape, dtype):
    S, N, H, KH, d = shape[:5]
    for layout, wide, positions in ((0, False, None), (1, False, near), (1, True, None)):
        i, p, t, lens = qk_case(shape, dtype, layout, wide, sum(shape[:6]), positions)
        got = layer.qk(p, **t)
        for side in "QK":
            check(batch_first(got["Y" + side], layout).to(got["YQ"].dtype), qk_reference(p, t, lens, side), f"Y{side}")
        t.update(dYQ=i.rows(S, N, H * d), dYK=i.rows(S, N, KH * d))
        got = layer.qk_grad(p, **t)
        for side in "QK":
            dY = batch_first(t["dY" + side], layout)
            dX, dScale = qk_reference(p, t, lens, side, dY)
            check(batch_first(got["d" + side], layout).to(got["dQ"].dtype), dX, f"d{side}",
                  absolute=cancelled(p, t, lens, side, dY))
            check(got[f"d{side}Scale"], dScale, f"d{side}Scale")
        same_bits(got, layer.qk_grad(p, **t))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(40, 64, 6, 3, 64, 32, False, "rms"), (9, 3, 6, 3, 90, 34, True, "l2")])
def test_qk_in_place(layer, shape, dtype):
    """Results may take the operands' place."""
    i, p, t, lens = qk_case(shape, dtype, 0, False, 3)
    want = {k: v.clone() for k, v in layer.qk(p, **t).items()}
    q, k = t["Q"].clone(), t["K"].clone()
    got = layer.qk(p, **dict(t, Q=q, K=k), YQ=q, YK=k)
    assert got["YQ"] is q and got["YK"] is k
    same_bits(got, want)


def test_qk_on_streams_and_in_graphs(layer):
    i, p, t, lens = qk_case((50, 8, 4, 2, 64, 64, False, "rms"), "bf16", 1, False, 5, near)
    g = dict(t, dYQ=i.rows(50, 8, 256), dYK=i.rows(50, 8, 128))
    want, gwant = layer.qk(p, **t), layer.qk_grad(p, **g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = layer.qk(p, stream=side, **t), layer.qk_grad(p, stream=side, **g)
    torch.cuda.current_stream().wait_stream(side)
    same_bits(a, want)
    same_bits(b, gwant)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = layer.qk(p, **t), layer.qk_grad(p, **g)
    for _ in range(2):
        for x in ("Q", "K", "positions"):
            t[x].copy_(i.rng.integers(0, 99) if x == "positions" else torch.randn_like(t[x].float()))
        graph.replay()
        torch.cuda.synchronize()
        same_bits(a, layer.qk(p, **t))
        same_bits(b, layer.qk_grad(p, **g))


# ---- attention ---------------------------------------------------------------------------------------

class Case:
    def __init__(self, S, N, H, dk, dv, dtype, layout=0, q=None, k=None, v=None, decay="rows", state=True, ragged=True,
                 wide=False, seed=0, lens=None, scale=None, grad=False):
        i = self.i = Inputs(seed + 7 * S + N + H + dk + dv, dtype, layout, wide)
        q, k, v = q or H, k or H, v or H
        p = self.p = rk.AttnProblem(seq=S, batch=N, heads=H, key_size=dk, value_size=dv, query_heads=q, key_heads=k,
                                    value_heads=v, dtype=dtype, layout=layout, scale=scale)
        t = self.t = dict(Q=i.rows(S, N, q * dk), K=i.rows(S, N, k * dk), V=i.rows(S, N, v * dv))
        if decay in ("rows", "both"):
            t["Decay"] = -torch.nn.functional.softplus(i.rows(S, N, H, scale=1.5, mean=-2.0, dtype=torch.float32))
            if wide:
                t["Decay"] = torch.nn.functional.pad(t["Decay"], (3, 2), value=float("nan"))[..., 3:-2]
        if decay in ("bias", "both"):
            t["decay_bias"] = -torch.exp2(-i.normal(H, dtype=torch.float32).abs() * 4)
        if state:
            t["initial_state"] = i.normal(N, H, dk, dv, dtype=torch.float32)
        self.lens = lens if lens is not None else [int(x) for x in i.rng.integers(0, S + 1, N)] if ragged else None
        if self.lens is not None:
            t["sequence_lens"] = torch.tensor(self.lens, dtype=torch.int32).cuda()
        if grad:
            t["dY"] = i.rows(S, N, H * dv)
            if state:
                t["d_final_state"] = i.normal(N, H, dk, dv, dtype=torch.float32)

    def reference(self):
        p, t = self.p, self.t
        scale = p.scale if p.scale is not None else p.key_size ** -0.5
        b = {k: batch_first(t[k], p.layout) for k in ("Q", "K", "V", "Decay", "dY") if t.get(k) is not None}
        f = {k: t[k].double().cpu() for k in ("decay_bias", "initial_state", "d_final_state") if t.get(k) is not None}
        return ref.attn(heads=p.heads, scale=scale, key_size=p.key_size, value_size=p.value_size, lens=self.lens, **b,
                        **f)

    def compare(self, got, name=""):
        want = self.reference()
        for k, v in got.items():
            x = batch_first(v, self.p.layout).to(v.dtype) if k in ("Y", "dQ", "dK", "dV", "dDecay") else v
            check(x, want[k], f"{k} {name}", absolute=self.summed(want, k))
            if self.lens is not None and k in ("Y", "dQ", "dK", "dV", "dDecay"):
                dead_steps_are_zero(v, self.p.layout, self.lens)

    def summed(self, want, name):
        """dDecay is a running sum of k dk - q dq over a row's steps, of which
        little may be left; each of those products of 128 elements at most is
        off by at most 16 roundings of 2^-24 of its terms' magnitudes."""
        if name not in ("dDecay", "d_decay_bias"):
            return 0.0
        p = self.p
        N, S = p.batch, p.seq
        sizes = []
        for x, dx in (("Q", "dQ"), ("K", "dK")):
            a = batch_first(self.t[x], p.layout)
            a = torch.where(ref._live(self.lens, N, S)[..., None], a, torch.zeros((), dtype=F64))
            sizes.append((a.abs() * want[dx].abs()).sum(-1).sum(1))
        off = 16 * 2.0 ** -24 * (sizes[0] + sizes[1])
        return float(off.max() if name == "dDecay" else off.sum() * S)

    def grads(self):
        return ("dQ", "dK", "dV") + (("dDecay",) if "Decay" in self.t else ()) + \
            (("d_decay_bias",) if "decay_bias" in self.t else ()) + ("d_initial_state",)


#             S, N, H, dk, dv
ATTN_SHAPES = [
    (1, 1, 1, 1, 1), (1, 5, 3, 128, 128), (1, 2, 4, 64, 64), (1, 3, 2, 7, 33), (2, 3, 2, 5, 3), (15, 2, 2, 64, 64),
    (16, 2, 1, 128, 64), (17, 3, 2, 64, 128), (31, 1, 2, 32, 32), (33, 1, 2, 24, 40), (63, 2, 2, 128, 128),
    (64, 2, 2, 64, 64), (65, 2, 2, 128, 128), (80, 3, 4, 72, 103), (128, 1, 2, 128, 128), (129, 2, 1, 65, 66),
    (200, 2, 3, 48, 80), (300, 1, 2, 128, 128), (257, 1, 1, 127, 1), (130, 2, 2, 1, 127),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", ATTN_SHAPES)
def test_attn(layer, shape, dtype):
    for layout, decay, state, ragged, wide in ((0, "rows", False, False, False), (1, "both", True, True, False),
                                               (0, "bias", True, False, True), (1, "none", False, True, True)):
        c = Case(*shape, dtype, layout=layout, decay=decay, state=state, ragged=ragged, wide=wide)
        got = layer.attn(c.p, **c.t)
        c.compare(got, f"{layout} {decay} {wide}")
        same_bits(got, layer.attn(c.p, **c.t))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", ATTN_SHAPES)
def test_attn_grad(layer, shape, dtype):
    for layout, decay, state, ragged, wide in ((0, "rows", False, False, False), (1, "both", True, True, False),
                                               (0, "bias", True, False, True), (1, "rows", False, True, True)):
        c = Case(*shape, dtype, layout=layout, decay=decay, state=state, ragged=ragged, wide=wide, grad=True)
        got = layer.attn_grad(c.p, want=c.grads(), **c.t)
        c.compare(got, f"{layout} {decay} {wide}")
        same_bits(got, layer.attn_grad(c.p, want=c.grads(), **c.t))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("q,k,v", [(2, 2, 4), (4, 1, 1), (4, 2, 1), (1, 4, 2), (1, 1, 1)])
def test_attn_shared_heads(layer, q, k, v, dtype):
    for S in (3, 70):
        c = Case(S, 2, 4, 48, 40, dtype, q=q, k=k, v=v, decay="both", grad=True, layout=S % 2)
        c.compare(layer.attn_grad(c.p, want=c.grads(), **c.t))
        for n in ("dY", "d_final_state"):
            c.t.pop(n)
        c.compare(layer.attn(c.p, **c.t))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S", [700, 1500])
def test_attn_long(layer, S, dtype):
    """One sequence and a batch, long enough to be cut into pieces that run
    side by side.  The decays here keep at most some hundred steps in sight,
    so the bound of the shorter ones holds."""
    for N, H in ((1, 2), (3, 2)):
        c = Case(S, N, H, 64, 48, dtype, ragged=N > 1, layout=N % 2, grad=True)
        c.compare(layer.attn_grad(c.p, want=c.grads(), **c.t))
        for n in ("dY", "d_final_state"):
            c.t.pop(n)
        c.compare(layer.attn(c.p, **c.t))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_in_pieces_and_token_by_token(layer, dtype):
    """A prompt, the same in pieces, and its last steps as single tokens with
    the state updated in place: the recurrence is the same one."""
    S, N, H, dk, dv = 150, 3, 2, 64, 128
    c = Case(S, N, H, dk, dv, dtype, ragged=False, decay="both")
    c.compare(layer.attn(c.p, **c.t))
    want = c.reference()
    state = c.t["initial_state"].clone()
    ys = []
    for a, b in ((0, 70), (70, 71), (71, 145), *((s, s + 1) for s in range(145, 150))):
        p = rk.AttnProblem(seq=b - a, batch=N, heads=H, key_size=dk, value_size=dv, dtype=dtype)
        t = {k: c.t[k][a:b] for k in ("Q", "K", "V", "Decay")}
        out = layer.attn(p, decay_bias=c.t["decay_bias"], initial_state=state, final_state=state, **t)
        assert out["final_state"] is state
        ys.append(out["Y"])
    y = torch.cat(ys)
    check(batch_first(y, 0).to(y.dtype), want["Y"], "Y in pieces")
    check(state, want["final_state"], "state in pieces")


@pytest.mark.parametrize("dtype", DTYPES)
def test_attn_documents_in_a_row(layer, dtype):
    """A decay of minus infinity forgets: what follows is as if it came first."""
    for S, cut in ((3, 1), (140, 70), (140, 64)):
        c = Case(S, 2, 2, 32, 24, dtype, ragged=False, state=True, layout=1, grad=True)
        c.t["Decay"][:, cut] = -float("inf")
        c.t["Decay"][:, S - 1] = -float("inf")
        got = layer.attn_grad(c.p, want=c.grads(), **c.t)
        c.compare(got)
        c.t.pop("dY"), c.t.pop("d_final_state")
        fwd = c.t
        got = layer.attn(c.p, **fwd)
        c.compare(got)
        other = dict(fwd, initial_state=torch.randn_like(fwd["initial_state"]))
        assert torch.equal(layer.attn(c.p, **other)["Y"][:, cut:], got["Y"][:, cut:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S", [5, 100])
def test_attn_strong_and_mixed_decays(layer, dtype, S):
    """Decays far beyond what a chunk's product can hold beside ones that keep all."""
    c = Case(S, 2, 3, 40, 48, dtype, ragged=False, layout=1, grad=True)
    g = c.t["Decay"]
    g[:, ::3] = -300.0
    g[:, 1::3] = 0.0
    g[0, 2::5] = -40.0
    c.compare(layer.attn_grad(c.p, want=c.grads(), **c.t))
    c.t.pop("dY"), c.t.pop("d_final_state")
    c.compare(layer.attn(c.p, **c.t))


@pytest.mark.parametrize("dtype", DTYPES)
def test_attn_growing_states(layer, dtype):
    """Decays above 0 are growth."""
    c = Case(100, 2, 2, 32, 32, dtype, ragged=False, layout=1, grad=True)
    c.t["Decay"].copy_(c.i.normal(2, 100, 2, scale=0.3, dtype=torch.float32))
    c.compare(layer.attn_grad(c.p, want=c.grads(), **c.t))
    c.t.pop("dY"), c.t.pop("d_final_state")
    c.compare(layer.attn(c.p, **c.t))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["Q", "K", "V", "Decay", "initial_state"])
def test_attn_numbers_that_are_none_reach_later_steps_only(layer, dtype, name):
    for S, at in ((4, 2), (150, 100)):
        c = Case(S, 2, 2, 48, 64, dtype, ragged=False, layout=1)
        clean = layer.attn(c.p, **c.t)["Y"].clone()
        x = c.t[name]
        if name == "initial_state":
            x[0, 0, 3, 5] = float("nan")
        else:
            x[0, at, 0] = float("nan")
        # NaN exactly where the definition has it: not in earlier steps, not in the other heads; the steps around
        # it are taken one by one, so their rounding is another one than without it
        got = layer.attn(c.p, **c.t)
        c.compare(got)
        assert torch.equal(got["Y"][1], clean[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_products_beyond_float32(layer, dtype):
    """Queries and keys whose products pass float32's range while the states
    and outputs, with values that small, do not."""
    c = Case(90, 1, 1, 32, 32, dtype, ragged=False, state=False, layout=1)
    c.t["Q"].mul_(1e20), c.t["K"].mul_(1e20), c.t["V"].mul_(1e-22)
    got = layer.attn(c.p, **c.t)
    assert torch.isfinite(got["Y"]).all()
    c.compare(got)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attn_operands_past_the_ends_are_not_used(layer, dtype):
    for S in (6, 90):
        c = Case(S, 3, 2, 32, 40, dtype, lens=[S - 2, 0, S + 9], layout=1, grad=True, decay="both")
        for n in ("Q", "K", "V", "Decay", "dY"):
            c.t[n][0, S - 2:] = float("nan")
            c.t[n][1] = float("inf")
        c.compare(layer.attn_grad(c.p, want=c.grads(), **c.t))
        c.t.pop("dY"), c.t.pop("d_final_state")
        c.compare(layer.attn(c.p, **c.t))


def cut(c):
    """Whether the case's sequences are cut into pieces that run side by side."""
    return rk.rk_attn_scratch_length(c.p.to_c()) > 0


def both_ways(layer, c, name=""):
    """Gradient and outputs against the definition."""
    c.compare(layer.attn_grad(c.p, want=c.grads(), **c.t), name)
    for n in ("dY", "d_final_state"):
        c.t.pop(n, None)
    c.compare(layer.attn(c.p, **c.t), name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", [(64, 48), (128, 128), (72, 30)])
def test_attn_documents_and_strong_decays_in_pieces(layer, sizes, dtype):
    """Forgetting and decays beyond a chunk's product, at and off the pieces'
    and chunks' ends, in sequences that are cut."""
    c = Case(700, 1, 2, *sizes, dtype, ragged=False, layout=1, grad=True)
    assert cut(c)
    g = c.t["Decay"]
    for at in (0, 63, 64, 65, 128, 300, 383, 448, 699):
        g[:, at, 0] = -float("inf")
    g[:, 200:260, 1] = -300.0
    g[:, 500:520:2, 1] = -90.0
    both_ways(layer, c)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["Q", "K", "V", "Decay", "initial_state"])
def test_attn_numbers_that_are_none_in_pieces(layer, dtype, name):
    for at in (70, 640):
        c = Case(700, 1, 3, 64, 64, dtype, ragged=False, layout=0)
        assert cut(c)
        clean = layer.attn(c.p, **c.t)
        x = c.t[name]
        if name == "initial_state":
            x[0, 1, 3, 5] = float("inf")
        else:
            x[at, 0, 0] = float("nan")
        got = layer.attn(c.p, **c.t)
        c.compare(got)
        # the head that goes with it may be rounded another way, as what the two share is taken step by step
        assert torch.equal(got["Y"][:, 0, 128:], clean["Y"][:, 0, 128:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_products_beyond_float32_in_pieces(layer, dtype):
    c = Case(700, 1, 1, 32, 32, dtype, ragged=False, state=False, layout=1)
    assert cut(c)
    c.t["Q"].mul_(1e20), c.t["K"].mul_(1e20), c.t["V"].mul_(1e-22)
    got = layer.attn(c.p, **c.t)
    assert torch.isfinite(got["Y"]).all()
    c.compare(got)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attn_growth_in_pieces(layer, dtype):
    """Decays of either sign: their sums stay within a few units."""
    c = Case(700, 1, 2, 32, 32, dtype, ragged=False, layout=1, grad=True)
    assert cut(c)
    c.t["Decay"].copy_(c.i.normal(1, 700, 2, scale=0.3, mean=-0.05, dtype=torch.float32))
    both_ways(layer, c)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attn_ragged_rows_in_pieces(layer, dtype):
    """Rows that end in the first piece, at a piece's end and past all."""
    c = Case(900, 5, 1, 48, 64, dtype, lens=[0, 1, 64, 899, 2000], layout=0, grad=True, decay="both")
    assert cut(c)
    both_ways(layer, c)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,H,dk,dv", [(6, 3, 64, 32), (6, 1, 128, 72), (60, 3, 24, 16)])
def test_attn_rows_that_end_where_sums_start_anew(layer, N, H, dk, dv, dtype):
    """The decays' gradient takes the state's product with its gradient every
    512 steps; rows end before, at and behind, in sequences cut and not."""
    lens = ([512, 513, 1024, 1030, 511, 0] * 10)[:N]
    both_ways(layer, Case(1030, N, H, dk, dv, dtype, lens=lens, layout=N % 2, decay="both", grad=True))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", [(3, 3, 3), (5, 1, 5), (3, 3, 1)])
def test_attn_heads_that_do_not_pair(layer, heads, dtype):
    """Heads of at most 64 elements go in pairs; of an odd number one goes alone."""
    H, q, k = heads
    for S, wide in ((70, False), (300, True)):
        both_ways(layer, Case(S, 2, H, 64, 32, dtype, q=q, k=k, v=k, decay="both", layout=1, wide=wide, grad=True))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S", [11, 12, 13, 14])
def test_attn_between_steps_and_chunks(layer, S, dtype):
    both_ways(layer, Case(S, 3, 2, 128, 96, dtype, decay="both", layout=S % 2, grad=True))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("at,extra", [(8, 8), (0, 16), (1, 8), (4, 4)])
def test_attn_slices_of_wider_rows(layer, at, extra, dtype):
    """Queries, keys and values as one projection's row holds them, on 16-byte
    boundaries and off them."""
    S, N, H, dk, dv = 200, 2, 2, 64, 128
    c = Case(S, N, H, dk, dv, dtype, layout=0, ragged=False, grad=True)
    width = 2 * H * dk + H * dv + at + extra
    row = torch.full((S, N, width), float("nan"), dtype=c.t["Q"].dtype, device="cuda")
    for n, w in (("Q", H * dk), ("K", H * dk), ("V", H * dv)):
        row[..., at:at + w] = c.t[n]
        c.t[n] = row[..., at:at + w]
        at += w
    both_ways(layer, c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_rows_far_apart(layer, dtype):
    """Offsets beyond 32 bits."""
    S, N, H, d = 20, 1, 2, 64
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    c = Case(S, N, H, d, d, dtype, layout=0, ragged=False, grad=True)
    far = torch.empty(S, 1, 2 ** 27 + 512, dtype=c.t["Q"].dtype, device="cuda")
    assert far.numel() > 2 ** 31
    at = 0
    for n in ("Q", "K", "V", "dY"):
        far[..., at:at + H * d] = c.t[n]
        c.t[n] = far[..., at:at + H * d]
        at += H * d
    both_ways(layer, c)
    p = rk.QkProblem(seq=S, batch=N, heads=H, size=d, norm="l2", dtype=dtype)
    near_, far_ = ({k: f(c.t[k]) for k in ("Q", "K")} for f in (torch.Tensor.contiguous, lambda x: x))
    same_bits(layer.qk(p, **far_), layer.qk(p, **near_))


def test_attn_no_decay_keeps_all(layer):
    """Without decays the state is the sum over all steps: 700 of 128 elements
    here, sqrt(89600) * 2^-21 by the reckoning at the top."""
    c = Case(700, 1, 2, 128, 64, "f32", decay="none", ragged=False)
    assert cut(c)
    got, want = layer.attn(c.p, **c.t), c.reference()
    for k in got:
        check(batch_first(got[k], 0).float() if k == "Y" else got[k], want[k], k, arithmetic=1.5e-4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 1e-12, -3.0, 1e30, 0.0])
def test_attn_scales_of_any_size(layer, scale, dtype):
    """Decays of 2^-92 over a chunk and a scale that is far from 1 itself."""
    c = Case(130, 1, 2, 64, 48, dtype, ragged=False, scale=scale, grad=True, layout=1)
    c.t["Decay"].fill_(-1.0)
    both_ways(layer, c)


def test_attn_state_in_place_in_pieces(layer):
    c = Case(900, 1, 2, 64, 64, "bf16", ragged=False, decay="both")
    assert cut(c)
    want = layer.attn(c.p, **c.t)
    state = c.t["initial_state"].clone()
    got = layer.attn(c.p, **dict(c.t, initial_state=state), final_state=state)
    assert got["final_state"] is state
    same_bits(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(513, 40, 4, 64, 64), (513, 20, 4, 128, 128), (700, 1, 4, 128, 64)])
def test_attn_many_calls_in_a_row(layer, shape, dtype):
    """The same bits every time, and no wait that gave up."""
    c = Case(*shape, dtype, decay="both", grad=True)
    f = {k: v for k, v in c.t.items() if k not in ("dY", "d_final_state")}
    want, gwant = layer.attn(c.p, **f), layer.attn_grad(c.p, want=c.grads(), **c.t)
    for _ in range(12):
        outs = [(layer.attn(c.p, **f), layer.attn_grad(c.p, want=c.grads(), **c.t)) for _ in range(3)]
        for a, b in outs:
            for k, v in want.items():
                assert torch.equal(a[k], v), k
            for k, v in gwant.items():
                assert torch.equal(b[k], v), k
    assert rk.rk_status_poll(layer.handle, torch.cuda.current_stream().cuda_stream) == rk.RK_OK


def test_attn_no_steps(layer):
    p = rk.AttnProblem(seq=0, batch=2, heads=3, key_size=8, value_size=4, dtype="f16")
    z = torch.zeros(0, 2, 24, dtype=torch.float16, device="cuda")
    v = torch.zeros(0, 2, 12, dtype=torch.float16, device="cuda")
    h = torch.randn(2, 3, 8, 4, device="cuda")
    out = layer.attn(p, z, K=z, V=v, initial_state=h)
    assert torch.equal(out["final_state"], h) and out["Y"].shape == (0, 2, 12)
    assert not layer.attn(p, z, K=z, V=v)["final_state"].any()
    g = layer.attn_grad(p, z, K=z, V=v, dY=v, d_final_state=h, want=("dQ", "d_decay_bias", "d_initial_state"))
    assert torch.equal(g["d_initial_state"], h) and not g["d_decay_bias"].any()
    p = rk.AttnProblem(seq=4, batch=0, heads=3, key_size=8, value_size=4, dtype="f16")
    z, v = torch.zeros(4, 0, 24, dtype=torch.float16, device="cuda"), torch.zeros(4, 0, 12, dtype=torch.float16, device="cuda")
    assert layer.attn(p, z, K=z, V=v)["Y"].shape == (4, 0, 12)
    g = layer.attn_grad(p, z, K=z, V=v, dY=v, want=("dQ", "d_decay_bias"))
    assert not g["d_decay_bias"].any()


def test_attn_wanted_alone(layer):
    """Each output by itself is what it is among the others."""
    c = Case(130, 2, 4, 40, 32, "bf16", q=2, k=2, decay="both", grad=True)
    names = c.grads()
    every = layer.attn_grad(c.p, want=names, **c.t)
    for n in names:
        same_bits({n: every[n]}, layer.attn_grad(c.p, want=(n,), **c.t))
    c.t.pop("dY"), c.t.pop("d_final_state")
    every = layer.attn(c.p, **c.t)
    for n in every:
        same_bits({n: every[n]}, layer.attn(c.p, want=(n,), **c.t))


def test_attn_outputs_into_slices(layer):
    """Outputs are written where their rows are and nowhere else."""
    S, N, H, dk, dv = 70, 2, 2, 24, 40
    c = Case(S, N, H, dk, dv, "f16", layout=1, ragged=True)
    for at, extra in ((0, 8), (3, 5)):
        wide = torch.full((N, S, H * dv + extra + at), 7.0, dtype=torch.float16, device="cuda")
        out = layer.attn(c.p, Y=wide[..., at:at + H * dv], **c.t)
        c.compare(out)
        assert (wide[..., :at] == 7).all() and (wide[..., at + H * dv:] == 7).all()
    # steps of a longer sequence
    long = torch.full((N, S + 9, H * dv), 7.0, dtype=torch.float16, device="cuda")
    c.compare(layer.attn(c.p, Y=long[:, 4:4 + S], **c.t))
    assert (long[:, :4] == 7).all() and (long[:, 4 + S:] == 7).all()


def test_attn_on_streams_and_in_graphs(layer):
    """Calls on another stream, and captured calls replayed on new inputs."""
    for S in (1, 600):
        c = Case(S, 2, 2, 64, 64, "bf16", grad=True, decay="both", lens=[S, S // 2 + 1])
        f = {k: v for k, v in c.t.items() if k not in ("dY", "d_final_state")}
        want, gwant = layer.attn(c.p, **f), layer.attn_grad(c.p, want=c.grads(), **c.t)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        a, b = layer.attn(c.p, stream=side, **f), layer.attn_grad(c.p, want=c.grads(), stream=side, **c.t)
        torch.cuda.current_stream().wait_stream(side)
        same_bits(a, want)
        same_bits(b, gwant)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a, b = layer.attn(c.p, **f), layer.attn_grad(c.p, want=c.grads(), **c.t)
        for _ in range(2):
            for x in ("Q", "K", "V"):
                c.t[x].copy_(torch.randn_like(c.t[x].float()))
            graph.replay()
            torch.cuda.synchronize()
            same_bits(a, layer.attn(c.p, **f))
            same_bits(b, layer.attn_grad(c.p, want=c.grads(), **c.t))


def test_attn_two_graphs_of_one_layer(layer):
    """Two captured calls replayed on two streams at once share nothing."""
    cases = [Case(900, 1, 2, 64, 64, "bf16", grad=True, seed=s) for s in (1, 2)]
    wants = [layer.attn_grad(c.p, want=c.grads(), **c.t) for c in cases]
    graphs, outs, streams = [], [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer.attn_grad(c.p, want=c.grads(), **c.t))
        graphs.append(g)
        streams.append(torch.cuda.Stream())
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, wants):
        same_bits(o, w)


def test_attn_handle_scratch(layer):
    """The C entry without placed scratch uses the handle's own."""
    import ctypes
    from onnx_lstm_gru_gb300 import state_space as ss
    c = Case(600, 1, 2, 64, 64, "f32", ragged=False, state=False, grad=True)
    want = layer.attn_grad(c.p, want=c.grads(), **c.t)
    ops = ss.rk_attn_grad_operands()
    outs = {n: torch.empty_like(v) for n, v in want.items()}
    for n, v in {**c.t, **outs}.items():
        words = (v.data_ptr(), 0, v.numel())
        setattr(ops, n, rk.rk_rows(*words, 0, 0) if n in ss._OPERANDS["attn_grad"][0] else rk.rk_tensor(*words))
    stream = torch.cuda.current_stream().cuda_stream
    assert rk.rk_attn_grad_encode(layer.handle, c.p.to_c(), ops, None, ctypes.c_void_p(stream)) == rk.RK_OK
    torch.cuda.synchronize()
    same_bits(outs, want)


def test_layer_together(layer):
    """Queries and keys through qk, then attention, then both backward: the
    gradients against those of the 64-bit definitions chained the same way,
    each operator given what the one before it wrote."""
    S, N, H, KH, d, dv = 90, 2, 4, 2, 64, 48
    for dtype in DTYPES:
        i, p, t, _ = qk_case((S, N, H, KH, d, d, False, "rms"), dtype, 1, False, 5, ragged=False)
        lens = [S, 33]
        t["sequence_lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
        y = layer.qk(p, **t)
        c = Case(S, N, H, d, dv, dtype, layout=1, k=KH, v=KH, lens=lens, state=False, grad=True)
        c.t.update(Q=y["YQ"], K=y["YK"])
        dY = c.t.pop("dY")
        c.compare(layer.attn(c.p, **c.t))
        c.t["dY"] = dY
        g = layer.attn_grad(c.p, want=c.grads(), **c.t)
        c.compare(g)
        t.update(dYQ=g["dQ"], dYK=g["dK"])
        out = layer.qk_grad(p, **t)
        for side in "QK":
            dX, dScale = qk_reference(p, t, lens, side, batch_first(g["d" + side], 1))
            check(batch_first(out["d" + side], 1).to(out["dQ"].dtype), dX)
            check(out[f"d{side}Scale"], dScale)
