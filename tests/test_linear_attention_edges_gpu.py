"""GPU tests of the linear attention where its chunks can go wrong: chunks run
step by step beside others, values and decays at the ends of float32's range,
waits that fail, scratch, and errors in the mean square.  Inputs, checks and
tolerances are those of ``test_linear_attention_gpu.py`` where a test does not
state its own."""
import pytest
import torch

import onnx_lstm_gru_gb300 as rk
from onnx_lstm_gru_gb300 import state_space as ss
from test_linear_attention_gpu import (  # noqa: F401  (layer: the fixture)
    DTYPES, F64, UNIT, Case, batch_first, both_ways, check, cut, layer, same_bits)

pytestmark = pytest.mark.gpu


# ---- chunks run step by step beside others ------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,S,H", [(80, 260, 2), (40, 260, 4), (1, 700, 2), (1, 700, 4)])
def test_attn_decays_that_are_none_in_the_second_head(layer, N, S, H, dtype):
    """Two heads share a block; whichever of them has the NaN, it is where the
    definition has it, in sequences whole and cut."""
    for at in (100, 128, 150, 191, 192):
        c = Case(S, N, H, 64, 64, dtype, ragged=False, layout=1)
        assert cut(c) == (N == 1)
        c.t["Decay"][:, at, 1::2] = float("nan")
        c.compare(layer.attn(c.p, **c.t), f"{at}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [(64, 64), (128, 128), (64, 128)])
def test_attn_every_second_chunk_step_by_step(layer, sizes, dtype):
    """Chunks whose products of queries and keys pass float32's range lie
    between ones where they do not; each is compared by itself, as the others'
    outputs are far larger, and equal calls give equal bits."""
    c = Case(450, 4, 2, *sizes, dtype, ragged=False, layout=1, state=False)
    for a in (64, 192, 320):
        c.t["Q"][:, a:a + 64] *= 1e20
        c.t["K"][:, a:a + 64] *= 1e20
        c.t["V"][:, a:a + 64] *= 1e-22
    got, want = layer.attn(c.p, **c.t), c.reference()
    check(got["final_state"], want["final_state"], "final_state")
    for a in range(0, 450, 64):
        check(got["Y"][:, a:a + 64], want["Y"][:, a:a + 64], f"Y {a}")
    for _ in range(10):
        same_bits(got, layer.attn(c.p, **c.t))


# ---- values beyond a chunk's range ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_attn_large_products_beside_decays(layer, d, dtype):
    """Chunks that decay by 2^-99.7, queries and keys whose products are 2^28:
    scaled by the decays' inverses they would pass float32's range, while the
    outputs are some 2^30."""
    c = Case(130, 2, 2, d, d, dtype, ragged=False, layout=1, scale=1.0, state=False, grad=True)
    c.t["Decay"].fill_(-1.08)
    c.t["Q"].fill_(2048.0), c.t["K"].fill_(2048.0)
    both_ways(layer, c)
    c = Case(130, 2, 2, d, d, dtype, ragged=False, layout=1, scale=1.0, state=False)
    c.t["Decay"].fill_(-1.08)
    c.t["Q"].fill_(2048.0), c.t["K"].fill_(2048.0), c.t["V"].fill_(2.0)
    c.compare(layer.attn(c.p, **c.t))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [(64, 48), (128, 72)])
@pytest.mark.parametrize("power", [30, 60, 85, 100])
def test_attn_inputs_of_thousands_beside_decays(layer, power, sizes, dtype):
    c = Case(200, 1, 2, *sizes, dtype, ragged=False, layout=0, grad=True)
    c.t["Decay"].fill_(-power / 64 * 0.6931471805599453)
    for n in ("Q", "K", "V", "dY"):
        c.t[n].mul_(3000.0)
    both_ways(layer, c)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_attn_large_states_beside_decays(layer, d, dtype):
    """A state whose product with the queries passes float32's range unless it
    decays first."""
    c = Case(130, 2, 2, d, d, dtype, ragged=False, layout=1, scale=1e-33)
    c.t["initial_state"].mul_(1e34), c.t["Q"].mul_(1e4)
    c.t["Decay"].fill_(-0.1)
    c.t["Decay"][:, 0] = -5.0
    c.compare(layer.attn(c.p, **c.t))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["Q", "K", "V", "dY"])
def test_attn_one_large_operand(layer, name, dtype):
    c = Case(200, 1, 3, 64, 64, dtype, ragged=False, layout=1, grad=True)
    c.t[name].mul_(1e12)
    both_ways(layer, c)


# ---- growth ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 160])
@pytest.mark.parametrize("steps", [{100: 85.0}, {70: 60.0, 140: 60.0, 150: 53.6, 200: -75.0},
                                   {66: 88.0, 67: 85.6, 200: -75.0}])
def test_attn_strong_growth(layer, steps, N, dtype):
    """A tiny state that grows by more than a power of two in float32 holds,
    within the first piece of a sequence that is cut, and in ones that are not."""
    c = Case(700, N, 1, 32, 32, dtype, ragged=False, layout=1)
    assert cut(c) == (N == 1)
    c.t["Decay"].zero_()
    for at, g in steps.items():
        c.t["Decay"][:, at] = g
    c.t["K"][:, :max(steps) + 1] = 0  # nothing else is written before
    c.t["Q"].mul_(0.02)
    c.t["initial_state"].copy_(c.t["initial_state"].sign() * (1e-33 if len(steps) == 1 else 2.0 ** -126))
    c.compare(layer.attn(c.p, **c.t))


# ---- waits that fail ------------------------------------------------------------------------------------

def test_attn_failed_waits_reach_every_handle(layer):
    """A wait that gives up (a phase that nothing ends, 0.2 ms) is reported
    once by each handle that has run attention in chunks, whichever polls first,
    and by none that has not."""
    c = Case(70, 2, 2, 64, 64, "f32", ragged=False)
    stream = torch.cuda.current_stream()
    other, idle, late = (rk.StateSpaceLayer() for _ in range(3))
    layer.attn(c.p, **c.t), other.attn(c.p, **c.t)
    layer.poll(), other.poll(stream), idle.poll()
    failing = rk.RecurrentLayer()
    assert rk.rk_selftest_timeout(failing.handle, stream.cuda_stream, 200_000) == rk.RK_OK
    for who in (other, layer, failing):
        with pytest.raises(rk.RkError) as e:
            who.poll()
        assert e.value.code == rk.RK_ERR_TIMEOUT
        who.poll()
    idle.poll()
    c.compare(late.attn(c.p, **c.t))
    late.poll()
    for who in (other, idle, late, failing):
        who.close()


# ---- scratch --------------------------------------------------------------------------------------------

@pytest.mark.parametrize("q,k,v", [(4, 4, 4), (2, 1, 2)])
@pytest.mark.parametrize("S,N", [(700, 1), (70, 3)])
def test_attn_grad_in_the_scratch_it_needs(layer, S, N, q, k, v):
    """Whatever is wanted, no more than that is taken, and the bits are those
    of all outputs together."""
    c = Case(S, N, 4, 48, 64, "bf16", q=q, k=k, v=v, decay="both", layout=1, grad=True)
    every = layer.attn_grad(c.p, want=c.grads(), **c.t)
    stream = torch.cuda.current_stream().cuda_stream
    for want in (("dQ",), ("dK", "dV"), ("d_initial_state",), ("dDecay",), ("d_decay_bias", "dQ"), c.grads()):
        ops = ss.rk_attn_grad_operands()
        outs = {n: torch.empty_like(every[n]) for n in want}
        for n, x in {**c.t, **outs}.items():
            words = (x.data_ptr(), 0, x.numel())
            setattr(ops, n, ss.rk_rows(*words, 0, 0) if n in ss._OPERANDS["attn_grad"][0] else rk.rk_tensor(*words))
        need = rk.rk_attn_grad_scratch_needed(c.p.to_c(), ops)
        room = torch.full((need + 64,), 7.0, device="cuda")
        work = ss.rk_workspace(room.data_ptr(), 32, 32 + need)
        assert rk.rk_attn_grad_encode(layer.handle, c.p.to_c(), ops, work, stream) == rk.RK_OK
        same_bits(outs, {n: every[n] for n in want})
        assert bool((room[:32] == 7).all()) and bool((room[32 + need:] == 7).all())
        if need:
            work.length -= 1
            assert rk.rk_attn_grad_encode(layer.handle, c.p.to_c(), ops, work, stream) == rk.RK_ERR_SHAPE


# ---- turns ----------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_turns_near_the_zeros_of_the_sine(layer, interleaved, dtype):
    """Pairs (0, 1) turned by about a multiple of half a turn: the first element
    is the sine, far smaller than the second.  An angle of up to half a turn in
    float32 is off by pi 2^-25, the sine by one unit of 2^-24 at most, and the
    element then by its own rounding: 2^-22.5 in all beside that, in gradients
    too, and 2^-25 for Half's numbers below its normal ones."""
    S, r = 3000, 64
    p = rk.QkProblem(seq=S, batch=1, heads=1, size=r, rotary=r, interleaved=interleaved, norm="none", dtype=dtype)
    f = (torch.pi * (1 + 3e-7 * torch.arange(r // 2, dtype=F64) ** 2)).float()
    x = torch.zeros(S, 1, r)
    x[..., slice(1, None, 2) if interleaved else slice(r // 2, None)] = 1.0
    x = x.to(rk.torch_dtype(dtype)).cuda()
    angle = torch.arange(S, dtype=F64)[:, None] * f.double()
    first = slice(0, None, 2) if interleaved else slice(0, r // 2)
    t = dict(K=x, Frequencies=f.cuda())
    for y, sign in ((layer.qk(p, x, **t)["YQ"], -1), (layer.qk_grad(p, x, dYQ=x, dYK=x, want=("dQ",), **t)["dQ"], 1)):
        got, want = y[:, 0, first].double().cpu(), sign * torch.sin(angle)
        bound = UNIT[y.dtype] * want.abs() + 2.0 ** -22.5 + 2.0 ** -25
        assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() - bound).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S,N,H,dk,dv", [(260, 6, 3, 64, 32), (330, 6, 1, 128, 72), (130, 60, 3, 24, 16),
                                         (700, 1, 2, 128, 128), (260, 40, 4, 128, 128)])
def test_attn_rows_that_end_where_sums_start_anew_with_a_bias(layer, S, N, H, dk, dv, dtype):
    """With a bias the sums start anew at every chunk, unless that takes more
    than 32 MB (the last shape); rows end before, at and behind chunks' ends, in
    sequences cut and not, and the bias' gradient is there without a bias too."""
    lens = ([64, 65, 128, 192, 63, 0] * 10)[:N] if N > 1 else None
    c = Case(S, N, H, dk, dv, dtype, lens=lens, ragged=False, layout=N % 2, decay="both", grad=True)
    c.compare(layer.attn_grad(c.p, want=c.grads(), **c.t))
    c.t["Decay"] = c.t["Decay"] + c.t.pop("decay_bias")
    c.compare(layer.attn_grad(c.p, want=("dDecay", "d_decay_bias"), **c.t))


# ---- errors in the mean square ----------------------------------------------------------------------------

TIGHT_SHAPES = [(300, 2, 4, 64, 64), (300, 2, 2, 128, 128), (700, 1, 2, 64, 48), (1500, 1, 1, 128, 128),
                (777, 2, 2, 72, 103), (513, 60, 3, 40, 64), (12, 3, 2, 128, 96)]


def relative(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", TIGHT_SHAPES)
def test_attn_mean_square(layer, shape, dtype):
    """What is float32 is off by 1e-6 of its size in the mean square.  An
    element goes through at most 250 roundings of 2^-24 of what it is then: 8 x 6
    of 128 elements' products for S (sums of sixteen, six pairs of terms), 4 x 6
    for P's and 8 x 6 for the state's, 3 each for the terms of P, of the scaled
    keys and of the state, 4 for each of two powers of two (off by 2^-22), and
    26 for a chunk that the state passes, of which the decays here leave
    at most four in sight.  Inputs have no sign of their own, so that roundings
    add up by their squares: sqrt(250) 2^-24 = 9.4e-7.  A term of a factor left
    out alone (two bfloat16 numbers in place of three, off by 2^-17 at most and
    by 0.4 of that in the mean square) is 3e-6.
    16-bit outputs are the definition's, rounded, but where that lies next to
    the middle of two numbers: P and the state as two bfloat16 numbers are off by
    2^-17, an output by 2^-16 of what its terms are, in the mean twice its size
    or less, on either side of a middle, and numbers are a unit roundoff or two
    apart: a share of 2^-14 of an output's size through that spacing.  With one
    number in place of two a third of bfloat16's outputs would differ.
    dDecay is a sum of k dk - q dq over the at most 512 steps to a mark, each
    element's product off by as much, again by their squares; what is left
    at the mark and taken back is at most as large again.  d_decay_bias adds up
    dDecay, and what a block of 512 steps is off by with it, at each of them."""
    c = Case(*shape, dtype, ragged=False, decay="both", layout=1, grad=True)
    p, got, want = c.p, layer.attn_grad(c.p, want=c.grads(), **c.t), c.reference()
    for n in ("dY", "d_final_state"):
        c.t.pop(n)
    got.update(layer.attn(p, **c.t))
    want.update(c.reference())
    far = {}
    for k, v in got.items():
        if v.dtype == torch.float32 and k not in ("dDecay", "d_decay_bias"):
            v = batch_first(v, 1) if k in ("Y", "dQ", "dK", "dV") else v
            off = relative(v, want[k])
            if off > 1e-6:
                far[k] = off
        elif v.dtype != torch.float32:
            near = want[k].to(v.dtype)
            share = float((batch_first(v, 1) != near.double()).float().mean())
            if share > 2.0 ** -14 / (2 * UNIT[v.dtype]):
                far[k] = share
    square = torch.zeros(p.batch, p.seq, p.heads, dtype=F64)
    for x, dx in (("Q", "dQ"), ("K", "dK")):
        a = (batch_first(c.t[x], 1) * want[dx]).square()
        square += a.unflatten(-1, (p.heads, -1)).sum(-1)
    pad = torch.nn.functional.pad(square, (0, 0, 0, -p.seq % 512)).unflatten(1, (-1, 512)).sum(2, keepdim=True)
    block = (4 * 1e-12 * pad).sqrt().expand(-1, -1, 512, -1)  # by step, the same for all of a block's
    steps = block.flatten(1, 2)[:, :p.seq]
    off = (got["dDecay"].double().cpu() - want["dDecay"]).norm() / steps.norm()
    if off > 1:
        far["dDecay"] = float(off)
    bias = (512 ** 2 * block[:, :, 0].square()).sum((0, 1)).sqrt()
    off = (got["d_decay_bias"].double().cpu() - want["d_decay_bias"]).norm() / bias.norm()
    if off > 1:
        far["d_decay_bias"] = float(off)
    assert not far, far


@pytest.mark.parametrize("shape", [(195, 2, 4, 64, 64), (784, 2, 2, 125, 128), (784, 20, 4, 128, 96)])
def test_attn_long_memories_in_the_mean_square(layer, shape):
    """Without decays an output is mostly what the state adds to it, a sum of
    eight products of sixteen elements to which four of P and the values are
    added.  The tensor cores cut sums off, towards zero: by half a unit of 2^-23
    in the mean, 0.72 of that where bits are spread evenly, of partial sums that
    grow as the root of their number: (5.6 + 4) 0.72 2^-24 = 4.1e-7, and what is
    rounded besides 2e-7, together 4.6e-7.  (The small products of the terms,
    added up before, cost nothing; 20 of them behind the large ones would be
    twice that.)"""
    c = Case(*shape, "f32", ragged=False, decay="none", layout=1, grad=True)
    got, want = layer.attn_grad(c.p, want=c.grads(), **c.t), c.reference()
    for n in ("dY", "d_final_state"):
        c.t.pop(n)
    got.update(layer.attn(c.p, **c.t))
    want.update(c.reference())
    far = {k: relative(batch_first(v, 1) if k in ("Y", "dQ", "dK", "dV") else v, want[k]) for k, v in got.items()}
    assert max(far.values()) <= 5e-7, far
