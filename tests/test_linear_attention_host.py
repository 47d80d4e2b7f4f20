"""Host side of the linear attention operators: refusals, scratch lengths,
packing and the 64-bit definitions the GPU tests compare with.  No GPU call is
made: every refused call is refused before anything is launched."""
import copy
import ctypes
import pickle

import pytest
import torch

import linear_attention_reference as ref
import onnx_lstm_gru_gb300 as rk
from onnx_lstm_gru_gb300 import state_space as ss

F64 = torch.float64


@pytest.fixture(scope="module")
def handle():
    rk.build()
    rk.load()
    h = rk.rk_create(0)
    yield h
    rk.rk_destroy(h)


QK = rk.QkProblem(seq=5, batch=2, heads=4, key_heads=2, size=10, rotary=6, dtype="f16")
ATTN = rk.AttnProblem(seq=5, batch=2, heads=4, key_size=6, value_size=10, query_heads=2, key_heads=2, dtype="bf16")
PROBLEMS = {"qk": QK, "qk_grad": QK, "attn": ATTN, "attn_grad": ATTN}
NAMES = {"qk": "QueryKey", "qk_grad": "QueryKeyGrad", "attn": "LinearAttention", "attn_grad": "LinearAttentionGrad"}
SCRATCH = {"qk_grad": rk.rk_qk_grad_scratch_length, "attn": rk.rk_attn_scratch_length,
           "attn_grad": rk.rk_attn_grad_scratch_length}


def operands(op, problem):
    """Fake device buffers (never touched), each exactly as long as it has to be."""
    ops = getattr(ss, f"rk_{op}_operands")()
    rows, tensors = ss._OPERANDS[op]
    for i, n in enumerate(rows + tensors):
        size = 1
        for d in problem.shapes()[n]:
            size *= d
        at = 0x10000000 + 0x100000 * i
        setattr(ops, n, ss.rk_rows(at, 0, size, 0, 0) if n in rows else rk.rk_tensor(at, 0, size))
    return ops


def encode(handle, op, c, ops):
    args = [handle, c, ops] + ([None] if op in SCRATCH else []) + [0]
    st = getattr(rk, f"rk_{op}_encode")(*args)
    return st, rk.rk_last_error(handle)


def refused(handle, op, c, ops, code, text):
    before = rk.rk_launch_count(handle)
    st, msg = encode(handle, op, c, ops)
    assert st == code and msg.startswith(NAMES[op] + ": ") and text in msg, (st, msg)
    assert rk.rk_launch_count(handle) == before


def test_null_arguments(handle):
    lib = rk.load()
    for op, p in PROBLEMS.items():
        c = p.to_c()
        extra = [None] if op in SCRATCH else []
        fn = getattr(lib, f"rk_{op}_encode")
        assert fn(None, ctypes.byref(c), None, *extra, None) == rk.RK_ERR_ARG
        assert fn(handle, None, None, *extra, None) == rk.RK_ERR_ARG
        assert fn(handle, ctypes.byref(c), None, *extra, None) == rk.RK_ERR_ARG
        assert "operands: null" in rk.rk_last_error(handle)
    for fn in (lib.rk_qk_grad_scratch_length, lib.rk_attn_scratch_length, lib.rk_attn_grad_scratch_length):
        assert fn(None) == -1


@pytest.mark.parametrize("op", list(PROBLEMS))
def test_operand_refusals(handle, op):
    p = PROBLEMS[op]
    rows, tensors = ss._OPERANDS[op]
    for n in rows + tensors:
        def change(**fields):
            ops = operands(op, p)
            t = getattr(ops, n)
            for k, v in fields.items():
                setattr(t, k, v)
            return ops
        size = getattr(operands(op, p), n).length
        if n in ss._REQUIRED[op] + ("Frequencies",):
            refused(handle, op, p.to_c(), change(ptr=None), rk.RK_ERR_SHAPE, f"{n}: required tensor is null")
        refused(handle, op, p.to_c(), change(offset=-1), rk.RK_ERR_SHAPE, f"{n}: negative offset")
        refused(handle, op, p.to_c(), change(length=-1), rk.RK_ERR_SHAPE, f"{n}: negative length")
        refused(handle, op, p.to_c(), change(offset=1), rk.RK_ERR_SHAPE, f"{n}: offset 1 + extent {size} exceeds")
        refused(handle, op, p.to_c(), change(offset=2 ** 63 - 1), rk.RK_ERR_SHAPE, f"{n}: offset")
        refused(handle, op, p.to_c(), change(ptr=0x20000001), rk.RK_ERR_SHAPE, f"{n}: address")
        if n in rows:
            refused(handle, op, p.to_c(), change(pitch=1), rk.RK_ERR_SHAPE, f"{n}: pitch 1 is less")
            refused(handle, op, p.to_c(), change(outer_pitch=1), rk.RK_ERR_SHAPE, f"{n}: outer_pitch 1 is less")
            refused(handle, op, p.to_c(), change(pitch=2 ** 62), rk.RK_ERR_SHAPE, f"{n}: pitch")
            # a wider pitch needs a longer buffer
            refused(handle, op, p.to_c(), change(pitch=50), rk.RK_ERR_SHAPE, f"{n}: offset 0 + extent")


@pytest.mark.parametrize("op,field,value,code,text", [
    ("qk", "dtype", 3, "SHAPE", "dtype: unknown value 3"),
    ("qk", "layout", 2, "SHAPE", "layout"),
    ("qk", "norm", 3, "SHAPE", "norm: unknown value 3"),
    ("qk", "interleaved", 2, "SHAPE", "interleaved"),
    ("qk", "rotary", 3, "SHAPE", "rotary: 3"),
    ("qk", "rotary", 12, "SHAPE", "rotary: 12"),
    ("qk_grad", "rotary", -2, "SHAPE", "rotary: -2"),
    ("qk_grad", "epsilon", -1.0, "SHAPE", "epsilon"),
    ("qk_grad", "epsilon", float("nan"), "SHAPE", "epsilon"),
    ("qk_grad", "size", 0, "SHAPE", "size: 0"),
    ("qk_grad", "size", 257, "UNSUPPORTED", "size"),
    ("qk", "heads", 0, "SHAPE", "heads: 0"),
    ("qk", "key_heads", 2 ** 23, "UNSUPPORTED", "key_heads"),
    ("qk", "seq", -1, "SHAPE", "seq: -1"),
    ("qk", "batch", 2 ** 30, "UNSUPPORTED", "seq*batch"),
    ("attn", "dtype", -1, "SHAPE", "dtype: unknown value -1"),
    ("attn", "layout", -1, "SHAPE", "layout"),
    ("attn", "key_size", 0, "SHAPE", "key_size: 0"),
    ("attn", "key_size", 129, "UNSUPPORTED", "key_size"),
    ("attn", "value_size", 129, "UNSUPPORTED", "value_size"),
    ("attn", "query_heads", 3, "SHAPE", "query_heads: 3 does not divide 4"),
    ("attn", "key_heads", -1, "SHAPE", "key_heads: -1 does not divide"),
    ("attn_grad", "value_heads", 8, "SHAPE", "value_heads: 8 does not divide"),
    ("attn_grad", "heads", 0, "SHAPE", "heads: 0"),
    ("attn_grad", "scale", float("inf"), "SHAPE", "scale"),
    ("attn_grad", "scale", float("nan"), "SHAPE", "scale"),
    ("attn_grad", "seq", 2 ** 30 + 1, "UNSUPPORTED", "seq"),
    ("attn_grad", "batch", 2 ** 24, "UNSUPPORTED", "batch*heads"),
])
def test_problem_refusals(handle, op, field, value, code, text):
    c = PROBLEMS[op].to_c()
    setattr(c, field, value)
    refused(handle, op, c, operands(op, PROBLEMS[op]), getattr(rk, f"RK_ERR_{code}"), text)
    if op in SCRATCH:
        assert SCRATCH[op](c) == -1


@pytest.mark.parametrize("op", list(PROBLEMS))
def test_nothing_wanted_launches_nothing(handle, op):
    ops = operands(op, PROBLEMS[op])
    rows, tensors = ss._OPERANDS[op]
    for n in rows + tensors:
        if n in ss._OUTPUTS[op]:
            getattr(ops, n).ptr = None
    before = rk.rk_launch_count(handle)
    st, msg = encode(handle, op, PROBLEMS[op].to_c(), ops)
    assert st == rk.RK_OK, msg
    assert rk.rk_launch_count(handle) == before


def test_no_heads_is_no_default(handle):
    """In the problem classes None stands for as many as heads; 0 is an error."""
    for name in ("query_heads", "key_heads", "value_heads"):
        p = rk.AttnProblem(seq=1, batch=1, heads=4, key_size=8, value_size=8, **{name: 0})
        refused(handle, "attn", p.to_c(), operands("attn", p), rk.RK_ERR_SHAPE, f"{name}: -1")
    p = rk.QkProblem(seq=1, batch=1, heads=4, key_heads=0, size=8)
    refused(handle, "qk", p.to_c(), operands("qk", p), rk.RK_ERR_SHAPE, "key_heads: 0")


def test_placed_scratch_is_checked(handle):
    for op in ("qk_grad", "attn_grad"):
        p = PROBLEMS[op]
        need = SCRATCH[op](p.to_c())
        assert need > 0
        ops = operands(op, p)
        for w, text in ((ss.rk_workspace(0x1000, 0, need - 1), "scratch: offset 0"),
                        (ss.rk_workspace(0x1000, -4, need), "scratch: offset -4"),
                        (ss.rk_workspace(0x1004, 0, need), "16-byte aligned")):
            assert getattr(rk, f"rk_{op}_encode")(handle, p.to_c(), ops, w, 0) == rk.RK_ERR_SHAPE
            assert text in rk.rk_last_error(handle)


def test_scratch_lengths():
    """Scratch follows from the problem alone; a single token needs none."""
    token = rk.AttnProblem(seq=1, batch=64, heads=16, key_size=128, value_size=128)
    assert rk.rk_attn_scratch_length(token.to_c()) == 0
    assert rk.rk_attn_scratch_length(rk.AttnProblem(seq=0, batch=4, heads=2, key_size=8, value_size=8).to_c()) == 0
    # one long sequence is cut into pieces, whose states are kept; many sequences fill the GPU as they are
    one = rk.AttnProblem(seq=4096, batch=1, heads=16, key_size=128, value_size=128)
    many = rk.AttnProblem(seq=512, batch=64, heads=16, key_size=64, value_size=64)
    assert rk.rk_attn_scratch_length(one.to_c()) > 0
    assert rk.rk_attn_scratch_length(many.to_c()) == 0
    assert rk.rk_attn_grad_scratch_length(one.to_c()) >= 2 * 16 * 4096
    # heads that share are added up in float32
    shared = rk.AttnProblem(seq=100, batch=2, heads=4, key_size=8, value_size=8, key_heads=1)
    alone = rk.AttnProblem(seq=100, batch=2, heads=4, key_size=8, value_size=8)
    more = rk.rk_attn_grad_scratch_length(shared.to_c()) - rk.rk_attn_grad_scratch_length(alone.to_c())
    assert more == 100 * 2 * 4 * 8


def test_scratch_of_what_is_wanted():
    """Gradients that are not wanted take no scratch; all of them take the length by the problem alone."""
    p = rk.AttnProblem(seq=4096, batch=64, heads=16, key_size=128, value_size=128)
    c, rows, outputs = p.to_c(), ss._OPERANDS["attn_grad"][0], ss._OUTPUTS["attn_grad"]

    def needed(p, *names):
        ops = ss.rk_attn_grad_operands()
        for n in names:
            setattr(ops, n, ss.rk_rows(0x1000, 0, 1, 0, 0) if n in rows else rk.rk_tensor(0x1000, 0, 1))
        return rk.rk_attn_grad_scratch_needed(p.to_c(), ops)
    every = rk.rk_attn_grad_scratch_length(c)
    assert every * 4 > 900e6
    assert needed(p, *outputs) == every and needed(p) == 0
    assert needed(p, "dQ", "dK", "dV", "d_initial_state") == 0
    assert every - 2 ** 16 < needed(p, "dDecay") < every
    shared = rk.AttnProblem(seq=100, batch=2, heads=4, key_size=8, value_size=16, query_heads=2, key_heads=1,
                            value_heads=2)
    assert [needed(shared, n) for n in ("dQ", "dK", "dV", "d_initial_state")] == [6400, 6400, 12800, 0]
    assert needed(shared, *outputs) == rk.rk_attn_grad_scratch_length(shared.to_c())
    # few sequences are cut into the same pieces, whatever is wanted
    one = rk.AttnProblem(seq=4096, batch=1, heads=16, key_size=128, value_size=128)
    assert needed(one, "dQ") == needed(one, "dQ", "dK", "dV") == needed(one, "d_initial_state") > 0
    # with a bias the decays take the states at every chunk, up to 32 MB: here of 3 x 12 heads, three chunks, both ways
    few = rk.AttnProblem(seq=201, batch=3, heads=12, key_size=48, value_size=80, dtype="f16")
    more = needed(few, "dDecay", "decay_bias") - needed(few, "dDecay")
    assert 36 * 3 * 2 * 128 * 128 <= more < 36 * 3 * 2 * 128 * 128 + 1024
    assert needed(few, "dDecay", "decay_bias") < needed(few, "d_decay_bias") == needed(few, "d_decay_bias", "decay_bias")
    many = rk.AttnProblem(seq=512, batch=8, heads=16, key_size=128, value_size=128)
    assert needed(many, "dDecay", "decay_bias") == needed(many, "dDecay")
    assert needed(rk.AttnProblem(seq=0, batch=4, heads=2, key_size=8, value_size=8), *outputs) == 0
    c.layout = 2
    assert rk.rk_attn_grad_scratch_needed(c, ss.rk_attn_grad_operands()) == -1
    assert rk.load().rk_attn_grad_scratch_needed(None, None) == -1


def test_defaults_of_the_problems():
    p = rk.AttnProblem(seq=1, batch=1, heads=4, key_size=64, value_size=8)
    c = p.to_c()
    assert (c.scale, c.query_heads, c.key_heads, c.value_heads) == (0.125, 4, 4, 4)
    assert rk.QkProblem(seq=1, batch=1, heads=4, size=8).to_c().key_heads == 4


@pytest.mark.parametrize("op", list(PROBLEMS))
def test_used_problems_are_copied_and_pickled(handle, op):
    p = PROBLEMS[op]
    plan = p._plan(op)
    for q in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p))):
        assert q == p and hash(q) == hash(p)
        assert q._plan(op) is plan
        assert bytes(q.to_c()) == bytes(p.to_c())


def test_binding_names_the_operand(handle):
    """The first operand goes by its own name, also in refusals."""
    layer = rk.StateSpaceLayer()
    with pytest.raises(ValueError, match="Q: expected a CUDA tensor"):
        layer.qk(QK, torch.zeros(5, 2, 40, dtype=torch.float16))
    with pytest.raises(TypeError, match="expected AttnProblem"):
        layer.attn(QK, torch.zeros(1))
    layer.close()


# ---- the definitions themselves ------------------------------------------------------------------

def normal(*shape, seed, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64) * scale


def directional(f, inputs, grads, seed, eps=1e-5, tol=1e-7):
    """sum over inputs of <gradient, direction> against the central difference
    of f along it.  The difference's own error is of the order of eps^2 and of
    2^-53 / eps, 1e-10 here, times the third derivative and the value; 1e-7 of
    the sum's size leaves room for both."""
    dirs = {k: normal(*v.shape, seed=seed + i) for i, (k, v) in enumerate(inputs.items())}
    up = f(**{k: v + eps * dirs[k] for k, v in inputs.items()})
    down = f(**{k: v - eps * dirs[k] for k, v in inputs.items()})
    want = (up - down) / (2 * eps)
    parts = [(grads[k] * dirs[k]).sum() for k in inputs]
    assert abs(sum(parts) - want) <= tol * (1 + sum(abs(x) for x in parts))


@pytest.mark.parametrize("norm", ["none", "rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_gradient_against_differences(norm, interleaved):
    N, S, H, d = 2, 4, 3, 7
    kw = dict(heads=H, Frequencies=normal(2, seed=1).abs(), positions=torch.tensor([[3, 0, -2, 9], [1, 2, 3, 4]]),
              lens=[4, 2], rotary=4, interleaved=interleaved, norm=norm, epsilon=1e-2)
    inp = dict(X=normal(N, S, H * d, seed=2), Scale=normal(d, seed=3))
    dY = normal(N, S, H * d, seed=4)
    dX, dScale = ref.qk(dY=dY, **inp, **kw)
    directional(lambda **t: (ref.qk(**t, **kw) * dY).sum(), inp, dict(X=dX, Scale=dScale), seed=5)


def test_qk_turns_by_the_angle():
    """The product of a query and a key depends on the distance of their positions alone."""
    f = normal(4, seed=1)
    q, k = normal(1, 1, 8, seed=2), normal(1, 1, 8, seed=3)
    for interleaved in (False, True):
        def at(x, p):
            return ref.qk(x, 1, Frequencies=f, positions=torch.tensor([[p]]), rotary=8, interleaved=interleaved)
        assert abs((at(q, 17) * at(k, 12)).sum() - (at(q, 5) * at(k, 0)).sum()) < 1e-12


def test_attn_gradient_against_differences():
    N, S, H, dk, dv = 3, 5, 4, 3, 2
    kw = dict(heads=H, scale=0.7, lens=[5, 2, 0], key_size=dk, value_size=dv)
    inp = dict(Q=normal(N, S, 2 * dk, seed=1), K=normal(N, S, dk, seed=2), V=normal(N, S, 4 * dv, seed=3),
               Decay=-normal(N, S, H, seed=4).abs(), decay_bias=normal(H, seed=5, scale=0.1),
               initial_state=normal(N, H, dk, dv, seed=6))
    dY, dF = normal(N, S, H * dv, seed=7), normal(N, H, dk, dv, seed=8)

    def loss(**t):
        o = ref.attn(**t, **kw)
        return (o["Y"] * dY).sum() + (o["final_state"] * dF).sum()
    g = ref.attn(dY=dY, d_final_state=dF, **inp, **kw)
    directional(loss, inp, {k: g[("d_" if k in ("decay_bias", "initial_state") else "d") + k] for k in inp}, seed=9)
