"""Host side of the state space operators: refusals, scratch lengths, packing
and the 64-bit definitions the GPU tests compare with.  No GPU call is made:
every refused call is refused before anything is launched."""
import copy
import ctypes
import dataclasses
import inspect
import pickle

import pytest
import torch

import onnx_lstm_gru_gb300 as rk
import state_space_reference as ref
from onnx_lstm_gru_gb300 import state_space as ss

F64 = torch.float64


@pytest.fixture(scope="module")
def handle():
    rk.build()
    rk.load()
    h = rk.rk_create(0)
    yield h
    rk.rk_destroy(h)


PROBLEMS = {
    "norm": rk.NormProblem(rows=4, cols=10, dtype="f16"),
    "norm_grad": rk.NormProblem(rows=4, cols=10, dtype="f16"),
    "conv": rk.ConvProblem(seq=5, batch=2, channels=6, width=4, dtype="bf16"),
    "conv_grad": rk.ConvProblem(seq=5, batch=2, channels=6, width=4, dtype="bf16"),
    "scan": rk.ScanProblem(seq=5, batch=2, channels=6, state=3, groups=2, dtype="f32"),
    "scan_grad": rk.ScanProblem(seq=5, batch=2, channels=6, state=3, groups=2, dtype="f32"),
}
NAMES = {"norm": "LayerNormalization", "norm_grad": "LayerNormalizationGrad", "conv": "CausalConv",
         "conv_grad": "CausalConvGrad", "scan": "SelectiveScan", "scan_grad": "SelectiveScanGrad"}


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
    args = [handle, c, ops] + ([] if op in ("norm", "conv") else [None]) + [0]
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
        extra = [] if op in ("norm", "conv") else [None]
        fn = getattr(lib, f"rk_{op}_encode")
        assert fn(None, ctypes.byref(c), None, *extra, None) == rk.RK_ERR_ARG
        assert fn(handle, None, None, *extra, None) == rk.RK_ERR_ARG
        assert fn(handle, ctypes.byref(c), None, *extra, None) == rk.RK_ERR_ARG
        assert "operands: null" in rk.rk_last_error(handle)
    for fn in (lib.rk_norm_grad_scratch_length, lib.rk_conv_grad_scratch_length, lib.rk_scan_scratch_length,
               lib.rk_scan_grad_scratch_length):
        assert fn(None) == -1


@pytest.mark.parametrize("op", list(PROBLEMS))
def test_operand_refusals(handle, op):
    p = PROBLEMS[op]
    rows, tensors = ss._OPERANDS[op]
    optional = {"Scale", "B", "Z", "D", "delta_bias", "sequence_lens", "initial_state", "d_final_state", "Y", "dX",
                "dDelta", "dB", "dC", "dZ", "Mean", "InvStdDev", "final_state", "dScale", "dW", "dA", "dD",
                "d_delta_bias", "d_initial_state"} - set(ss._REQUIRED[op])
    for n in rows + tensors:
        def change(**fields):
            ops = operands(op, p)
            t = getattr(ops, n)
            for k, v in fields.items():
                setattr(t, k, v)
            return ops
        size = getattr(operands(op, p), n).length
        if n not in optional:
            refused(handle, op, p.to_c(), change(ptr=None), rk.RK_ERR_SHAPE, f"{n}: required tensor is null")
        refused(handle, op, p.to_c(), change(offset=-1), rk.RK_ERR_SHAPE, f"{n}: negative offset")
        refused(handle, op, p.to_c(), change(length=-1), rk.RK_ERR_SHAPE, f"{n}: negative length")
        refused(handle, op, p.to_c(), change(offset=1), rk.RK_ERR_SHAPE, f"{n}: offset 1 + extent {size} exceeds")
        refused(handle, op, p.to_c(), change(offset=2 ** 63 - 1), rk.RK_ERR_SHAPE, f"{n}: offset")
        refused(handle, op, p.to_c(), change(ptr=0x20000001), rk.RK_ERR_SHAPE, f"{n}: address")
        if n in rows:
            refused(handle, op, p.to_c(), change(pitch=1), rk.RK_ERR_SHAPE, f"{n}: pitch 1 is less")
            if p.shapes()[n][0] > 1 and op not in ("norm", "norm_grad"):
                refused(handle, op, p.to_c(), change(outer_pitch=1), rk.RK_ERR_SHAPE, f"{n}: outer_pitch 1 is less")
            refused(handle, op, p.to_c(), change(pitch=2 ** 62), rk.RK_ERR_SHAPE, f"{n}: pitch")
            # a wider pitch needs a longer buffer
            refused(handle, op, p.to_c(), change(pitch=50), rk.RK_ERR_SHAPE, f"{n}: offset 0 + extent")


@pytest.mark.parametrize("op,field,value,code,text", [
    ("norm", "dtype", 3, "SHAPE", "dtype: unknown value 3"),
    ("norm", "epsilon", -1.0, "SHAPE", "epsilon"),
    ("norm", "epsilon", float("nan"), "SHAPE", "epsilon"),
    ("norm", "rows", -1, "SHAPE", "rows: -1"),
    ("norm_grad", "cols", 0, "SHAPE", "cols: 0"),
    ("norm_grad", "cols", 2 ** 24 + 1, "UNSUPPORTED", "cols"),
    ("norm_grad", "rows", 2 ** 31, "UNSUPPORTED", "rows"),
    ("conv", "layout", 2, "SHAPE", "layout"),
    ("conv", "activation", 2, "SHAPE", "activation: unknown value 2"),
    ("conv", "width", 0, "SHAPE", "width: 0"),
    ("conv_grad", "width", 9, "UNSUPPORTED", "width"),
    ("conv_grad", "seq", -3, "SHAPE", "seq: -3"),
    ("conv_grad", "batch", 2 ** 30, "UNSUPPORTED", "seq*batch"),
    ("scan", "state", 0, "SHAPE", "state: 0"),
    ("scan", "state", 129, "UNSUPPORTED", "state"),
    ("scan", "groups", 4, "SHAPE", "groups: 4 does not divide 6"),
    ("scan", "groups", 0, "SHAPE", "groups: 0"),
    ("scan_grad", "softplus", 2, "SHAPE", "softplus"),
    ("scan_grad", "channels", 0, "SHAPE", "channels: 0"),
])
def test_problem_refusals(handle, op, field, value, code, text):
    c = PROBLEMS[op].to_c()
    setattr(c, field, value)
    refused(handle, op, c, operands(op, PROBLEMS[op]), getattr(rk, f"RK_ERR_{code}"), text)
    length = {"norm_grad": rk.rk_norm_grad_scratch_length, "conv_grad": rk.rk_conv_grad_scratch_length,
              "scan": rk.rk_scan_scratch_length, "scan_grad": rk.rk_scan_grad_scratch_length}.get(op)
    if length:
        assert length(c) == -1


def test_gate_gradient_needs_the_gate(handle):
    p = PROBLEMS["scan_grad"]
    ops = operands("scan_grad", p)
    ops.Z = ss.rk_rows(None, 0, 0, 0, 0)
    refused(handle, "scan_grad", p.to_c(), ops, rk.RK_ERR_SHAPE, "dZ: exists only with Z")


def test_placed_scratch_is_checked(handle):
    p = rk.ScanProblem(seq=400, batch=1, channels=64, state=16)
    need = rk.rk_scan_grad_scratch_length(p.to_c())
    assert need > 0
    ops = operands("scan_grad", p)
    for w, text in ((ss.rk_workspace(0x1000, 0, need - 1), "scratch: offset 0"),
                    (ss.rk_workspace(0x1000, -4, need), "scratch: offset -4"),
                    (ss.rk_workspace(0x1004, 0, need), "16-byte aligned")):
        assert rk.rk_scan_grad_encode(handle, p.to_c(), ops, w, 0) == rk.RK_ERR_SHAPE
        assert text in rk.rk_last_error(handle)


def test_scratch_lengths():
    """Scratch follows from the problem alone: none for a single token or a
    batch that fills the card, chunk states for one long sequence."""
    assert rk.rk_scan_scratch_length(rk.ScanProblem(seq=1, batch=64, channels=2048, state=16).to_c()) == 0
    assert rk.rk_scan_scratch_length(rk.ScanProblem(seq=512, batch=512, channels=2048, state=16).to_c()) == 0
    assert rk.rk_scan_scratch_length(rk.ScanProblem(seq=4096, batch=1, channels=2048, state=16).to_c()) > 0
    assert rk.rk_scan_scratch_length(rk.ScanProblem(seq=0, batch=4, channels=8, state=16).to_c()) == 0
    assert rk.rk_norm_grad_scratch_length(rk.NormProblem(rows=3, cols=5).to_c()) > 0
    assert rk.rk_conv_grad_scratch_length(rk.ConvProblem(seq=0, batch=4, channels=8).to_c()) == 0


def test_structs_are_packed_as_declared():
    for op, (rows, tensors) in ss._OPERANDS.items():
        struct = getattr(ss, f"rk_{op}_operands")
        assert ctypes.sizeof(struct) == 40 * len(rows) + 24 * len(tensors)


def test_row_distance(handle):
    """Slices of wider rows, steps of longer sequences and transposed views are
    taken as they are; rows that are not dense or that overlap are not."""
    pitches = ss._binding().row_pitches
    wide = torch.zeros(5, 3, 16)
    assert pitches(wide[..., :4]) == (16, 48, 4 * 48 + 2 * 16 + 4)
    assert pitches(wide[:, :2, 4:]) == (16, 48, 4 * 48 + 16 + 12)
    assert pitches(wide[:, :1, 4:]) == (12, 48, 4 * 48 + 12)
    assert pitches(wide[:1, :, 4:]) == (16, 0, 2 * 16 + 12)
    assert pitches(wide.transpose(0, 1)) == (48, 16, 4 * 48 + 2 * 16 + 16)
    assert pitches(torch.zeros(7, 9)[:, :2]) == (9, 0, 6 * 9 + 2)
    for bad in (wide[..., ::2], torch.zeros(1, 1, 4).expand(5, 3, 4), torch.zeros(5, 1, 4).expand(5, 3, 4)):
        assert pitches(bad) is None


def test_every_operand_is_an_input_or_an_output():
    """The outputs are what the header's operand lists write; each operator's
    default choice is among them."""
    for op, outputs in ss._OUTPUTS.items():
        names = sum(ss._OPERANDS[op], ())
        assert set(outputs) <= set(names) and not set(outputs) & set(ss._REQUIRED[op])
        want = inspect.signature(getattr(rk.StateSpaceLayer, op)).parameters["want"].default
        assert set(want) <= set(outputs)


@pytest.mark.parametrize("op", list(PROBLEMS))
def test_used_problems_are_copied_and_pickled(handle, op):
    """A problem that a call has packed its operands by is still plain data."""
    p = PROBLEMS[op]
    plan = p._plan(op)
    for q in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p)), dataclasses.replace(p)):
        assert q == p and hash(q) == hash(p) and type(q) is type(p)
        assert q._plan(op) is plan  # and finds what equal problems share
        assert bytes(q.to_c()) == bytes(p.to_c())


def test_overlapping_rows_are_refused(handle):
    """By the C entry too: two steps of five batch rows each that share rows."""
    p = rk.ConvProblem(seq=2, batch=5, channels=6, dtype="f32")
    ops = operands("conv", p)
    for pitch, outer, ok in ((6, 6, False), (6, 29, False), (12, 6, True), (11, 6, False), (6, 30, True)):
        ops.X = ss.rk_rows(0x10000000, 0, 10 ** 6, pitch, outer)
        c = p.to_c()
        if ok:
            c.width = 0  # refused later, for another reason
            st, msg = encode(handle, "conv", c, ops)
            assert st == rk.RK_ERR_SHAPE and "width" in msg
        else:
            refused(handle, "conv", c, ops, rk.RK_ERR_SHAPE, "X: ")


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


def test_norm_gradient_against_differences():
    X, S, B, dY = normal(5, 9, seed=1), normal(9, seed=2), normal(9, seed=3), normal(5, 9, seed=4)
    f = ref.norm(X, S, B)
    g = ref.norm_grad(X, dY, f["Mean"], f["InvStdDev"], S)
    directional(lambda X, Scale, B: (ref.norm(X, Scale, B)["Y"] * dY).sum(), dict(X=X, Scale=S, B=B),
                dict(X=g["dX"], Scale=g["dScale"], B=g["dB"]), seed=5)


@pytest.mark.parametrize("silu", [False, True])
def test_conv_gradient_against_differences(silu):
    N, S, C, w = 3, 6, 4, 4
    lens = [6, 2, 0]
    inp = dict(X=normal(N, S, C, seed=1), W=normal(C, w, seed=2), B=normal(C, seed=3),
               initial_state=normal(N, w - 1, C, seed=4))
    dY, dF = normal(N, S, C, seed=5), normal(N, w - 1, C, seed=6)

    def loss(**t):
        o = ref.conv(lens=lens, silu=silu, **t)
        return (o["Y"] * dY).sum() + (o["final_state"] * dF).sum()
    g = ref.conv(lens=lens, silu=silu, dY=dY, d_final_state=dF, **inp)
    directional(loss, inp, dict(X=g["dX"], W=g["dW"], B=g["dB"], initial_state=g["d_initial_state"]), seed=7)


@pytest.mark.parametrize("softplus", [False, True])
def test_scan_gradient_against_differences(softplus):
    N, S, C, K, G = 3, 5, 6, 3, 2
    lens = [5, 1, 0]
    inp = dict(X=normal(N, S, C, seed=1), Delta=normal(N, S, C, seed=2, scale=0.3), A=-normal(C, K, seed=3).abs(),
               B=normal(N, S, G * K, seed=4), C=normal(N, S, G * K, seed=5), D=normal(C, seed=6),
               Z=normal(N, S, C, seed=7), delta_bias=normal(C, seed=8, scale=0.3),
               initial_state=normal(N, C, K, seed=9))
    dY, dF = normal(N, S, C, seed=10), normal(N, C, K, seed=11)

    def loss(**t):
        o = ref.scan(lens=lens, softplus=softplus, groups=G, **t)
        return (o["Y"] * dY).sum() + (o["final_state"] * dF).sum()
    g = ref.scan(lens=lens, softplus=softplus, groups=G, dY=dY, d_final_state=dF, **inp)
    directional(loss, inp, {k: g[("d_" if k in ("delta_bias", "initial_state") else "d") + k] for k in inp}, seed=12)
