"""What is measured of the operators of a linear attention layer: their cases, inputs, plain forms and definitions.

Four operators, each over ranges of sizes and types: the normalisation and rotation of queries and keys by head and
its gradient, and attention through a state that decays by head and its gradient.  They run as prompts (many steps),
as single tokens (one step with the state carried over) and backward.

Where ``own`` is true ``run`` calls the library's operators through ``StateSpaceLayer``; where it is false it computes
the same outputs from elementary torch operations in 32 bits (angles and sums of decays in 64).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F32, F64 = torch.float32, torch.float64
EPSILON = 1e-6


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step's queries and keys of 64 requests, each at its own position: latency counts
        dict(name="qk_token", op="qk", seq=1, batch=64, heads=16, key_heads=4, size=128, rotary=128, interleaved=False,
             norm="rms", dtype="bf16", layout=0, ragged=False, far=True),
        # the queries and keys of the library's largest layer: 512 steps of 64 rows of 1024 elements
        dict(name="qk_layer", op="qk", seq=512, batch=64, heads=16, key_heads=16, size=64, rotary=64, interleaved=False,
             norm="rms", dtype="bf16", layout=0, ragged=False, far=False),
        # the same of a training step, heads of 128
        dict(name="qk_grad_layer", op="qk_grad", seq=512, batch=64, heads=8, key_heads=8, size=128, rotary=128,
             interleaved=False, norm="rms", dtype="bf16", layout=1, ragged=False, far=False),
        # float32 training on odd sizes: ragged rows, shared keys, part of each head rotated, neighbours as pairs
        dict(name="qk_grad_odd", op="qk_grad", seq=201, batch=7, heads=6, key_heads=3, size=90, rotary=34,
             interleaved=True, norm="l2", dtype="f32", layout=1, ragged=True, far=False),
        # one decode step of 64 requests: states read and written once
        dict(name="attn_token", op="attn", seq=1, batch=64, heads=16, query_heads=16, key_heads=16, value_heads=16,
             key_size=128, value_size=128, dtype="bf16", layout=0, decay="rows", ragged=False, state=True),
        # one long prompt alone: a single sequence has to fill the card
        dict(name="attn_prompt", op="attn", seq=4096, batch=1, heads=16, query_heads=16, key_heads=16, value_heads=16,
             key_size=128, value_size=128, dtype="bf16", layout=0, decay="rows", ragged=False, state=False),
        # the library's largest layer: 512 steps of 64 rows, sixteen heads of 64
        dict(name="attn_layer", op="attn", seq=512, batch=64, heads=16, query_heads=16, key_heads=16, value_heads=16,
             key_size=64, value_size=64, dtype="bf16", layout=0, decay="bias", ragged=False, state=False),
        # float32 prompts of different lengths, odd sizes, queries and keys shared by two heads, states carried over
        dict(name="attn_ragged", op="attn", seq=777, batch=8, heads=10, query_heads=5, key_heads=5, value_heads=10,
             key_size=72, value_size=103, dtype="f32", layout=1, decay="both", ragged=True, state=True),
        # a training batch of eight sequences of 512 steps
        dict(name="attn_grad", op="attn_grad", seq=512, batch=8, heads=16, query_heads=16, key_heads=16,
             value_heads=16, key_size=128, value_size=128, dtype="bf16", layout=1, decay="rows", ragged=False,
             state=False),
        # one long sequence of a training step
        dict(name="attn_grad_long", op="attn_grad", seq=4096, batch=1, heads=16, query_heads=16, key_heads=16,
             value_heads=16, key_size=128, value_size=128, dtype="bf16", layout=0, decay="rows", ragged=False,
             state=False),
        # truncated back-propagation on odd sizes: ragged float16 sequences, shared keys and values, the state's
        # gradients too
        dict(name="attn_grad_odd", op="attn_grad", seq=201, batch=3, heads=12, query_heads=12, key_heads=4,
             value_heads=4, key_size=48, value_size=80, dtype="f16", layout=0, decay="both", ragged=True, state=True),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _even(rng, n, of=8):
    """Half of the sizes keep to multiples of `of`, as a model's do; the others stay odd or even as they came."""
    return max(of, n // of * of) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["qk", "qk_grad", "attn", "attn", "attn_grad", "attn_grad"])
    case = dict(op=op, dtype=rng.choice(["f32", "f16", "bf16", "bf16"]), layout=rng.randrange(2),
                ragged=rng.random() < 0.4)
    token = op in ("qk", "attn") and rng.random() < 0.25
    if op in ("qk", "qk_grad"):
        size = rng.choice([64, 64, 128, 128, _spread(rng, 8, 256)])
        key_heads = _spread(rng, 1, 16)
        heads = key_heads * rng.choice([1, 1, 2, 4])
        case.update(heads=heads, key_heads=key_heads, size=size,
                    rotary=rng.choice([size // 2 * 2, size // 2 * 2, size // 4 * 2, 0]),
                    interleaved=rng.random() < 0.4, norm=rng.choice(["rms", "rms", "l2", "none"]),
                    far=rng.random() < 0.5)
        room = (1 << 24) // ((heads + key_heads) * size)
    else:
        heads = rng.choice([1, 2, 4, 8, 12, 16, 16, 20])
        shares = [d for d in (1, 1, 1, 2, 4) if heads % d == 0]
        shared = heads // rng.choice(shares)
        which = rng.choice(["none", "qk", "kv"])
        case.update(heads=heads, query_heads=shared if which == "qk" else heads,
                    key_heads=heads if which == "none" else shared,
                    value_heads=shared if which == "kv" else heads,
                    key_size=rng.choice([64, 64, 128, 128, _even(rng, _spread(rng, 8, 128))]),
                    value_size=rng.choice([64, 64, 128, 128, _even(rng, _spread(rng, 8, 128))]),
                    decay=rng.choice(["rows", "rows", "bias", "both", "none"]), state=rng.random() < 0.5)
        room = (1 << (24 if op == "attn" else 23)) // (heads * (case["key_size"] + case["value_size"]))
    batch = _spread(rng, 1, max(1, min(64, room)))
    case.update(batch=batch, seq=1 if token else _spread(rng, 2, max(2, min(8192, room // batch))))
    if token:
        case.update(ragged=False, **({"state": True} if op == "attn" else {}))
    return case


def _tokens(case):
    """Tokens that hold work: lengths are uniform in 1..seq where the batch is ragged."""
    return case["batch"] * (case["seq"] + 1) / 2 if case["ragged"] else case["batch"] * case["seq"]


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op, t, full = case["op"], _tokens(case), case["batch"] * case["seq"]
    if op in ("qk", "qk_grad"):
        x = (case["heads"] + case["key_heads"]) * case["size"]
        if op == "qk":
            return {"bytes": (t + full) * x * e, "flops": 8 * t * x}
        return {"bytes": (2 * t + full) * x * e + 4 * case["size"], "flops": 20 * t * x}
    h, dk, dv = case["heads"], case["key_size"], case["value_size"]
    inputs = (case["query_heads"] + case["key_heads"]) * dk + case["value_heads"] * dv
    decay = 4 * h * (1 if case["decay"] in ("rows", "both") else 0)
    state = 4 * case["batch"] * h * dk * dv
    if op == "attn":
        return {"bytes": t * (inputs * e + decay) + full * h * dv * e + state * (2 if case["state"] else 1),
                "flops": 4 * t * h * dk * dv}
    return {"bytes": (t + full) * (inputs * e + decay) + t * h * dv * e + (3 * state if case["state"] else 0),
            "flops": 12 * t * h * dk * dv}


# ---- inputs -----------------------------------------------------------------------------------

_handle = []


def _layer():
    """The program's one handle."""
    if not _handle:
        import onnx_lstm_gru_gb300 as rk
        _handle.append(rk.StateSpaceLayer())
    return _handle[0]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    op, S, N, H = case["op"], case["seq"], case["batch"], case["heads"]
    rows = (S, N) if case["layout"] == 0 else (N, S)

    def normal(*shape, scale=1.0, mean=0.0, dtype=dt):
        x = torch.randn(*shape, generator=gen, device="cuda", dtype=F32)
        return x.mul_(scale).add_(mean).to(dtype)

    s, t = {"case": case, "op": op}, {}
    if case["ragged"]:
        t["sequence_lens"] = torch.randint(1, S + 1, (N,), generator=gen, device="cuda", dtype=torch.int32)
    if op in ("qk", "qk_grad"):
        d, kh, r = case["size"], case["key_heads"], case["rotary"]
        # one projection writes queries, keys and values side by side
        wide = normal(*rows, (H + 2 * kh) * d)
        t["Q"], t["K"] = wide[..., :H * d], wide[..., H * d:(H + kh) * d]
        t["QScale"], t["KScale"] = normal(d, scale=0.1, mean=1.0), normal(d, scale=0.1, mean=1.0)
        if r:
            t["Frequencies"] = torch.exp(torch.arange(r // 2, device="cuda", dtype=F64) * (-2 / r * math.log(10000.0))).float()
            if case["far"]:  # each request goes on from where it is, some far into a long context
                start = torch.randint(0, 100000, (N,), generator=gen, device="cuda", dtype=torch.int32)
                step = torch.arange(S, device="cuda", dtype=torch.int32)
                t["positions"] = (start[None, :] + step[:, None] if case["layout"] == 0
                                  else start[:, None] + step[None, :]).contiguous()
        if op == "qk_grad":
            t["dYQ"], t["dYK"] = normal(*rows, H * d, scale=0.1), normal(*rows, kh * d, scale=0.1)
        s["tensors"] = t
        if own:
            import onnx_lstm_gru_gb300 as rk
            s.update(layer=_layer(), problem=rk.QkProblem(
                seq=S, batch=N, heads=H, key_heads=kh, size=d, rotary=r, interleaved=case["interleaved"],
                norm=case["norm"], epsilon=EPSILON, dtype=case["dtype"], layout=case["layout"]))
        return s

    dk, dv = case["key_size"], case["value_size"]
    qd, kd, vd = case["query_heads"] * dk, case["key_heads"] * dk, case["value_heads"] * dv
    # normalised queries and keys, values as the projection's slice of a wider row
    t["Q"], t["K"] = normal(*rows, qd), normal(*rows, kd)
    t["V"] = normal(*rows, vd + kd)[..., kd:]
    if case["decay"] in ("rows", "both"):  # gates: most steps keep nearly all, some forget
        x = normal(*rows, H, scale=1.5, mean=3.0, dtype=F32)
        t["Decay"] = -torch.log1p(torch.exp(-x))
    if case["decay"] in ("bias", "both"):  # memories from some ten steps to some thousand
        t["decay_bias"] = -torch.exp2(-3 - 7 * (torch.arange(H, device="cuda", dtype=F32) + 0.5) / H)
    if case["state"]:
        t["initial_state"] = normal(N, H, dk, dv, dtype=F32)
    if op == "attn_grad":
        t["dY"] = normal(*rows, H * dv, scale=0.1)
        if case["state"]:
            t["d_final_state"] = normal(N, H, dk, dv, scale=0.1, dtype=F32)
    s["tensors"] = t
    if own:
        import onnx_lstm_gru_gb300 as rk
        s.update(layer=_layer(), problem=rk.AttnProblem(
            seq=S, batch=N, heads=H, key_size=dk, value_size=dv, query_heads=case["query_heads"],
            key_heads=case["key_heads"], value_heads=case["value_heads"], scale=_scale(case), dtype=case["dtype"],
            layout=case["layout"]))
    return s


def _scale(case):
    return 1 / math.sqrt(case["key_size"])


def _names(case):
    """The outputs of a case, by the names that the library's operators give them."""
    op = case["op"]
    if op == "qk":
        return ("YQ", "YK")
    if op == "qk_grad":
        return ("dQ", "dK", "dQScale", "dKScale")
    if op == "attn":
        return ("Y", "final_state")
    names = ("dQ", "dK", "dV")
    names += ("dDecay",) if case["decay"] in ("rows", "both") else ()
    names += ("d_decay_bias",) if case["decay"] in ("bias", "both") else ()
    return names + (("d_initial_state",) if case["state"] else ())


def run(s):
    case = s["case"]
    if own:
        return getattr(s["layer"], s["op"])(s["problem"], want=_names(case), **s["tensors"])
    return {"qk": _qk, "qk_grad": _qk_grad, "attn": _attn, "attn_grad": _attn_grad}[s["op"]](case, **s["tensors"])


# ---- plain forms: elementary torch operations in 32 bits, rounded once at the end ----------------

def _live(case, sequence_lens, device):
    """Truth values of the case's rows: steps within each row's length."""
    S, N = case["seq"], case["batch"]
    step = torch.arange(S, device=device)
    if sequence_lens is None:
        live = torch.ones(N, S, dtype=torch.bool, device=device)
    else:
        live = step[None, :] < sequence_lens[:, None]
    return live if case["layout"] == 1 else live.transpose(0, 1)


def _turn(case, Frequencies, positions, device):
    """Cosines and sines by row, [.., 1, rotary / 2]; the angles are taken in 64 bits."""
    if positions is None:
        step = torch.arange(case["seq"], device=device)
        positions = step[:, None] if case["layout"] == 0 else step[None, :]
    angle = (positions.double()[..., None, None] * Frequencies.double()).remainder(2 * math.pi).float()
    return torch.cos(angle), torch.sin(angle)


def _pairs(case, x):
    """The two elements of each rotated pair, and the elements that stay."""
    r = case["rotary"]
    if case["interleaved"]:
        return x[..., :r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def _join(case, a, b, rest):
    if case["interleaved"]:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _inverse(case, x):
    if case["norm"] == "none":
        return torch.ones_like(x[..., :1])
    square = x.square()
    return ((square.mean(-1, keepdim=True) if case["norm"] == "rms" else square.sum(-1, keepdim=True)) + EPSILON).rsqrt()


def _qk(case, Q, K, QScale, KScale, Frequencies=None, positions=None, sequence_lens=None):
    live = _live(case, sequence_lens, Q.device)[..., None]
    zero = torch.zeros((), device=Q.device)

    def one(X, scale, heads):
        x = X.float().unflatten(-1, (heads, case["size"]))
        n = x * _inverse(case, x) * scale.float()
        if case["rotary"]:
            c, s = _turn(case, Frequencies, positions, Q.device)
            a, b, rest = _pairs(case, n)
            n = _join(case, a * c - b * s, b * c + a * s, rest)
        return torch.where(live, n.flatten(-2), zero).to(X.dtype)

    return {"YQ": one(Q, QScale, case["heads"]), "YK": one(K, KScale, case["key_heads"])}


def _qk_grad(case, Q, K, QScale, KScale, dYQ, dYK, Frequencies=None, positions=None, sequence_lens=None):
    live = _live(case, sequence_lens, Q.device)[..., None, None]
    zero = torch.zeros((), device=Q.device)
    d = case["size"]

    def one(X, dY, scale, heads):
        x = torch.where(live, X.float().unflatten(-1, (heads, d)), zero)
        g = torch.where(live, dY.float().unflatten(-1, (heads, d)), zero)
        if case["rotary"]:
            c, s = _turn(case, Frequencies, positions, Q.device)
            a, b, rest = _pairs(case, g)
            g = _join(case, a * c + b * s, b * c - a * s, rest)
        inv = _inverse(case, x)
        dscale = (g * x * inv).sum((0, 1, 2))
        g = g * scale.float()
        if case["norm"] == "none":
            dx = g
        else:
            dot = (g * x).sum(-1, keepdim=True) / (d if case["norm"] == "rms" else 1)
            dx = inv * g - x * (inv * inv * inv * dot)
        return torch.where(live, dx, zero).flatten(-2).to(X.dtype), dscale

    dQ, dQScale = one(Q, dYQ, QScale, case["heads"])
    dK, dKScale = one(K, dYK, KScale, case["key_heads"])
    return {"dQ": dQ, "dK": dK, "dQScale": dQScale, "dKScale": dKScale}


CHUNK = 64


def _chunks(case, x, heads, live):
    """[N, heads, chunks, steps, elements] in 32 bits from rows, steps past a row's end zero, heads that share repeated."""
    x = torch.where(live[..., None], x.float(), torch.zeros((), device=x.device))
    x = x if case["layout"] == 1 else x.transpose(0, 1)
    L = min(CHUNK, case["seq"])
    pad = -case["seq"] % L
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[0], pad, x.shape[2])], 1)
    x = x.unflatten(-1, (heads, -1)).unflatten(1, (-1, L)).permute(0, 3, 1, 2, 4)
    return x.repeat_interleave(case["heads"] // heads, 1)


def _rows(case, x, heads, dtype):
    """Back to rows; heads that shared are added up."""
    x = x.flatten(2, 3)[:, :, :case["seq"]]
    x = x.unflatten(1, (heads, -1)).sum(2) if heads < case["heads"] else x
    x = x.permute(0, 2, 1, 3).flatten(-2)
    return (x if case["layout"] == 1 else x.transpose(0, 1)).to(dtype).contiguous()


def _decays(case, live, Decay, decay_bias, device):
    """The sums of the logarithms of decays within a chunk up to each step, and the decays themselves between any two
    steps of a chunk, from its start, to its end, and between the starts of any two chunks (the last: the end)."""
    S, N, H = case["seq"], case["batch"], case["heads"]
    g = torch.zeros(*live.shape, H, dtype=F64, device=device)
    if Decay is not None:
        g = g + Decay
    if decay_bias is not None:
        g = g + decay_bias
    g = torch.where(live[..., None], g, torch.zeros((), dtype=F64, device=device))
    g = g if case["layout"] == 1 else g.transpose(0, 1)
    L = min(CHUNK, S)
    g = torch.cat([g, g.new_zeros(N, -S % L, H)], 1).unflatten(1, (-1, L)).permute(0, 3, 1, 2)
    G = g.cumsum(-1)
    total = G[..., -1]
    T = torch.cat([torch.zeros_like(total[..., :1]), total.cumsum(-1)], -1)

    def between(x):
        n = x.shape[-1]
        upto = torch.ones(n, n, dtype=torch.bool, device=device).tril()
        return torch.where(upto, torch.exp((x[..., :, None] - x[..., None, :]).clamp(max=0)).float(), torch.zeros((), device=device))

    return between(G), torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None], between(T)


def _states(W, U, first):
    """States before each chunk and behind the last, from what each chunk adds."""
    if first is None:
        first = torch.zeros_like(U[:, :, 0])
    all_ = torch.cat([first[:, :, None], U], 2)
    return (W @ all_.flatten(3)).unflatten(3, U.shape[3:])


def _attn(case, Q, K, V, Decay=None, decay_bias=None, sequence_lens=None, initial_state=None):
    live = _live(case, sequence_lens, Q.device)
    D, a, b, W = _decays(case, live, Decay, decay_bias, Q.device)
    q, k, v = (_chunks(case, x, case[n], live) for x, n in ((Q, "query_heads"), (K, "key_heads"), (V, "value_heads")))
    h = _states(W, (k * b).transpose(-1, -2) @ v, initial_state)
    y = _scale(case) * ((q @ k.transpose(-1, -2) * D) @ v + a * (q @ h[:, :, :-1]))
    return {"Y": _rows(case, y, case["heads"], V.dtype), "final_state": h[:, :, -1].clone()}


def _attn_grad(case, Q, K, V, dY, Decay=None, decay_bias=None, sequence_lens=None, initial_state=None,
               d_final_state=None):
    live = _live(case, sequence_lens, Q.device)
    D, a, b, W = _decays(case, live, Decay, decay_bias, Q.device)
    q, k, v = (_chunks(case, x, case[n], live) for x, n in ((Q, "query_heads"), (K, "key_heads"), (V, "value_heads")))
    do = _chunks(case, dY, case["heads"], live) * _scale(case)
    h = _states(W, (k * b).transpose(-1, -2) @ v, initial_state)
    # the state's gradient at each chunk's start and behind the last
    last = torch.zeros_like(h[:, :, 0]) if d_final_state is None else d_final_state
    back = torch.cat([(q * a).transpose(-1, -2) @ do, last[:, :, None]], 2)
    r = (W.transpose(-1, -2) @ back.flatten(3)).unflatten(3, h.shape[3:])
    P, dP = q @ k.transpose(-1, -2) * D, do @ v.transpose(-1, -2)
    dS = dP * D
    dq_far, dk_far = a * (do @ h[:, :, :-1].transpose(-1, -2)), b * (v @ r[:, :, 1:].transpose(-1, -2))
    out = {"dQ": _rows(case, dS @ k + dq_far, case["query_heads"], Q.dtype),
           "dK": _rows(case, dS.transpose(-1, -2) @ q + dk_far, case["key_heads"], K.dtype),
           "dV": _rows(case, P.transpose(-1, -2) @ do + b * (k @ r[:, :, 1:]), case["value_heads"], V.dtype)}
    if case["decay"] != "none":
        # a step's decay lies between every pair of steps around it: pairs within the chunk, with what comes before
        # the chunk, with what comes after it, and those two
        M = (P * dP).tril(-1).double()
        to, of = M.sum(-1) + (q * dq_far).sum(-1).double(), M.sum(-2)
        at = (k * dk_far).sum(-1).double()
        over = (h[:, :, :-1] * r[:, :, 1:]).sum((-1, -2)).double()[..., None] * a[..., -1:, 0].double()
        dg = (to - of).flip(-1).cumsum(-1).flip(-1) + at.cumsum(-1) - at + over
        dg = dg.flatten(2)[..., :case["seq"]].permute(0, 2, 1)
        dg = torch.where(live[..., None], dg if case["layout"] == 1 else dg.transpose(0, 1), torch.zeros((), dtype=F64, device=Q.device))
        if Decay is not None:
            out["dDecay"] = dg.float().contiguous()
        if decay_bias is not None:
            out["d_decay_bias"] = dg.sum((0, 1)).float()
    if case["state"]:
        out["d_initial_state"] = r[:, :, 0].clone()
    return out


# ---- the definitions in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    whole = (torch.int32,)
    t = {k: v if v.dtype in whole else v.double() for k, v in prepare(case, seed)["tensors"].items()}
    lens = t["sequence_lens"].tolist() if "sequence_lens" in t else [case["seq"]] * case["batch"]
    rows = {k: v if case["layout"] == 1 else v.transpose(0, 1) for k, v in t.items()
            if k in ("Q", "K", "V", "Decay", "dY", "dYQ", "dYK", "positions")}
    out = (_qk_exact if case["op"].startswith("qk") else _attn_exact)(case, t, rows, lens)
    for k in ("YQ", "YK", "dQ", "dK", "dV", "Y", "dDecay"):
        if k in out and case["layout"] == 0:
            out[k] = out[k].transpose(0, 1).contiguous()
    return {k: out[k] for k in _names(case)}


def _qk_exact(case, t, rows, lens):
    """Each head as a vector of complex pairs, turned by e^(i angle)."""
    d, r, back = case["size"], case["rotary"], case["op"] == "qk_grad"
    end = torch.tensor(lens, device=t["Q"].device)
    out = {}
    for X, name, heads in ((rows["Q"], "Q", case["heads"]), (rows["K"], "K", case["key_heads"])):
        N, S = X.shape[:2]
        dead = torch.arange(S, device=X.device)[None, :] >= end[:, None]
        x, w = X.reshape(N, S, heads, d).masked_fill(dead[..., None, None], 0), t[name + "Scale"]
        if r:
            position = rows["positions"].double() if "positions" in rows else torch.arange(S, device=X.device).double()[None]
            angle = position[..., None, None] * t["Frequencies"]
            wheel = torch.polar(torch.ones_like(angle), angle)

        def turned(v, by):
            z = v[..., :r].unflatten(-1, (r // 2, 2) if case["interleaved"] else (2, r // 2))
            z = z if case["interleaved"] else z.transpose(-1, -2)
            z = torch.view_as_real(torch.complex(z[..., 0], z[..., 1]) * by)
            z = z if case["interleaved"] else z.transpose(-1, -2)
            return torch.cat([z.flatten(-2), v[..., r:]], -1)

        size = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2
        m = {"rms": d, "l2": 1, "none": 1}[case["norm"]]
        inv = torch.ones_like(size) if case["norm"] == "none" else 1 / torch.sqrt(size / m + EPSILON)
        if not back:
            y = x * inv * w
            out["Y" + name] = (turned(y, wheel) if r else y).reshape(N, S, heads * d)
            continue
        g = rows["dY" + name].reshape(N, S, heads, d).masked_fill(dead[..., None, None], 0)
        g = turned(g, wheel.conj()) if r else g
        out["d" + name + "Scale"] = torch.einsum("nshd,nshd,nsh->d", g, x, inv[..., 0])
        g = g * w
        dx = inv * g
        if case["norm"] != "none":
            dx = dx - torch.einsum("nshd,nshd->nsh", g, x)[..., None] * inv ** 3 * x / m
        out["d" + name] = dx.reshape(N, S, heads * d)
    return out


def _attn_exact(case, t, rows, lens):
    """One sequence and head at a time, as a triangular matrix over all its pairs of steps."""
    N, S, H, dk, dv = case["batch"], case["seq"], case["heads"], case["key_size"], case["value_size"]
    dev, c = t["Q"].device, _scale(case)
    head = {n: [h * case[m] // H for h in range(H)] for n, m in
            (("Q", "query_heads"), ("K", "key_heads"), ("V", "value_heads"))}
    new = lambda *shape: torch.zeros(*shape, dtype=F64, device=dev)  # noqa: E731
    Y, final = new(N, S, H, dv), new(N, H, dk, dv)
    dQ, dK, dV = new(N, S, case["query_heads"], dk), new(N, S, case["key_heads"], dk), new(N, S, case["value_heads"], dv)
    dDecay, dI = new(N, S, H), new(N, H, dk, dv)
    for n in range(N):
        L = lens[n]
        for h in range(H):
            q, k, v = (rows[x][n, :L].reshape(L, -1, w)[:, head[x][h]] for x, w in (("Q", dk), ("K", dk), ("V", dv)))
            g = rows["Decay"][n, :L, h] if "Decay" in rows else new(L)
            g = g + t["decay_bias"][h] if "decay_bias" in t else g
            G = torch.cumsum(g, 0)
            h0 = t["initial_state"][n, h] if "initial_state" in t else new(dk, dv)
            D = torch.exp(torch.tril(G[:, None] - G[None, :])).tril()
            a, b = torch.exp(G)[:, None], torch.exp(G[-1] - G)[:, None]
            P = (q @ k.T).mul_(D)
            if case["op"] == "attn":
                Y[n, :L, h] = c * (P @ v + a * (q @ h0))
                final[n, h] = a[-1] * h0 + (b * k).T @ v
                continue
            do = c * rows["dY"][n, :L].reshape(L, H, dv)[:, h]
            hT = t["d_final_state"][n, h] if "d_final_state" in t else new(dk, dv)
            dV[n, :L, head["V"][h]] += P.T @ do + b * (k @ hT)
            dP = do @ v.T
            M = (P * dP).tril(-1)
            dS = dP.mul_(D)
            dQ[n, :L, head["Q"][h]] += dS @ k + a * (do @ h0.T)
            dK[n, :L, head["K"][h]] += dS.T @ q + b * (v @ hT.T)
            dI[n, h] = a[-1] * hT + (a * q).T @ do
            # pairs (i, j) with i >= step > j, the initial state before all and the final state's gradient behind all
            far, near = ((q @ h0) * do).sum(1) * a[:, 0], ((k @ hT) * v).sum(1) * b[:, 0]
            to, of = M.sum(1) + far, M.sum(0)
            suffix = (to - of).sum() - torch.cumsum(to - of, 0) + (to - of)
            dDecay[n, :L, h] = suffix + torch.cumsum(near, 0) - near + (h0 * hT).sum() * a[-1, 0]
    flat = lambda x: x.reshape(N, S, -1)  # noqa: E731
    return {"Y": flat(Y), "final_state": final, "dQ": flat(dQ), "dK": flat(dK), "dV": flat(dV), "dDecay": dDecay,
            "d_decay_bias": dDecay.sum((0, 1)), "d_initial_state": dI}
