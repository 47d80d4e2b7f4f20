"""Plain 64-bit definitions of the linear attention operators, for the tests.

Everything is a float64 CPU tensor; rows are [batch, seq, ...].  The gradients
are the formulas written out; ``tests/test_linear_attention_host.py`` holds
them against differences of the forward definitions.
"""
import torch

F64 = torch.float64


def _live(lens, N, S):
    end = torch.full((N,), S) if lens is None else torch.as_tensor([min(max(int(x), 0), S) for x in lens])
    return torch.arange(S)[None, :] < end[:, None]


def qk(X, heads, Scale=None, Frequencies=None, positions=None, lens=None, rotary=0, interleaved=False, norm="rms",
       epsilon=1e-6, dY=None):
    """One side, queries or keys: Y, or with dY dX and dScale."""
    N, S = X.shape[:2]
    x = X.reshape(N, S, heads, -1)
    d = x.shape[-1]
    live = _live(lens, N, S)[..., None, None]
    x = torch.where(live, x, torch.zeros((), dtype=F64))
    w = torch.ones(d, dtype=F64) if Scale is None else Scale
    m = d if norm == "rms" else 1
    inv = torch.ones_like(x[..., :1]) if norm == "none" else ((x * x).sum(-1, keepdim=True) / m + epsilon) ** -0.5
    i = torch.arange(rotary // 2)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    if rotary:
        at = torch.arange(S)[None, :].expand(N, S) if positions is None else positions
        # the float32 frequency is taken as it is: the product with a whole number below 2^29 is exact
        angle = at.to(F64)[..., None, None] * Frequencies
        c, s = torch.cos(angle), torch.sin(angle)

    def turn(v, sign):
        v = v.clone()
        if rotary:
            a, b = v[..., one].clone(), v[..., two].clone()
            v[..., one], v[..., two] = a * c - sign * b * s, b * c + sign * a * s
        return v
    if dY is None:
        y = torch.where(live, turn(x * inv * w, 1), torch.zeros((), dtype=F64))
        return y.reshape(N, S, -1)
    g = torch.where(live, turn(torch.where(live, dY.reshape(N, S, heads, d), torch.zeros((), dtype=F64)), -1),
                    torch.zeros((), dtype=F64))
    dScale = (g * x * inv).sum((0, 1, 2))
    g = g * w
    dX = g if norm == "none" else inv * g - x * inv ** 3 * (g * x).sum(-1, keepdim=True) / m
    return dX.reshape(N, S, -1), dScale


def attn(Q, K, V, heads, scale, Decay=None, decay_bias=None, lens=None, initial_state=None, key_size=None,
         value_size=None, dY=None, d_final_state=None):
    """The outputs, and with dY the gradients: every step in turn."""
    N, S = Q.shape[:2]
    dk, dv = key_size, value_size
    live = _live(lens, N, S)

    def split(x, size):
        own = x.reshape(N, S, -1, size)
        return own.repeat_interleave(heads // own.shape[2], 2), own.shape[2]

    def join(x, own):
        return x.reshape(N, S, own, heads // own, -1).sum(3).reshape(N, S, -1)
    zero = torch.zeros((), dtype=F64)
    Q, K, V = (torch.where(live[..., None], x, zero) for x in (Q, K, V))
    (q, qh), (k, kh), (v, vh) = split(Q, dk), split(K, dk), split(V, dv)
    g = torch.zeros(N, S, heads, dtype=F64)
    if Decay is not None:
        g = g + Decay
    if decay_bias is not None:
        g = g + decay_bias
    g = torch.where(live[..., None], g, zero)
    h = torch.zeros(N, heads, dk, dv, dtype=F64) if initial_state is None else initial_state
    kept, Y = [], torch.zeros(N, S, heads, dv, dtype=F64)
    for t in range(S):
        on = live[:, t, None, None, None]
        kept.append(h)
        new = torch.exp(g[:, t])[..., None, None] * h + k[:, t][..., None] * v[:, t][..., None, :]
        h = torch.where(on, new, h)
        y = scale * torch.einsum("nhkv,nhk->nhv", h, q[:, t])
        Y[:, t] = torch.where(live[:, t, None, None], y, torch.zeros((), dtype=F64))
    out = dict(Y=Y.reshape(N, S, -1), final_state=h)
    if dY is None:
        return out
    do = dY.reshape(N, S, heads, dv)
    r = torch.zeros_like(h) if d_final_state is None else d_final_state
    dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg = torch.zeros_like(g)
    for t in reversed(range(S)):
        on = live[:, t, None, None].to(F64)
        y = scale * torch.where(live[:, t, None, None], do[:, t], torch.zeros((), dtype=F64))
        before, after = kept[t], (kept[t + 1] if t + 1 < S else h)
        dq[:, t] = torch.einsum("nhkv,nhv->nhk", after, y) * on
        r = r + q[:, t][..., None] * y[..., None, :] * on[..., None]
        dk_[:, t] = torch.einsum("nhkv,nhv->nhk", r, v[:, t]) * on
        dv_[:, t] = torch.einsum("nhkv,nhk->nhv", r, k[:, t]) * on
        e = torch.exp(g[:, t])[..., None, None]
        dg[:, t] = (r * e * before).sum((-1, -2)) * on[..., 0]
        r = torch.where(live[:, t, None, None, None], e * r, r)
    return dict(dQ=join(dq, qh), dK=join(dk_, kh), dV=join(dv_, vh), dDecay=dg, d_decay_bias=dg.sum((0, 1)),
                d_initial_state=r)
