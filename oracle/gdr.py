"""The gated delta rule's definitions in float64, for tests: plain numpy token
loops that share no code with the library.  Arrays or torch tensors in,
float64 arrays out."""
import numpy as np

SOFTPLUS, BETA_SIGMOID, QK_L2NORM = 1, 8, 16


def _f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        a = a.detach().cpu().double().numpy()
    return np.array(a, dtype=np.float64)


def _silu(v):
    return v / (1 + np.exp(-v))


def gdr_scan(q, k, v, dt, A, beta, dt_bias=None, h0=None, *, scale, flags=25, l2_eps=1e-6):
    """q, k [b, L, Hk, K]; v [b, L, H, V]; dt (or None), beta [b, L, H]; A,
    dt_bias [H]; h0 [b, H, K, V].  Returns y [b, L, H, V], the last state and
    the state after every token [b, L, H, K, V]."""
    q, k, v, dt, A, beta, dt_bias, h0 = map(_f64, (q, k, v, dt, A, beta, dt_bias, h0))
    b, L, H, V = v.shape
    K, per = k.shape[3], H // k.shape[2]
    if flags & QK_L2NORM:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True) + l2_eps) for x in (q, k))
    q, k = np.repeat(q, per, axis=2), np.repeat(k, per, axis=2)
    a = np.ones((b, L, H))
    if dt is not None:
        d = dt + (0 if dt_bias is None else dt_bias)
        a = np.exp((np.logaddexp(0, d) if flags & SOFTPLUS else d) * A)
    if flags & BETA_SIGMOID:
        beta = 1 / (1 + np.exp(-beta))
    S = np.zeros((b, H, K, V)) if h0 is None else h0
    y, states = np.zeros(v.shape), np.zeros((b, L, H, K, V))
    for t in range(L):
        S = S * a[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - np.einsum("bhkv,bhk->bhv", S, k[:, t]))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        y[:, t] = scale * np.einsum("bhkv,bhk->bhv", S, q[:, t])
        states[:, t] = S
    return y, S, states


def head_rmsnorm(x, z=None, weight=None, eps=1e-5):
    x, z, weight = map(_f64, (x, z, weight))
    out = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        out = out * weight
    return out if z is None else out * _silu(z)


def conv1d_packed(x, w, bias, state, lengths, act=True):
    """x [T, C], the sequences of `lengths` one behind the other; state
    [n, C, W - 1] or None.  Returns the rows of the sequences and the states
    after them."""
    x, w, bias, state = map(_f64, (x, w, bias, state))
    W, begin, rows, states = w.shape[1], 0, [], []
    for i, length in enumerate(lengths):
        before = np.zeros((W - 1, x.shape[1])) if state is None else state[i].T
        line = np.concatenate([before, x[begin:begin + length]])
        out = np.zeros((length, x.shape[1])) + (0 if bias is None else bias)
        for j in range(W):
            out = out + line[j:j + length] * w[:, j]
        rows.append(_silu(out) if act else out)
        states.append(line[length:].T)
        begin += length
    return np.concatenate(rows), np.stack(states)
