"""fp64 definitions of the operators around the delta rule: the per-channel gated linear recurrence
and its gradient, layer norm and its gradient, beam selection and the reorder of states.  Plain
loops and sorts over numpy arrays, sharing nothing with the CUDA library."""
import numpy as np

GATE_LOGDECAY, GATE_NEG_SOFTPLUS = 0, 1


def decay(g, gate_mode):
    """a and 1 - a of a gate, each formed directly."""
    g = np.asarray(g, np.float64)
    if gate_mode == GATE_LOGDECAY:
        return np.exp(g), -np.expm1(g)
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, e, 1.0) / (1 + e), np.where(g >= 0, 1.0, e) / (1 + e)


def scan_fwd(x, g, h0=None, gate_mode=1, tied=False, lengths=None):
    """x, g [B,T,D]: (h with zeros behind each sequence, h_T, the state before every token)."""
    x = np.asarray(x, np.float64)
    B, T, D = x.shape
    a, rest = decay(g, gate_mode)
    n = np.full(B, T) if lengths is None else np.clip(lengths, 0, T)
    h, before = np.zeros((B, T, D)), np.zeros((B, T, D))
    s = np.zeros((B, D)) if h0 is None else np.array(h0, np.float64)
    for b in range(B):
        for t in range(T):
            before[b, t] = s[b]
            if t < n[b]:
                s[b] = a[b, t] * s[b] + (rest[b, t] if tied else 1.0) * x[b, t]
                h[b, t] = s[b]
    return h, s, before


def scan_bwd(x, g, h0, dh, dh_T, gate_mode=1, tied=False, lengths=None):
    """Gradients (dx, dg, dh0) of <dh, h> + <dh_T, h_T>."""
    x = np.asarray(x, np.float64)
    B, T, D = x.shape
    a, rest = decay(g, gate_mode)
    _, _, before = scan_fwd(x, g, h0, gate_mode, tied, lengths)
    n = np.full(B, T) if lengths is None else np.clip(lengths, 0, T)
    dx, dg = np.zeros((B, T, D)), np.zeros((B, T, D))
    m = np.zeros((B, D)) if dh_T is None else np.array(dh_T, np.float64)
    slope = a if gate_mode == GATE_LOGDECAY else -a * rest
    for b in range(B):
        for t in range(n[b] - 1, -1, -1):
            lam = m[b] + (0.0 if dh is None else dh[b, t])
            dx[b, t] = lam * (rest[b, t] if tied else 1.0)
            dg[b, t] = lam * (before[b, t] - (x[b, t] if tied else 0.0)) * slope[b, t]
            m[b] = a[b, t] * lam
    return dx, dg, m


def layernorm_fwd(x, w=None, b=None, eps=1e-5):
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if w is not None:
        y = y * w
    return (y if b is None else y + b), mean, rstd


def layernorm_bwd(x, dy, w=None, eps=1e-5):
    """(dx, dweight, dbias)."""
    hat, _, rstd = layernorm_fwd(x, eps=eps)
    dy = np.asarray(dy, np.float64)
    wd = dy if w is None else dy * w
    dx = rstd[..., None] * (wd - wd.mean(-1, keepdims=True) - hat * (wd * hat).mean(-1, keepdims=True))
    axes = tuple(range(dy.ndim - 1))
    return dx, (dy * hat).sum(axes), dy.sum(axes)


def beam_scores(logits, scores, finished=None, eos=0):
    """The 64-bit score of every continuation [G,K,V]."""
    x, sc = np.asarray(logits, np.float64), np.asarray(scores, np.float64)
    with np.errstate(all="ignore"):
        top = x.max(-1, keepdims=True)
        c = sc[..., None] + (x - (np.log(np.exp(x - top).sum(-1, keepdims=True)) + top))
        c = np.where(np.isnan(c) | (c == np.inf), -np.inf, c)
    if finished is not None:
        for g, k in np.argwhere(finished):
            c[g, k] = -np.inf
            c[g, k, eos] = sc[g, k] if sc[g, k] < np.inf else -np.inf
    return c


def beam_select(logits, scores, M, finished=None, eos=0):
    """(scores, parent, token) [G,M]: best first, equal ones by the lowest k * V + v."""
    c = beam_scores(logits, scores, finished, eos)
    G, K, V = c.shape
    flat = c.reshape(G, K * V)
    at = np.argsort(-flat, axis=1, kind="stable")[:, :M]
    return np.take_along_axis(flat, at, 1), at // V, at % V


def state_reorder(S, parent, layers=False):
    S = S if layers else S[None]
    G, K = parent.shape
    out = S.copy()
    for g in range(G):
        for j in range(K):
            if 0 <= parent[g, j] < K:
                out[:, g * K + j] = S[:, g * K + parent[g, j]]
    return out if layers else out[0]
