"""Float64 definitions of the gated linear recurrence, of its gradients and of
values kept in 8 bits, in numpy (tests only).

The recurrence, per sequence and channel, with a weight lam per channel:
    w_t = c softplus(lam) sigmoid(r_t)   a_t = exp(-w_t)
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t   y_t = h_t
"""
import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, np.float64)


def sigmoid(x):
    """exp(min(x, 0)) / (1 + exp(-|x|)): no overflow, and small values keep their digits."""
    return np.exp(np.minimum(x, 0)) / (1 + np.exp(-np.abs(x)))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def lengths(seqlens, B, L):
    return [L if seqlens is None else min(L, max(0, int(seqlens[b]))) for b in range(B)]


def gates(x, r, i, lam, c):
    """w, a, beta and sigmoid(i) of [..., D]."""
    w = c * softplus(lam) * sigmoid(r)
    return w, np.exp(-w), np.sqrt(-np.expm1(-2 * w)), sigmoid(i)


def linear_seq(x, r, i, lam, c=8.0, init=None, seqlens=None, states=None):
    """x/r/i[B,L,D] -> y[B,L,D], the final state [B,D], and the states before token 0, 64, ... (the final one past a
    sequence's end). `states`, if given, are what each 64 tokens go on from."""
    x, r, i, lam = _f(x), _f(r), _f(i), _f(lam)
    B, L, D = x.shape
    y, final, kept = np.zeros((B, L, D)), np.zeros((B, D)), np.zeros((B, -(-L // 64), D))
    for b, n in enumerate(lengths(seqlens, B, L)):
        h = np.zeros(D) if init is None else _f(init)[b].copy()
        _, a, beta, iota = gates(x[b, :n], r[b, :n], i[b, :n], lam, c)
        for t in range(L):
            if t % 64 == 0:
                h = h if states is None else _f(states)[b, t // 64]
                kept[b, t // 64] = h
            if t < n:
                h = a[t] * h + beta[t] * iota[t] * x[b, t]
                y[b, t] = h
        final[b] = h
    return y, final, kept


def linear_seq_bwd(x, r, i, lam, dy, c=8.0, init=None, dfinal=None, seqlens=None, states=None):
    """Gradients of <dy, y> + <dfinal, final> as a dict dx, dr, di, dlam, dinit; h_{t-1} as linear_seq has it."""
    x, r, i, lam, dy = _f(x), _f(r), _f(i), _f(lam), _f(dy)
    B, L, D = x.shape
    y, _, kept = linear_seq(x, r, i, lam, c, init, seqlens, states)
    g = dict(dx=np.zeros(x.shape), dr=np.zeros(x.shape), di=np.zeros(x.shape), dlam=np.zeros(D), dinit=np.zeros((B, D)))
    for b, n in enumerate(lengths(seqlens, B, L)):
        m = np.zeros(D) if dfinal is None else _f(dfinal)[b].copy()
        w, a, beta, iota = gates(x[b, :n], r[b, :n], i[b, :n], lam, c)
        rho = sigmoid(r[b, :n])
        for t in reversed(range(n)):
            before = kept[b, t // 64] if t % 64 == 0 else y[b, t - 1]
            dh = dy[b, t] + m
            g["dx"][b, t] = dh * beta[t] * iota[t]
            g["di"][b, t] = dh * beta[t] * x[b, t] * iota[t] * sigmoid(-i[b, t])
            with np.errstate(divide="ignore", invalid="ignore"):
                slope = np.where(w[t] > 0, a[t] ** 2 * w[t] / beta[t], 0.0)  # w dbeta/dw
            psi = dh * (slope * iota[t] * x[b, t] - a[t] * w[t] * before)
            g["dr"][b, t] = psi * sigmoid(-r[b, t])
            g["dlam"] += psi * sigmoid(lam) / softplus(lam)
            m = a[t] * dh
        g["dinit"][b] = m
    return g


def linear_step(state, x, r, i, lam, c=8.0, slots=None):
    """One token over a pool of states [S,D]; returns y[B,D] and the new pool."""
    new, y = _f(state).copy(), np.zeros(x.shape)
    for b in range(x.shape[0]):
        s = b if slots is None else int(slots[b])
        if 0 <= s < new.shape[0]:
            one = linear_seq(x[b][None, None], r[b][None, None], i[b][None, None], lam, c, _f(state)[s][None])
            y[b], new[s] = one[0][0, 0], one[1][0]
    return y, new


def pack8(x, seqlens=None):
    """x[B,L,...] -> whole numbers [B,L,...] and e + 127 [B,ceil(L/16),...]: 16 tokens of a channel share 2^e, e the
    least with max |x| <= 127 2^e and e >= -127; 255 and zeros for a group that is not finite."""
    x = _f(x)
    B, L = x.shape[:2]
    q, code = np.zeros(x.shape, np.int8), np.zeros((B, -(-L // 16), *x.shape[2:]), np.uint8)
    for b, n in enumerate(lengths(seqlens, B, L)):
        for j in range(-(-L // 16)):
            v = x[b, 16 * j:16 * j + 16][:max(0, n - 16 * j)]
            if not len(v):
                continue
            with np.errstate(invalid="ignore"):
                top = np.abs(v).max(0)
            fine = np.isfinite(top)
            top = np.where(fine, top, 0.0)
            e = np.full(top.shape, -127)
            while (short := top > 127 * np.exp2(e)).any():
                e = np.where(short, e + 1, e)
            q[b, 16 * j:16 * j + len(v)] = np.rint(np.where(fine, v, 0.0) / np.exp2(e))
            code[b, j] = np.where(fine, e + 127, 255)
    return q, code


def unpack8(q, code):
    scale = np.where(code == 255, np.nan, np.exp2(code.astype(np.float64) - 127))
    return q * np.repeat(scale, 16, axis=1)[:, :q.shape[1]]
