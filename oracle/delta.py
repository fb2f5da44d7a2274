"""Float64 definitions of the gated delta rule, of the block norm, and of their
gradients, in numpy (tests only).

The rule, per batch b and head h, keys and queries of group h // (H // G):
    F = exp(g_t) S_{t-1}   w = v_t - F k_t   S_t = F + beta_t w k_t^T   y_t = scale S_t q_t
"""
import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, np.float64)


def _heads(x, H):
    return np.repeat(_f(x), H // x.shape[-2], axis=-2)


def delta_seq(q, k, v, g, beta, init=None, seqlens=None, scale=None):
    """q/k[B,L,G,N], v[B,L,H,P], g/beta[B,L,H] -> y[B,L,H,P], final state [B,H,P,N]."""
    B, L, H, P = v.shape
    N = q.shape[-1]
    scale = N ** -0.5 if scale is None else scale
    q, k, v, g, beta = _heads(q, H), _heads(k, H), _f(v), _f(g), _f(beta)
    S = np.zeros((B, H, P, N)) if init is None else _f(init).copy()
    y = np.zeros((B, L, H, P))
    for b in range(B):
        for t in range(L if seqlens is None else min(L, max(0, int(seqlens[b])))):
            F = np.exp(g[b, t])[:, None, None] * S[b]
            w = v[b, t] - np.einsum("hpn,hn->hp", F, k[b, t])
            S[b] = F + (beta[b, t][:, None] * w)[..., None] * k[b, t][:, None, :]
            y[b, t] = scale * np.einsum("hpn,hn->hp", S[b], q[b, t])
    return y, S


def delta_seq_bwd(q, k, v, g, beta, dy, init=None, dfinal=None, seqlens=None, scale=None):
    """Gradients of <dy, y> + <dfinal, final> as a dict dq, dk, dv, dg, dbeta, dinit."""
    B, L, H, P = v.shape
    G, N = q.shape[-2:]
    scale = N ** -0.5 if scale is None else scale
    qh, kh, v, g, beta, dy = _heads(q, H), _heads(k, H), _f(v), _f(g), _f(beta), _f(dy)
    d = dict(dq=np.zeros(qh.shape), dk=np.zeros(kh.shape), dv=np.zeros(v.shape), dg=np.zeros(g.shape),
             dbeta=np.zeros(beta.shape), dinit=np.zeros((B, H, P, N)))
    for b in range(B):
        n = L if seqlens is None else min(L, max(0, int(seqlens[b])))
        S = np.zeros((H, P, N)) if init is None else _f(init)[b]
        kept = []
        for t in range(n):
            kept.append(S)
            F = np.exp(g[b, t])[:, None, None] * S
            w = v[b, t] - np.einsum("hpn,hn->hp", F, kh[b, t])
            S = F + (beta[b, t][:, None] * w)[..., None] * kh[b, t][:, None, :]
        E = np.zeros((H, P, N)) if dfinal is None else _f(dfinal)[b].copy()
        for t in reversed(range(n)):
            a, bt, kt = np.exp(g[b, t])[:, None, None], beta[b, t][:, None], kh[b, t]
            F = a * kept[t]
            w = v[b, t] - np.einsum("hpn,hn->hp", F, kt)
            S = F + (bt * w)[..., None] * kt[:, None, :]
            o = scale * dy[b, t]
            d["dq"][b, t] = np.einsum("hp,hpn->hn", o, S)
            E = E + o[..., None] * qh[b, t][:, None, :]
            du = np.einsum("hpn,hn->hp", E, kt)
            d["dv"][b, t] = bt * du
            d["dbeta"][b, t] = (du * w).sum(-1)
            d["dk"][b, t] = np.einsum("hp,hpn->hn", bt * w, E) - np.einsum("hp,hpn->hn", bt * du, F)
            E = E - (bt * du)[..., None] * kt[:, None, :]
            d["dg"][b, t] = (E * F).sum((-1, -2))
            E = a * E
        d["dinit"][b] = E
    for n in ("dq", "dk"):
        d[n] = d[n].reshape(B, L, G, H // G, N).sum(3)
    return d


def delta_step(state, q, k, v, g, beta, slots=None, scale=None):
    """One token over a pool of states [S,H,P,N]; returns y[B,H,P] and the new pool."""
    new, y = _f(state).copy(), np.zeros(v.shape)
    for b in range(v.shape[0]):
        s = b if slots is None else int(slots[b])
        if 0 <= s < new.shape[0]:
            yb, Sb = delta_seq(*(x[b][None, None] for x in (q, k, v, g, beta)), init=_f(state)[s][None], scale=scale)
            y[b], new[s] = yb[0, 0], Sb[0]
    return y, new


def block_norm(y, res, pre, post=None, z=None, scale=None, eps=1e-5):
    u, res = _f(y), _f(res)
    if z is not None:
        u = u * _f(z) / (1 + np.exp(-_f(z)))
    n = u if post is None else u / np.sqrt((u * u).mean(1, keepdims=True) + eps) * _f(post)
    r = res + (n if scale is None else _f(scale) * n)
    return r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * _f(pre), r


def block_norm_bwd(y, res, dout, pre, dres_out=None, post=None, z=None, scale=None, eps=1e-5):
    y, res, dout, pre = _f(y), _f(res), _f(dout), _f(pre)
    sg = None if z is None else 1 / (1 + np.exp(-_f(z)))
    u = y if z is None else y * _f(z) * sg
    tau = 1.0 if post is None else 1 / np.sqrt((u * u).mean(1, keepdims=True) + eps)
    n = u if post is None else u * tau * _f(post)
    s = 1.0 if scale is None else _f(scale)
    r = res + s * n
    rho = 1 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    a = dout * pre
    dr = rho * (a - r * rho ** 2 * (a * r).mean(1, keepdims=True))
    if dres_out is not None:
        dr = dr + _f(dres_out)
    dn = dr * s
    du = dn
    if post is not None:
        b = dn * _f(post)
        du = tau * (b - u * tau ** 2 * (b * u).mean(1, keepdims=True))
    return dict(dy=du if z is None else du * _f(z) * sg,
                dz=None if z is None else du * y * sg * (1 + _f(z) * (1 - sg)), dres=dr,
                dpre_weight=(dout * r * rho).sum(0), dpost_weight=None if post is None else (dn * u * tau).sum(0),
                dscale=None if scale is None else (dr * n).sum(0))
