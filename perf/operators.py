"""The gated delta rule (chunked, its backward, the one-token step) and the block norm (and its backward) as measured cases.

Each case is a dict of plain values. ``prepare`` draws its inputs on the GPU, ``run`` makes one pass through the operator
(the plain form in elementary torch operations, or the library's call where ``own`` is true), ``work`` counts what a pass
cannot do without, and ``exact`` evaluates the operator's definition token by token in float64.

The gated delta rule, per batch b and head h (keys and queries of group i = h // (H // G)), state S [P, N] in float32:

    a_t = exp(g_t)    u_t = beta_t (v_t - a_t S_{t-1} k_t)    S_t = a_t S_{t-1} + u_t k_t^T    y_t = scale S_t q_t

The block norm, per row:

    u = y silu(z)   n = u rsqrt(mean u^2 + eps) w_post   r = res + s n   out = r rsqrt(mean r^2 + eps) w_pre
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64
EPS = 1e-5


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one request decoding on the 130M-shaped layer (24 heads): the smallest call, latency alone
        dict(name="step_b1_h24", op="step", io="bf16", B=1, H=24, G=12, P=64, N=128, slots=1, idle=0),
        # a serving batch on the 2.7B-shaped layer: 64 rows of a pool of 72 states, 3 rows idle
        dict(name="step_b64_h80", op="step", io="bf16", B=64, H=80, G=40, P=64, N=128, slots=72, idle=3),
        # one prompt on the 130M-shaped layer: few chains, latency of the chain of chunks
        dict(name="prefill_b1_l4096_h24", op="prefill", io="bf16", B=1, L=4096, H=24, G=12, P=64, N=128, ragged=False),
        # a prefill batch on the 2.7B-shaped layer
        dict(name="prefill_b8_l2048_h80", op="prefill", io="bf16", B=8, L=2048, H=80, G=40, P=64, N=128, ragged=False),
        # right-padded prompts continued from cached states, square heads with their own keys; one sequence is empty
        dict(name="prefill_ragged_b6_l1000_h16_p128", op="prefill", io="bf16", B=6, L=1000, H=16, G=16, P=128, N=128,
             ragged=True),
        # a float32 model of small, odd sizes
        dict(name="prefill_f32_b2_l777_h6", op="prefill", io="f32", B=2, L=777, H=6, G=3, P=48, N=64, ragged=False),
        # training, one sequence on the 130M-shaped layer
        dict(name="train_b1_l2048_h24", op="train", io="bf16", B=1, L=2048, H=24, G=12, P=64, N=128, ragged=False),
        # training, a batch on the 2.7B-shaped layer: the largest case
        dict(name="train_b4_l2048_h80", op="train", io="bf16", B=4, L=2048, H=80, G=40, P=64, N=128, ragged=False),
        # between two blocks, one decoded token, width of the 130M-shaped model, residual in float32
        dict(name="norm_r1_d768", op="norm", io="bf16", rows=1, dim=768, z=False, post=True, res="f32"),
        # between two blocks over a prefill batch, width of the 2.7B-shaped model, gate and both norms
        dict(name="norm_r16384_d2560", op="norm", io="bf16", rows=16384, dim=2560, z=True, post=True, res="bf16"),
        # training over a batch, residual in float32
        dict(name="norm_bwd_r8192_d2560", op="norm_bwd", io="bf16", rows=8192, dim=2560, z=True, post=True, res="f32"),
        # training, float32, odd sizes
        dict(name="norm_bwd_f32_r1031_d1537", op="norm_bwd", io="f32", rows=1031, dim=1537, z=True, post=True,
             res="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """A case of the listed ranges: step and prefill up to the listed batches, training up to its largest."""
    op = rng.choice(["step", "prefill", "prefill", "train", "norm", "norm_bwd"])
    io = "f32" if rng.random() < 0.2 else "bf16"
    if op in ("norm", "norm_bwd"):
        dim = rng.choice([768, 1024, 2048, 2560, 4096, 5120, rng.randint(65, 5119)])
        rows = _log(rng, 1, 16384 * 2560 // dim // (2 if op == "norm_bwd" else 1))
        return dict(op=op, io=io, rows=rows, dim=dim, z=rng.random() < 0.6, post=rng.random() < 0.75,
                    res=rng.choice([io, "f32"]))
    P, N = rng.choice([(64, 128), (64, 128), (128, 128), (64, 64)] if io == "bf16" else [(64, 64), (48, 64), (32, 16)])
    H = rng.choice([4, 6, 8, 16, 24, 32, 80])
    G = H // rng.choice([r for r in (1, 2, 2, 4, 8) if H % r == 0])
    if op == "step":
        B = _log(rng, 1, 64 * 80 // H if P * N <= 8192 else 32 * 80 // H)
        idle = rng.randint(0, B // 4)
        return dict(op=op, io=io, B=B, H=H, G=G, P=P, N=N, slots=B + rng.randint(0, 8), idle=idle)
    most = (4 * 2048 * 80 * 64 if op == "train" else 8 * 2048 * 80 * 64) // (H * P)  # tokens of the largest case
    if io == "f32":
        most //= 64
    L = _log(rng, 1, min(8192, most))
    B = _log(rng, 1, max(1, min(8, most // L)))
    return dict(op=op, io=io, B=B, L=L, H=H, G=G, P=P, N=N, ragged=B > 1 and rng.random() < 0.4)


# ----------------------------------------------------------------- the inputs

def _unit(x):
    return x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()


def _tokens(case, gen, lead):
    """q, k (rows of norm 1), v, g (log decay of a layer with steps of 1e-3 to 1e-1) and beta in (0, 1)."""
    t, H, G, P, N = TYPES[case["io"]], case["H"], case["G"], case["P"], case["N"]
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, k = _unit(rand(*lead, G, N)).to(t), _unit(rand(*lead, G, N)).to(t)
    v = rand(*lead, H, P).to(t)
    rate = 1 + 15 * torch.rand(H, generator=gen, device="cuda")
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand((*lead, H), generator=gen, device="cuda"))
    return dict(q=q, k=k, v=v, g=(-rate * step).to(t), beta=torch.sigmoid(rand(*lead, H)).to(t))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    op, t = case["op"], TYPES[case["io"]]
    if op == "step":
        B, H, P, N, S = case["B"], case["H"], case["P"], case["N"], case["slots"]
        st = _tokens(case, gen, (B,))
        st["state"] = 0.2 * rand(S, H, P, N)
        st["new_state"] = torch.zeros_like(st["state"])
        slots = torch.randperm(S, generator=gen, device="cuda")[:B].to(torch.int32)
        idle = torch.randperm(B, generator=gen, device="cuda")[:case["idle"]]
        slots[idle] = -1
        st["slots"] = slots
    elif op in ("prefill", "train"):
        B, L, H, P, N = case["B"], case["L"], case["H"], case["P"], case["N"]
        st = _tokens(case, gen, (B, L))
        st["seqlens"] = st["init"] = None
        if case["ragged"]:  # right-padded sequences that go on from cached states; the first is whole, the last empty
            lens = 1 + (torch.rand(B, generator=gen, device="cuda") * L).long().clamp(max=L - 1)
            lens[0], lens[-1] = L, 0
            st["seqlens"] = lens.to(torch.int32)
            st["init"] = 0.2 * rand(B, H, P, N)
        if op == "train":
            st["dy"] = rand(B, L, H, P).to(t)
            st["dfinal"] = 0.1 * rand(B, H, P, N) if case["ragged"] else None
    else:
        R, D, tr = case["rows"], case["dim"], TYPES[case["res"]]
        st = dict(y=rand(R, D).to(t), res=(2 * rand(R, D)).to(tr), z=rand(R, D).to(t) if case["z"] else None,
                  pre=1 + 0.1 * rand(D), post=1 + 0.1 * rand(D) if case["post"] else None, scale=0.5 + 0.1 * rand(D))
        if op == "norm_bwd":
            st["dout"], st["dres"] = rand(R, D).to(t), rand(R, D).to(tr)
    st["op"] = op
    return st


# ------------------------------------------------------------- the plain form

def _inverse(A):
    """(I + A)^-1 of strictly lower [.., C, C], C a power of two: the blocks of size s on the diagonal, then pairs of them."""
    C = A.shape[-1]
    i = torch.arange(C, device=A.device)
    T = torch.eye(C, device=A.device).expand_as(A)
    s = 1
    while s < C:
        below = ((i[:, None] // s) == (i[None, :] // s) + 1) & ((i[:, None] // (2 * s)) == (i[None, :] // (2 * s)))
        T = T - T @ (A * below) @ T
        s *= 2
    return T


def _plain_chunked(q, k, v, g, beta, init, seqlens):
    """The chunked delta rule in float32: y [B, L, H, P] and the final state."""
    B, L, G, N = q.shape
    H, P = v.shape[2:]
    nc = -(-L // CHUNK)
    pad = nc * CHUNK - L

    def chunks(x):  # [B, L, heads, ..] -> [B, H, nc, C, ..], keys of a group for each of its heads
        if seqlens is not None:
            on = torch.arange(L, device=x.device)[None, :] < seqlens[:, None]
            x = torch.where(on.reshape(B, L, *[1] * (x.dim() - 2)), x, 0.0)
        x = x.repeat_interleave(H // x.shape[2], 2).transpose(1, 2)
        if pad:
            x = torch.cat([x, x.new_zeros(B, H, pad, *x.shape[3:])], 2)
        return x.reshape(B, H, nc, CHUNK, *x.shape[3:])

    q, k, v, g, beta = (chunks(x) for x in (q, k, v, g, beta))
    c = g.cumsum(-1)
    i = torch.arange(CHUNK, device=q.device)
    D = torch.exp(torch.where(i[:, None] >= i[None, :], c[..., :, None] - c[..., None, :], -math.inf))
    T = _inverse((i[:, None] > i[None, :]) * (beta[..., None] * D * (k @ k.transpose(-1, -2))))
    M = D * (q @ k.transpose(-1, -2))
    e = torch.exp(c)[..., None]
    tail = torch.exp(c[..., -1:] - c)[..., None]
    S = init if init is not None else q.new_zeros(B, H, P, N)
    ys = []
    for n in range(nc):
        St = S.transpose(-1, -2)
        U = T[:, :, n] @ (beta[:, :, n, :, None] * (v[:, :, n] - e[:, :, n] * (k[:, :, n] @ St)))
        ys.append(e[:, :, n] * (q[:, :, n] @ St) + M[:, :, n] @ U)
        S = e[:, :, n, -1:] * S + (tail[:, :, n] * U).transpose(-1, -2) @ k[:, :, n]
    y = torch.stack(ys, 2).reshape(B, H, nc * CHUNK, P)[:, :, :L].transpose(1, 2) * (1.0 / math.sqrt(N))
    if seqlens is not None:
        y = torch.where((torch.arange(L, device=y.device)[None, :] < seqlens[:, None])[:, :, None, None], y, 0.0)
    return y, S


def _plain_step(s):
    q, k, v, g, beta = (s[n].float() for n in ("q", "k", "v", "g", "beta"))
    r = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    on = s["slots"] >= 0
    at = s["slots"].long().clamp(min=0)
    S = s["state"][at] * torch.exp(g)[..., None, None]
    u = beta[..., None] * (v - (S @ k[..., None])[..., 0])
    S = S + u[..., None] * k[..., None, :]
    y = (S @ q[..., None])[..., 0] * (1.0 / math.sqrt(q.shape[-1]))
    y = torch.where(on[:, None, None], y, 0.0).to(s["v"].dtype)
    s["new_state"][at[on]] = S[on]
    return y, s["new_state"]


def _plain_norm(y, res, z, pre, post, scale):
    u = y if z is None else y * z * torch.sigmoid(z)
    n = u if post is None else u * torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS) * post
    r = res + scale * n
    return r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * pre, r


def _plain_norm_bwd(s):
    y, res, dout, dres, pre, post, scale = (None if s[n] is None else s[n].float()
                                            for n in ("y", "res", "dout", "dres", "pre", "post", "scale"))
    z = None if s["z"] is None else s["z"].float()
    sig = None if z is None else torch.sigmoid(z)
    u = y if z is None else y * z * sig
    tau = None if post is None else torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
    n = u if post is None else u * tau * post
    r = res + scale * n
    rho = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
    a = dout * pre
    dr = dres + rho * (a - r * rho * rho * (a * r).mean(-1, keepdim=True))
    dn = dr * scale
    du = dn
    if post is not None:
        b = dn * post
        du = tau * (b - u * tau * tau * (b * u).mean(-1, keepdim=True))
    return dict(dy=(du if z is None else du * z * sig).to(s["y"].dtype),
                dz=None if z is None else (du * y * sig * (1 + z * (1 - sig))).to(s["y"].dtype),
                dres=dr.to(s["res"].dtype), dpre_weight=(dout * r * rho).sum(0),
                dpost_weight=None if post is None else (dn * u * tau).sum(0), dscale=(dr * n).sum(0))


def _plain(s):
    op = s["op"]
    if op == "step":
        return _plain_step(s)
    if op == "prefill":
        y, S = _plain_chunked(*(s[n].float() for n in ("q", "k", "v", "g", "beta")), s["init"], s["seqlens"])
        return y.to(s["v"].dtype), S
    if op == "train":
        leaf = {n: s[n].float().requires_grad_() for n in ("q", "k", "v", "g", "beta")}
        init = None if s["init"] is None else s["init"].clone().requires_grad_()
        y, S = _plain_chunked(*leaf.values(), init, s["seqlens"])
        outs, cot = [y], [s["dy"].float()]
        if s["dfinal"] is not None:
            outs, cot = outs + [S], cot + [s["dfinal"]]
        got = torch.autograd.grad(outs, [*leaf.values()] + ([] if init is None else [init]), cot)
        out = {"d" + n: x.to(s[n].dtype) for n, x in zip(leaf, got)}
        out["dinit"] = None if init is None else got[-1]
        return out
    if op == "norm":
        x = [None if s[n] is None else s[n].float() for n in ("y", "res", "z", "pre", "post", "scale")]
        out, r = _plain_norm(*x)
        return out.to(s["y"].dtype), r.to(s["res"].dtype)
    return _plain_norm_bwd(s)


# -------------------------------------------------------------------- one pass

def run(state):
    s = state
    if not own:
        return _plain(s)
    from mamba_ssd_selective_gb300 import binding
    op = s["op"]
    if op == "step":
        y = binding.gated_delta_step(s["state"], s["q"], s["k"], s["v"], s["g"], s["beta"], slots=s["slots"],
                                     new_state=s["new_state"])
        return y, s["new_state"]
    if op == "prefill":
        return binding.gated_delta_chunked(s["q"], s["k"], s["v"], s["g"], s["beta"], init_state=s["init"],
                                           seqlens=s["seqlens"])
    if op == "train":
        return binding.gated_delta_chunked_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dy"],
                                               init_state=s["init"], dfinal_state=s["dfinal"], seqlens=s["seqlens"],
                                               want_dinit=s["init"] is not None)
    if op == "norm":
        return binding.block_norm(s["y"], s["res"], s["pre"], post_weight=s["post"], z=s["z"], scale=s["scale"],
                                  eps=EPS)
    return binding.block_norm_bwd(s["y"], s["res"], s["dout"], s["pre"], dres_out=s["dres"], post_weight=s["post"],
                                  z=s["z"], scale=s["scale"], eps=EPS)


# -------------------------------------------------------------------- its work

def work(case):
    op, e = case["op"], 2 if case["io"] == "bf16" else 4
    if op in ("norm", "norm_bwd"):
        n, er, nz = case["rows"] * case["dim"], 2 if case["res"] == "bf16" else 4, 1 if case["z"] else 0
        if op == "norm":  # y, z, out; res, res_out
            return {"bytes": n * (e * (2 + nz) + 2 * er) + 12 * case["dim"], "flops": n * (12 + 4 * nz)}
        # y, z, dout, dy, dz; res, dres_out, dres
        return {"bytes": n * (e * (3 + 2 * nz) + 3 * er) + 24 * case["dim"], "flops": n * (30 + 10 * nz)}
    B, H, G, P, N = (case[x] for x in ("B", "H", "G", "P", "N"))
    if op == "step":
        rows = B - case["idle"]
        return {"bytes": 8 * rows * H * P * N + e * (rows * (2 * G * N + H * P + 2 * H) + B * H * P) + 4 * B,
                "flops": 7 * rows * H * P * N}
    T = B * case["L"] if not case["ragged"] else case["L"] + (B - 2) * (case["L"] + 1) // 2  # tokens, the mean if ragged
    states = 4 * B * H * P * N
    tok = e * (2 * G * N + H * P + 2 * H)
    if op == "prefill":  # tokens in, y whole, final state out, the initial one in
        return {"bytes": T * tok + e * B * case["L"] * H * P + states * (2 if case["ragged"] else 1),
                "flops": 6 * T * H * P * N}
    # tokens and dy in, gradients whole
    return {"bytes": T * (tok + e * H * P) + B * case["L"] * tok + (3 * states if case["ragged"] else 0),
            "flops": 16 * T * H * P * N}


# -------------------------------------------------- the definition in 64 bits

def _exact_tokens(s):
    r = s["v"].shape[-2] // s["q"].shape[-2]
    x = {n: s[n].double() for n in ("q", "k", "v", "g", "beta")}
    x["q"], x["k"] = x["q"].repeat_interleave(r, -2), x["k"].repeat_interleave(r, -2)
    return x, r, 1.0 / math.sqrt(s["q"].shape[-1])


def _dot(a, b):
    return (a * b).sum(-1)


def exact(case, seed):
    """Token by token in float64; the backward walks the stored states in reverse."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = [None if s[n] is None else s[n].double() for n in ("y", "res", "z", "pre", "post", "scale")]
        y, res, z, pre, post, scale = x
        if z is not None:
            y = y * z / (1 + torch.exp(-z))
        if post is not None:
            y = y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS) * post
        r = res + scale * y
        return r / torch.sqrt((r * r).mean(1, keepdim=True) + EPS) * pre, r
    if op == "norm_bwd":
        leaf = {n: s[n].double().requires_grad_() for n in ("y", "z", "res", "pre", "post", "scale") if s[n] is not None}
        u = leaf["y"] * leaf["z"] / (1 + torch.exp(-leaf["z"])) if "z" in leaf else leaf["y"]
        if "post" in leaf:
            u = u / torch.sqrt((u * u).mean(1, keepdim=True) + EPS) * leaf["post"]
        r = leaf["res"] + leaf["scale"] * u
        out = r / torch.sqrt((r * r).mean(1, keepdim=True) + EPS) * leaf["pre"]
        got = dict(zip(leaf, torch.autograd.grad([out, r], [*leaf.values()], [s["dout"].double(), s["dres"].double()])))
        return dict(dy=got["y"], dz=got.get("z"), dres=got["res"], dpre_weight=got["pre"], dpost_weight=got.get("post"),
                    dscale=got["scale"])
    x, r, scale = _exact_tokens(s)
    if op == "step":
        on = (s["slots"] >= 0).nonzero()[:, 0]
        at = s["slots"][on].long()
        k, q = x["k"][on], x["q"][on]
        S = s["state"][at].double() * torch.exp(x["g"][on])[..., None, None]
        S = S + (x["beta"][on, :, None] * (x["v"][on] - _dot(S, k[:, :, None])))[..., None] * k[:, :, None]
        y = torch.zeros_like(x["v"])
        y[on] = _dot(S, q[:, :, None]) * scale
        new = s["new_state"].double()
        new[at] = S
        return y, new
    B, L, H, P = s["v"].shape
    N = s["q"].shape[-1]
    if op == "train" and 8 * B * L * H * P * N > 60e9:
        return None
    lens = torch.full((B,), L, device="cuda") if s["seqlens"] is None else s["seqlens"]
    on = (torch.arange(L, device="cuda")[None, :] < lens[:, None])[..., None]  # [B, L, 1]
    x["g"], x["beta"] = torch.where(on, x["g"], 0.0), torch.where(on, x["beta"], 0.0)
    S = torch.zeros(B, H, P, N, dtype=torch.float64, device="cuda") if s["init"] is None else s["init"].double()
    a = torch.exp(x["g"])
    kept, y = [], torch.zeros_like(x["v"])
    for t in range(L):
        if op == "train":
            kept.append(S)
        k = x["k"][:, t, :, None]
        S = S * a[:, t, :, None, None]
        S = S + (x["beta"][:, t, :, None] * (x["v"][:, t] - _dot(S, k)))[..., None] * k
        y[:, t] = _dot(S, x["q"][:, t, :, None]) * scale
    if op == "prefill":
        return torch.where(on[..., None], y, 0.0), S
    del y
    E = torch.zeros_like(S) if s["dfinal"] is None else s["dfinal"].double()
    dy = torch.where(on[..., None], s["dy"].double(), 0.0) * scale
    d = {n: torch.zeros_like(x[n]) for n in x}
    for t in reversed(range(L)):
        k, q, b = x["k"][:, t, :, None], x["q"][:, t, :, None], x["beta"][:, t, :, None]
        F = kept.pop() * a[:, t, :, None, None]  # the decayed state, before the update
        w = x["v"][:, t] - _dot(F, k)
        S = F + (b * w)[..., None] * k
        d["q"][:, t] = (dy[:, t, ..., None] * S).sum(-2)
        E = E + dy[:, t, ..., None] * q
        du = _dot(E, k)
        d["v"][:, t] = b * du
        d["beta"][:, t] = (du * w).sum(-1)
        d["k"][:, t] = ((b * w)[..., None] * E - (b * du)[..., None] * F).sum(-2)
        E = E - (b * du)[..., None] * k
        d["g"][:, t] = (E * F).sum((-1, -2))
        E = E * a[:, t, :, None, None]
    for n in ("q", "k"):
        d[n] = torch.where(on[..., None], d[n], 0.0).reshape(B, L, H // r, r, N).sum(3)
    for n in ("g", "beta"):
        d[n] = torch.where(on, d[n], 0.0)
    out = {"d" + n: d[n] for n in ("q", "k", "v", "g", "beta")}
    out["dinit"] = None if s["init"] is None else E
    return out
