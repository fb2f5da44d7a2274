"""The gated linear recurrence (over sequences, its backward, one token over a pool of states) and activation checkpoints in
8 bits (written by the forward, read by the backward, and on their own) as measured cases.

Each case is a dict of plain values. ``prepare`` draws its inputs on the GPU, ``run`` makes one pass through the operator
(the plain form in elementary torch operations, or the library's calls where ``own`` is true), ``work`` counts what a pass
cannot do without, and ``exact`` evaluates the operator's definition token by token in float64.

The recurrence, per sequence and channel, with lam a weight per channel:

    w_t = c softplus(lam) sigmoid(r_t)    a_t = exp(-w_t)    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t    y_t = h_t

A checkpoint keeps x, r and i in 8 bits: 16 tokens of a channel (tokens 16 j to 16 j + 15 of a sequence) share 2^e, e the
least whole number with max |x| <= 127 2^e and e >= -127, and each value is the whole number nearest to x / 2^e (ties to even).
With it go the states that enter each 64 tokens, in float32, from which the backward forms h again.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
C = 8.0
GROUP = 16
CHUNK = 64


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one request decoding, width of the 130M-shaped layer: the smallest call, latency alone
        dict(name="step_b1_d1536", op="step", io="bf16", B=1, D=1536, slots=1, idle=0),
        # a serving batch on the 2.7B-shaped layer: 256 rows of a pool of 300 states, 7 rows idle
        dict(name="step_b256_d5120", op="step", io="bf16", B=256, D=5120, slots=300, idle=7),
        # one long prompt on the 130M-shaped layer: few channels, the sequence has to be split
        dict(name="prefill_b1_l65536_d1536", op="prefill", io="bf16", B=1, L=65536, D=1536, ragged=False),
        # a prefill batch on the 2.7B-shaped layer: the largest case
        dict(name="prefill_b8_l2048_d5120", op="prefill", io="bf16", B=8, L=2048, D=5120, ragged=False),
        # right-padded prompts that go on from cached states; one sequence is empty
        dict(name="prefill_ragged_b6_l1000_d2560", op="prefill", io="bf16", B=6, L=1000, D=2560, ragged=True),
        # a float32 model of odd sizes
        dict(name="prefill_f32_b2_l777_d1537", op="prefill", io="f32", B=2, L=777, D=1537, ragged=False),
        # training, a batch on the 2.7B-shaped layer, the forward's states kept
        dict(name="train_b4_l2048_d5120", op="train", io="bf16", B=4, L=2048, D=5120, ragged=False, states=True),
        # training, float32, odd sizes, right-padded sequences from given states, from the inputs alone
        dict(name="train_f32_ragged_b5_l333_d1001", op="train", io="f32", B=5, L=333, D=1001, ragged=True, states=False),
        # training with checkpoints in 8 bits: forward that writes them, then the backward that reads them
        dict(name="train8_b4_l2048_d5120", op="train8", io="bf16", B=4, L=2048, D=5120, ragged=False),
        # the same on a small right-padded batch of an odd width
        dict(name="train8_ragged_b3_l517_d771", op="train8", io="bf16", B=3, L=517, D=771, ragged=True),
        # the activations of any other layer to 8 bits and back, at the 2.7B-shaped layer's model width
        dict(name="pack_b8_l2048_d2560", op="pack", io="bf16", B=8, L=2048, D=2560),
        # the same in float32, odd sizes
        dict(name="pack_f32_b3_l1031_d769", op="pack", io="f32", B=3, L=1031, D=769),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """A case of the listed ranges: any length from one token, widths even and odd, up to the largest listed case's work."""
    op = rng.choice(["step", "prefill", "prefill", "train", "train", "train8", "pack"])
    io = "f32" if rng.random() < 0.25 else "bf16"
    D = rng.choice([768, 1024, 1536, 2560, 4096, 5120, 2 * rng.randint(33, 2559), rng.randint(65, 5119)])
    if op == "step":
        B = _log(rng, 1, 256)
        return dict(op=op, io=io, B=B, D=D, slots=B + rng.randint(0, 44), idle=rng.randint(0, B // 4))
    most = {"prefill": 8, "train": 4, "train8": 4, "pack": 8}[op] * 2048 * 5120 // D
    if io == "f32":
        most //= 2
    L = _log(rng, 1, min(65536, most))
    B = _log(rng, 1, max(1, min(64, most // L)))
    case = dict(op=op, io=io, B=B, L=L, D=D)
    if op != "pack":
        case["ragged"] = B > 1 and rng.random() < 0.4
    if op == "train":
        case["states"] = rng.random() < 0.6
    return case


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    unif = lambda *s: torch.rand(s, generator=gen, device="cuda")  # noqa: E731
    op, t, B, D = case["op"], TYPES[case["io"]], case["B"], case["D"]
    if op == "pack":  # activations with a few strong channels
        return dict(op=op, x=(rand(B, case["L"], D) * torch.exp(rand(D))).to(t))
    lead = (B,) if op == "step" else (B, case["L"])
    # a decay between 0.9 and 0.999 a token where the gate is open, as such layers start out
    rate = -torch.log(0.9 + 0.099 * unif(D)) / C
    s = dict(op=op, x=rand(*lead, D).to(t), r=rand(*lead, D).to(t), i=rand(*lead, D).to(t), lam=torch.log(torch.expm1(rate)))
    if op == "step":
        s["state"] = 0.5 * rand(case["slots"], D)
        s["new_state"] = torch.zeros_like(s["state"])
        slots = torch.randperm(case["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
        slots[torch.randperm(B, generator=gen, device="cuda")[:case["idle"]]] = -1
        s["slots"] = slots
        return s
    s["seqlens"] = s["init"] = s["dfinal"] = s["states"] = None
    if case["ragged"]:  # right-padded, from cached states; the first sequence is whole, the last empty
        lens = 1 + (unif(B) * case["L"]).long().clamp(max=case["L"] - 1)
        lens[0], lens[-1] = case["L"], 0
        s["seqlens"], s["init"] = lens.to(torch.int32), 0.5 * rand(B, D)
    if op in ("train", "train8"):
        s["dy"] = rand(*lead, D).to(t)
        if case["ragged"]:
            s["dfinal"] = 0.3 * rand(B, D)
    if op == "train" and case["states"]:
        s["states"] = _plain_forward(s)[1]
    return s


# ------------------------------------------------------------- the plain form

def _scan(a, b, h):
    """h_t = a_t h_{t-1} + b_t along dimension 1 from h (or zero), by doubling."""
    if h is not None:
        b = torch.cat([b[:, :1] + a[:, :1] * h[:, None], b[:, 1:]], 1)
    s = 1
    while s < b.shape[1]:
        b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _on(s):
    if s["seqlens"] is None:
        return None
    return (torch.arange(s["x"].shape[1], device="cuda")[None, :] < s["seqlens"][:, None])[..., None]


def _gates(x, r, i, lam, on):
    """w, a, beta, sigmoid(r), sigmoid(i) and b of every token; nothing happens at the tokens that are not on."""
    x, r, i = x.float(), r.float(), i.float()
    if on is not None:
        x, r, i = (torch.where(on, v, 0.0) for v in (x, r, i))
    rho, iota = torch.sigmoid(r), torch.sigmoid(i)
    w = C * torch.log1p(torch.exp(lam)) * rho
    if on is not None:
        w = torch.where(on, w, 0.0)
    beta = torch.sqrt(-torch.expm1(-2 * w))
    return w, torch.exp(-w), beta, rho, iota, beta * iota * x


def _chunked(v, fill):
    """[B, L, D] as [B * chunks, CHUNK, D], the end filled up."""
    B, L, D = v.shape
    pad = -L % CHUNK
    if pad:
        v = torch.cat([v, v.new_full((B, pad, D), fill)], 1)
    return v.reshape(-1, CHUNK, D)


def _plain_forward(s):
    """h in float32 [B, L, D], and the states that enter each CHUNK tokens."""
    on = _on(s)
    _, a, _, _, _, b = _gates(s["x"], s["r"], s["i"], s["lam"], on)
    h = _scan(a, b, s["init"])
    first = torch.zeros_like(h[:, 0]) if s["init"] is None else s["init"]
    return h, torch.cat([first[:, None], h[:, CHUNK - 1:-1:CHUNK]], 1).contiguous(), on


def _plain_backward(s, x, r, i, states, on):
    """The gradients at x, r, i; h goes on from `states` in each chunk, or from the initial state."""
    B, L, D = x.shape
    w, a, beta, rho, iota, b = _gates(x, r, i, s["lam"], on)
    if states is None:
        h = _scan(a, b, s["init"])
        first = torch.zeros_like(h[:, 0]) if s["init"] is None else s["init"]
        before = torch.cat([first[:, None], h[:, :-1]], 1)
    else:
        first = states.reshape(-1, D)
        h = _scan(_chunked(a, 1.0), _chunked(b, 0.0), first)
        before = torch.cat([first[:, None], h[:, :-1]], 1).reshape(B, -1, D)[:, :L]
    dy = s["dy"].float()
    if on is not None:
        dy = torch.where(on, dy, 0.0)
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)  # the decay between this token and the next
    dh = _scan(after.flip(1), dy.flip(1), s["dfinal"]).flip(1)
    ratio = torch.where(w > 0, w / (beta * beta), 0.5)  # w / (1 - exp(-2 w))
    psi = dh * (a * a * ratio * b - a * w * before)
    out = dict(dx=dh * beta * iota, dr=psi * (1 - rho), di=dh * b * (1 - iota))
    if on is not None:
        out = {n: torch.where(on, v, 0.0) for n, v in out.items()}
    out = {n: v.to(s["dy"].dtype) for n, v in out.items()}
    out["dlam"] = torch.sigmoid(s["lam"]) / torch.log1p(torch.exp(s["lam"])) * psi.sum((0, 1))
    out["dinit"] = None if s["init"] is None else a[:, 0] * dh[:, 0]
    return out


def _plain_pack(x):
    """What x stands for after 8 bits."""
    B, L, D = x.shape
    pad = -L % GROUP
    v = x.float()
    if pad:
        v = torch.cat([v, v.new_zeros(B, pad, D)], 1)
    v = v.reshape(B, -1, GROUP, D)
    m, e = torch.frexp(v.abs().amax(2, keepdim=True))  # m 2^e, 1/2 <= m < 1
    e = torch.where(m <= 127 / 128, e - 7, e - 6).clamp(min=-127)
    v = torch.ldexp(torch.round(torch.ldexp(v, -e)), e)
    return v.reshape(B, -1, D)[:, :L].to(x.dtype)


def _plain(s):
    op = s["op"]
    if op == "pack":
        return _plain_pack(s["x"])
    if op == "step":
        on = s["slots"] >= 0
        at = s["slots"].long().clamp(min=0)
        _, a, _, _, _, b = _gates(s["x"], s["r"], s["i"], s["lam"], None)
        h = a * s["state"][at] + b
        s["new_state"][at[on]] = h[on]
        return torch.where(on[:, None], h, 0.0).to(s["x"].dtype), s["new_state"]
    if op == "train":
        return _plain_backward(s, s["x"], s["r"], s["i"], s["states"], _on(s))
    h, states, on = _plain_forward(s)
    y = (h if on is None else torch.where(on, h, 0.0)).to(s["x"].dtype)
    out = dict(y=y, final=h[:, -1].contiguous())
    if op == "train8":
        kept = [s[n] if on is None else torch.where(on, s[n], 0.0) for n in ("x", "r", "i")]
        out.update(_plain_backward(s, *(_plain_pack(v) for v in kept), states, on))
    return out


# -------------------------------------------------------------------- one pass

def run(state):
    s = state
    if not own:
        return _plain(s)
    from mamba_ssd_selective_gb300 import binding
    op = s["op"]
    if op == "pack":
        values, scales = binding.pack8(s["x"])
        return binding.unpack8(values, scales, s["x"].dtype)
    if op == "step":
        y = binding.gated_linear_step(s["state"], s["x"], s["r"], s["i"], s["lam"], c=C, slots=s["slots"],
                                      new_state=s["new_state"])
        return y, s["new_state"]
    if op == "train":
        g = binding.gated_linear_chunked_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], c=C, init_state=s["init"],
                                             states=s["states"], dfinal_state=s["dfinal"], seqlens=s["seqlens"],
                                             want_dinit=s["init"] is not None)
        return dict(dx=g["dx"], dr=g["dr"], di=g["di"], dlam=g["dlam"], dinit=g["dinit"])
    kept = binding.gated_linear_checkpoint(s["x"]) if op == "train8" else {}
    y, final = binding.gated_linear_chunked(s["x"], s["r"], s["i"], s["lam"], c=C, init_state=s["init"],
                                            seqlens=s["seqlens"], **kept)
    out = dict(y=y, final=final)
    if op == "train8":
        g = binding.gated_linear_chunked_bwd_packed(lam=s["lam"], dy=s["dy"], c=C, dfinal_state=s["dfinal"],
                                                    seqlens=s["seqlens"], want_dinit=s["init"] is not None, **kept)
        out.update(dx=g["dx"], dr=g["dr"], di=g["di"], dlam=g["dlam"], dinit=g["dinit"])
    return out


# -------------------------------------------------------------------- its work

def work(case):
    op, e, B, D = case["op"], 2 if case["io"] == "bf16" else 4, case["B"], case["D"]
    if op == "step":
        rows = B - case["idle"]
        return {"bytes": rows * D * (3 * e + 8) + B * D * e + 4 * D + 4 * B, "flops": 24 * rows * D}
    L = case["L"]
    whole = B * L * D
    groups = B * -(-L // GROUP) * D
    if op == "pack":  # in, 8 bits and scales written and read, out
        return {"bytes": 2 * e * whole + 2 * (whole + groups), "flops": 5 * whole}
    n = whole if not case["ragged"] else (L + max(0, B - 2) * (L + 1) // 2) * D  # the mean if ragged
    state = 4 * B * D
    states = 4 * B * -(-L // CHUNK) * D
    some = 2 if case["ragged"] else 0  # an initial state and its gradient, a gradient of the final one
    forward = 3 * e * n + e * whole + state * (2 if case["ragged"] else 1) + 4 * D
    if op == "prefill":  # tokens in, y whole, final state
        return {"bytes": forward, "flops": 24 * n}
    grads = e * n + 3 * e * whole + 8 * D + some * state  # dy in, gradients whole
    if op == "train":
        return {"bytes": grads + 3 * e * n + (states if case["states"] else state * (some // 2)), "flops": 50 * n}
    packed = 3 * (whole + groups)
    return {"bytes": forward + packed + states + grads + 3 * n + 3 * groups + states, "flops": 80 * n}


# -------------------------------------------------- the definition in 64 bits

def _exact_round(x, on):
    """What 8 bits keep of x[B, L, D], in float64: every step is exact but the logarithm, whose result is put right."""
    x = x.double()
    if on is not None:
        x = x * on
    out = torch.empty_like(x)
    for j in range(0, x.shape[1], GROUP):
        top = x[:, j:j + GROUP].abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 127))
        e = torch.where(top > 127 * torch.exp2(e), e + 1, e)
        e = torch.where(top <= 127 * torch.exp2(e - 1), e - 1, e).clamp(min=-127.0)
        unit = torch.exp2(e)
        q = torch.floor(x[:, j:j + GROUP] / unit)
        rest = x[:, j:j + GROUP] / unit - q
        up = (rest > 0.5) | ((rest == 0.5) & (torch.remainder(q, 2) == 1))
        out[:, j:j + GROUP] = (q + up) * unit
    return out


def exact(case, seed):
    """Token by token in float64; the backward walks the states in reverse."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "pack":
        return _exact_round(s["x"], None)
    rate = C * torch.log1p(torch.exp(s["lam"].double()))

    def token(x, r, i):
        rho, iota = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-i))
        w = rate * rho
        return rho, iota, w, torch.exp(-w), torch.sqrt(-torch.expm1(-2 * w))

    if op == "step":
        on = (s["slots"] >= 0).nonzero()[:, 0]
        at = s["slots"][on].long()
        x, r, i = (s[n][on].double() for n in ("x", "r", "i"))
        _, iota, _, a, beta = token(x, r, i)
        h = a * s["state"][at].double() + beta * iota * x
        y = torch.zeros_like(s["x"], dtype=torch.float64)
        y[on] = h
        new = s["new_state"].double()
        new[at] = h
        return y, new
    B, L, D = s["x"].shape
    lens = torch.full((B,), L, device="cuda") if s["seqlens"] is None else s["seqlens"]
    live = [(lens > t)[:, None] for t in range(L)] if s["seqlens"] is not None else None
    h0 = torch.zeros(B, D, dtype=torch.float64, device="cuda") if s["init"] is None else s["init"].double()
    out = {}
    h, entering = h0, []
    if op != "train":
        y = torch.zeros(B, L, D, dtype=torch.float64, device="cuda")
        for t in range(L):
            if t % CHUNK == 0:
                entering.append(h)
            x, r, i = (s[n][:, t].double() for n in ("x", "r", "i"))
            _, iota, _, a, beta = token(x, r, i)
            new = a * h + beta * iota * x
            h = new if live is None else torch.where(live[t], new, h)
            y[:, t] = h if live is None else h * live[t]
        out.update(y=y, final=h)
        if op == "prefill":
            return out
    on = None if s["seqlens"] is None else torch.arange(L, device="cuda")[None, :, None] < lens[:, None, None]
    x, r, i = (_exact_round(s[n], on) if op == "train8" else s[n].double() for n in ("x", "r", "i"))
    before = torch.empty(B, L, D, dtype=torch.float64, device="cuda")
    h = h0
    for t in range(L):
        if entering and t % CHUNK == 0:
            h = entering[t // CHUNK]
        before[:, t] = h
        _, iota, _, a, beta = token(x[:, t], r[:, t], i[:, t])
        new = a * h + beta * iota * x[:, t]
        h = new if live is None else torch.where(live[t], new, h)
    m = torch.zeros_like(h0) if s["dfinal"] is None else s["dfinal"].double()
    d = {n: torch.zeros(B, L, D, dtype=torch.float64, device="cuda") for n in ("dx", "dr", "di")}
    dlam = torch.zeros(D, dtype=torch.float64, device="cuda")
    for t in reversed(range(L)):
        rho, iota, w, a, beta = token(x[:, t], r[:, t], i[:, t])
        dh = s["dy"][:, t].double() + m
        u = iota * x[:, t]
        dw = dh * (a * a / beta * u - a * before[:, t])
        g = dict(dx=dh * beta * iota, dr=dw * w * (1 - rho), di=dh * beta * u * (1 - iota))
        if live is None:
            m = a * dh
        else:
            m, dw = torch.where(live[t], a * dh, m), dw * live[t]
            g = {n: v * live[t] for n, v in g.items()}
        for n in g:
            d[n][:, t] = g[n]
        dlam += (dw * rho).sum(0)
    out.update(d)
    out["dlam"] = C * torch.sigmoid(s["lam"].double()) * dlam
    out["dinit"] = None if s["init"] is None else m
    return out
