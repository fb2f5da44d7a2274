"""The gated linear recurrence where it can go wrong: gates that are nearly open or shut, number by number; float32's last digits;
sequences of every length alone and padded, bit by bit; results in the place of inputs."""
import numpy as np
import pytest
import torch

from mamba_ssd_selective_gb300 import inputs
from oracle import linear
from tests.helpers import IO_TORCH, dev, host

pytestmark = pytest.mark.gpu


def on_device(d, io):
    return {n: dev(v, IO_TORCH[io] if n in ("x", "r", "i", "dy") else torch.float32) for n, v in d.items()}


def tokens(t):
    return [t[n] for n in ("x", "r", "i", "lam")]


# ------------------------------------------------------------- saturated gates

@pytest.mark.parametrize("size", [(2, 7, 64), (1, 16, 5), (2, 100, 72), (1, 130, 33), (2, 90, 6)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rate", [1.0, 40.0])
@pytest.mark.parametrize("packed", [False, True])
def test_gradients_of_saturated_gates_number_by_number(ssd, size, io, rate, packed):
    """r and i from 8 to 30 (a quarter of them from -30 to -8), where 1 - sigmoid is 3e-4 to 1e-13: dr and di each within the error of
    its own terms. x, dy and the states are positive, so that only the two terms of dr can cancel.

    An exponential at |30| is off by 30e-7 of its argument and 2 units of 2^-23: 3.3e-6. di = dh b (1 - iota): dh 3.3e-6 by the decays and
    20 units of 2^-24; b 3.3e-6 by iota and half of it by the root of rho; 1 - iota twice: 16e-6. dr has w (3.3e-6), h (that of b and of
    dh) or the polynomial of the ratio (1.2e-6): 23e-6 of the sum of its terms. Results in bf16 are off by another 2^-8 at most."""
    d = inputs.linear_inputs(*size, io, seed=21, rate=rate)
    rng = np.random.default_rng(22)
    for n in ("r", "i"):
        d[n] = inputs.round_to(rng.uniform(8, 30, size) * np.where(rng.random(size) < 0.25, -1, 1), io)
    for n in ("x", "dy", "init", "dfinal"):
        d[n] = np.abs(d[n])
    t = on_device(d, io)
    kept = ssd.gated_linear_checkpoint(t["x"])
    ssd.gated_linear_chunked(*tokens(t), init_state=t["init"], **kept)
    if packed:
        for n in ("x", "r", "i"):
            d[n] = linear.unpack8(*linear.pack8(d[n]))
        got = ssd.gated_linear_chunked_bwd_packed(lam=t["lam"], dy=t["dy"], dfinal_state=t["dfinal"], **kept)
    else:
        got = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], states=kept["states"], dfinal_state=t["dfinal"])
    want = linear.linear_seq_bwd(*(d[n] for n in ("x", "r", "i", "lam", "dy")), 8.0, d["init"], d["dfinal"], states=host(kept["states"]))
    w, a, beta, iota = linear.gates(d["x"], d["r"], d["i"], d["lam"], 8.0)
    y, _, entering = linear.linear_seq(d["x"], d["r"], d["i"], d["lam"], 8.0, d["init"], states=host(kept["states"]))
    before = np.concatenate([entering[:, :1], y[:, :-1]], 1)
    before[:, ::64] = entering
    dh = want["dx"] / (beta * iota)
    terms = dict(di=np.abs(want["di"]), dr=dh * linear.sigmoid(-d["r"]) * (a * a * w / beta * iota * np.abs(d["x"]) + a * w * before))
    for n, whole in terms.items():
        off = np.abs(host(got[n]) - want[n])
        most = 2.5e-5 * whole + (2.0 ** -8 * np.abs(want[n]) if io == "bf16" else 0)
        assert (off <= most).all(), f"{n}: {np.max(off / np.maximum(whole, 1e-300)):.2e} of its terms"
    assert (host(got["di"]) >= 0).all()


# ------------------------------------------------------------ float32's digits

@pytest.mark.parametrize("size", [(2, 777, 97), (2, 777, 96), (3, 16, 130), (1, 2000, 34)])
@pytest.mark.parametrize("rate", [1.0, 40.0])
def test_float32_keeps_its_digits(ssd, size, rate):
    """In the 2-norm, 20 units of 2^-24 for y and the states (gates 4, w 6, what h makes of it 6, sums and joints 4) and twice that for
    gradients, which are products of two such sums; with t up to 1 the polynomials of a and of the root add 3.5e-7 and 6e-7, that of the
    gradients' ratio 1.2e-6 (dlam, a sum of both signs, is left to the other tests)."""
    d = inputs.linear_inputs(*size, "f32", seed=25, rate=rate)
    t = on_device(d, "f32")
    kept = ssd.gated_linear_checkpoint(t["x"], packed=False)
    y, final = ssd.gated_linear_chunked(*tokens(t), init_state=t["init"], **kept)
    g = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], states=kept["states"], dfinal_state=t["dfinal"])
    args = [d[n] for n in ("x", "r", "i", "lam")]
    want = dict(zip(("y", "final", "states"), linear.linear_seq(*args, 8.0, d["init"])))
    grads = linear.linear_seq_bwd(*args, d["dy"], 8.0, d["init"], d["dfinal"])
    one = 20 * 2.0 ** -24 + (9.5e-7 if rate > 1 else 0)
    for got, w, most in [(y, want["y"], one), (final, want["final"], one), (kept["states"], want["states"], one)] + [
            (g[n], grads[n], 2 * one + (1.2e-6 if rate > 1 else 0)) for n in ("dx", "dr", "di", "dinit")]:
        off = np.linalg.norm(host(got) - w) / np.linalg.norm(w)
        assert off <= most, f"{off:.2e} of {most:.2e}"


# ------------------------------------------------- alone and in a padded batch

@pytest.mark.parametrize("D", [72, 33, 6])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rate", [1.0, 40.0])
def test_a_sequence_cut_to_its_length_is_bitwise_the_padded_one(ssd, D, io, rate):
    """y, the states and the 8 bits do not depend on what a sequence is padded to, zeros' signs in its first state included."""
    lens = [0, 1, 5, 10, 15, 16, 17, 33, 63, 64, 65, 100, 128, 150]
    L = max(lens)
    d = inputs.linear_inputs(len(lens), L, D, io, seed=23, rate=rate)
    d["init"][:, ::5] = -0.0
    d["x"][:, ::3, ::5] = 0.0
    t = on_device(d, io)
    seqlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kept = ssd.gated_linear_checkpoint(t["x"])
    y, final = ssd.gated_linear_chunked(*tokens(t), init_state=t["init"], seqlens=seqlens, **kept)
    bits = lambda v: v.contiguous().view(torch.uint8)  # noqa: E731
    for b, n in enumerate(lens):
        one = [t[k][b:b + 1, :n].clone() for k in ("x", "r", "i")]
        k1 = ssd.gated_linear_checkpoint(one[0])
        y1, f1 = ssd.gated_linear_chunked(*one, t["lam"], init_state=t["init"][b:b + 1].clone(), **k1)
        assert torch.equal(bits(y1[0]), bits(y[b, :n])), f"y, {n} tokens"
        assert torch.equal(bits(f1[0]), bits(final[b])), f"final state, {n} tokens"
        assert torch.equal(bits(k1["states"][0]), bits(kept["states"][b, :-(-n // 64)])), f"states, {n} tokens"
        assert (bits(kept["states"][b, -(-n // 64):]) == bits(final[b][None].expand(-(-L // 64) - -(-n // 64), D))).all()
        assert torch.equal(k1["values"][:, 0], kept["values"][:, b, :n]) and torch.equal(k1["scales"][:, 0], kept["scales"][:, b, :-(-n // 16)])


# ------------------------------------------------- results in the place of inputs

@pytest.mark.parametrize("D", [64, 65])
def test_results_in_the_place_of_what_they_come_from(ssd, D):
    """The pairs that may be one buffer give the bits that two buffers give, the others are refused."""
    d = inputs.linear_inputs(4, 50, D, "f32", seed=24)
    t = on_device(d, "f32")
    kept = ssd.gated_linear_checkpoint(t["x"], packed=False)
    y, final = ssd.gated_linear_chunked(*tokens(t), init_state=t["init"], **kept)
    own = t["init"].clone()
    y2, _ = ssd.gated_linear_chunked(*tokens(t), init_state=own, final_state=own)
    assert torch.equal(y, y2) and torch.equal(own, final)
    own = t["init"].clone()  # the states of up to 64 tokens are the first one
    y2, final2 = ssd.gated_linear_chunked(*tokens(t), init_state=own, states=own.view(4, 1, D))
    assert torch.equal(y, y2) and torch.equal(final, final2) and torch.equal(own, t["init"])
    one = [t[n][:, 0].contiguous() for n in ("x", "r", "i")]
    pool = t["init"].clone()
    want = ssd.gated_linear_step(t["init"], *one, t["lam"], new_state=pool)
    for k in range(3):
        mine, state = [v.clone() for v in one], t["init"].clone()
        assert torch.equal(ssd.gated_linear_step(state, *mine, t["lam"], y=mine[k]), want) and torch.equal(state, pool)
        assert mine[k].equal(want)
    g = ssd.gated_linear_chunked_bwd(*tokens(t), t["dy"], states=kept["states"], dfinal_state=t["dfinal"])
    out = {n: torch.empty_like(v) for n, v in g.items() if n != "dinit"}
    own, ws = t["dfinal"].clone(), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    status = ssd.load().ssd_gated_linear_chunked_bwd(
        4, 50, D, 0, *(v.data_ptr() for v in tokens(t)), 8.0, None, kept["states"].data_ptr(), None, t["dy"].data_ptr(), own.data_ptr(),
        out["dx"].data_ptr(), out["dr"].data_ptr(), out["di"].data_ptr(), out["dlam"].data_ptr(), own.data_ptr(), ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream)
    assert status == ssd.SSD_OK and torch.equal(own, g["dinit"]) and all(torch.equal(out[n], g[n]) for n in out)
    wide = torch.empty(400 * D, device="cuda")
    x, y = wide[:200 * D].view(4, 50, D), wide[100 * D:300 * D].view(4, 50, D)
    for refused in (lambda: ssd.gated_linear_chunked(x, t["r"], t["i"], t["lam"], y=y), lambda: ssd.gated_linear_chunked(
            *tokens(t), init_state=t["init"], final_state=wide[:4 * D].view(4, D), states=wide[:4 * D].view(4, 1, D)),
            lambda: ssd.pack8(x, values=wide.view(torch.int8)[:200 * D].view(4, 50, D))):
        with pytest.raises(ssd.SsdError, match="shares memory"):
            refused()
