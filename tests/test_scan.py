"""gdn_scan_fwd / gdn_scan_bwd / gdn_scan_update: the oracle against differences and the refusals (CPU), the kernels against the oracle
(GPU). The oracle derives the error that fp32 arithmetic may add to every value (oracle/scan.py); a bf16 output adds half a step,
2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_42_amd import binding as gb
from oracle import scan as SC

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
P = 1 << 12   # any aligned non-NULL pointer: the checks run before any launch


# ------------------------------------------------------------------------------------------ CPU
@pytest.mark.parametrize("blend", [False, True])
def test_oracle_gradients_match_differences(blend):
    rng = np.random.default_rng(2)
    D, cu = 3, [0, 4, 4, 5, 9]
    ins = dict(x=rng.standard_normal((1, 9, D)), g=-rng.random((1, 9, D)) * 2, h0=rng.standard_normal((4, D)))
    dh, dT = rng.standard_normal((1, 9, D)), rng.standard_normal((4, D))

    def f(x, g, h0):
        h, last, *_ = SC.forward(x, g, h0, cu, blend)
        return float((h * dh).sum() + (last * dT).sum())

    grads = dict(zip(("x", "g", "h0"), SC.backward(ins["x"], ins["g"], ins["h0"], dh, dT, cu, blend)))
    e0 = 1e-5   # central differences: error of order e0^2 times third derivatives of order 1
    for n, a in ins.items():
        for i in range(a.size):
            e = np.zeros(a.size)
            e[i] = e0
            e = e.reshape(a.shape)
            d = (f(**{**ins, n: a + e}) - f(**{**ins, n: a - e})) / (2 * e0)
            assert abs(d - grads[n].reshape(-1)[i]) < 1e-7, n


def test_oracle_closed_form():
    """Constant decay: h_t = a^t h0 + x (1 - a^t) / (1 - a); blended: a^t h0 + (1 - a^t) x."""
    a, t = 0.9, np.arange(1, 8)
    g = np.full((1, 7, 1), np.log(a))
    x, h0 = np.full((1, 7, 1), 2.0), np.full((1, 1), 3.0)
    assert np.allclose(SC.forward(x, g, h0, None, False)[0][0, :, 0], a ** t * 3 + 2 * (1 - a ** t) / (1 - a))
    assert np.allclose(SC.forward(x, g, h0, None, True)[0][0, :, 0], a ** t * 3 + (1 - a ** t) * 2)


def c_fwd(**kw):
    a = dict(x=P, g=P, h0=None, cu=None, h=P, hT=None, car=None, B=2, T=8, N=2, D=64, xs=64, blend=0, dtype=1, hd=1, ws=None, wb=0)
    a.update(kw)
    return gb.lib().gdn_scan_fwd(*a.values(), None)


def c_bwd(**kw):
    a = dict(x=P, g=P, car=P, dh=P, dhT=None, cu=None, dx=P, dg=P, dh0=None, B=2, T=8, N=2, D=64, xs=64, blend=0, dtype=1, hd=1, ws=None,
             wb=0)
    a.update(kw)
    return gb.lib().gdn_scan_bwd(*a.values(), None)


def c_update(**kw):
    a = dict(x=P, g=P, st=P, slots=P, cu=P, out=None, h=P, T=8, N=2, D=64, ns=4, xs=64, blend=0, dtype=1, hd=1)
    a.update(kw)
    return gb.lib().gdn_scan_update(*a.values(), None)


KIND = [(dict(dtype=2), -3), (dict(hd=2), -3), (dict(dtype=0, hd=1), -3), (dict(D=60), -5), (dict(D=0), -5), (dict(D=(1 << 20) + 8), -5),
        (dict(xs=-64), -2), (dict(xs=65), -4), (dict(x=P + 8), -4), (dict(g=P + 4), -4), (dict(x=None), -1), (dict(g=None), -1), (dict(T=-1), -2)]
SEQ = KIND + [(dict(B=0, N=0), -2), (dict(N=3), -2), (dict(cu=P), -2), (dict(B=1, N=0, cu=P), -2), (dict(T=1 << 28), -2),
              (dict(B=1, N=1, T=1 << 28, D=512), -2), (dict(B=1, N=(1 << 24) + 1, cu=P), -2), (dict(B=1 << 23, N=1 << 23, T=1), -2),
              (dict(B=1, N=2, cu=P + 2), -4), (dict(T=600), -6), (dict(T=600, ws=P, wb=1000), -6), (dict(T=600, ws=P + 16, wb=1 << 30), -4)]


@pytest.mark.parametrize("kw,status", SEQ + [(dict(h=None), -1), (dict(h=P + 8), -4), (dict(hT=P + 8), -4), (dict(h0=P + 2), -4), (dict(car=P + 2), -4)])
def test_fwd_refuses(kw, status):
    assert c_fwd(**kw) == status


@pytest.mark.parametrize("kw,status", SEQ + [
    (dict(car=None), -1), (dict(dh=None), -1), (dict(dx=None), -1), (dict(dg=None), -1), (dict(dh=P + 8), -4), (dict(dx=P + 8), -4),
    (dict(dg=P + 8), -4), (dict(dh0=P + 8), -4), (dict(dhT=P + 2), -4), (dict(car=P + 1), -4)])
def test_bwd_refuses(kw, status):
    assert c_bwd(**kw) == status


@pytest.mark.parametrize("kw,status", KIND + [
    (dict(cu=None), -2), (dict(N=-1), -2), (dict(ns=-1), -2), (dict(N=1 << 22), -2), (dict(slots=None), -1), (dict(st=None), -1), (dict(h=None), -1),
    (dict(st=P + 4), -4), (dict(slots=P + 2), -4), (dict(out=P + 2), -4), (dict(cu=P + 1), -4), (dict(h=P + 8), -4)])
def test_update_refuses(kw, status):
    assert c_update(**kw) == status


def test_sizes():
    rows, ws = gb.gdn_scan_carry_rows, gb.gdn_scan_workspace_bytes
    assert rows(2, 0, 2, False) == rows(2, 1, 2, False) == rows(2, 256, 2, False) == 2 and rows(2, 257, 2, False) == 4
    assert rows(1, 100, 7, True) == 7 and rows(1, 1000, 7, True) == 7 + 3 and rows(1, 100, 7, False) == 0
    # fewer than 128 tokens a sequence: tiles of 32, where the call is large enough
    assert rows(1, 1024, 8, True) == 8 + 4 and rows(1, 1025, 9, True) == 9 + 32 and rows(1, 1023, 8, True) == 8 + 31 and rows(1, 1023, 7, True) == 7 + 3 and rows(1, 256, 8, True) == 8 + 1 and rows(1, 32, 2, True) == 2 + 1
    assert rows(64, 64, 64, False) == 128 and rows(63, 64, 63, False) == 63 and rows(64, 128, 64, False) == 64
    assert ws(2, 256, 2, 64, False) == ws(1, 256, 9, 64, True) == 0
    assert ws(2, 512, 2, 72, False) == ws(1, 1024, 2, 72, True) == ws(1, 512, 1, 72, True) == ws(64, 100, 64, 72, False) == 0   # walked
    assert ws(2, 513, 2, 72, False) == 256 + 6 * 128 * 12   # counters, then maps and states of 6 x 2 tiles of 64 channels
    assert ws(17, 512, 17, 2048, False) == 2048 + 34 * 2048 * 12 and ws(16, 512, 16, 2048, False) == 0
    assert ws(1, 1000, 100, 328, True) == 512 + 512 + 131 * 384 * 12 and ws(1, 1000, 85, 328, True) == 0
    assert ws(1, 1000, 2, 60, True) == 0 and c_update(T=0, x=None, h=None) == 0 and c_update(T=0, N=0, cu=None, slots=None) == 0


def test_binding_refuses_on_the_host():
    m = lambda *s, dt=torch.float32: torch.empty(*s, device="meta", dtype=dt)  # noqa: E731
    i32 = torch.int32
    x, g = m(2, 300, 64), m(2, 300, 64)
    for args, text in (((m(8, 64), g), r"\[B, T, D\]"), ((x, m(2, 300, 32)), "g has shape"), ((x, m(2, 300, 64, dt=torch.bfloat16)), "g has dtype"),
                       ((x, g, m(1, 64)), "h0 has shape"), ((x, g, None, m(3)), "cu_seqlens must"), ((x, g), "on a GPU")):
        with pytest.raises(ValueError, match=text):
            gb.gdn_scan_fwd(*args)
    for args, text in (((x, g, m(2, 3, 64), m(4, 64)), "dh has shape"), ((x, g, x, m(2, 64)), "carries has shape"),
                       ((x, g, m(2, 300, 64, dt=torch.bfloat16), m(4, 64)), "dh has dtype"), ((x, g, x, m(4, 64)), "on a GPU")):
        with pytest.raises(ValueError, match=text):
            gb.gdn_scan_bwd(*args)
    with pytest.raises(ValueError, match="exceeds"):
        gb.gdn_scan_fwd(m(1, (1 << 32) + 8, 64), m(1, (1 << 32) + 8, 64))
    with pytest.raises(ValueError, match="exceeds"):
        gb.gdn_scan_update(m(8, 64), m(8, 64), m((1 << 32) + 5, 64), m(8, dt=i32))
    good = dict(x=m(8, 64), g=m(8, 64), states=m(5, 64), slots=m(8, dt=i32))
    for change, text in ((dict(x=m(1, 8, 64)), r"\[T, D\]"), (dict(states=m(5, 32)), "states has shape"), (dict(states=m(5, 1, 64)), "states must"),
                         (dict(g=m(8, 32)), "g has shape"), (dict(slots=m(3, dt=i32)), "without cu_seqlens"), (dict(), "on a GPU")):
        with pytest.raises(ValueError, match=text):
            gb.gdn_scan_update(**{**good, **change})


# ------------------------------------------------------------------------------------------ GPU
def make(seed, B, T, N, D, dtype, rate=1.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    speed = torch.exp(torch.empty(D).uniform_(-7.0, 1.0, generator=gen)) * rate
    return dict(x=r(B, T, D).to(DT[dtype]), g=-speed * torch.nn.functional.softplus(r(B, T, D)), h0=r(N, D), dh=r(B, T, D).to(DT[dtype]), dhT=r(N, D))


def inside(got, ref, tol, name):
    """got within tol of ref (and half a step of its type), in the rows that ref has."""
    full = got.cpu().double().numpy()
    assert full.shape == ref.shape, name
    cover = ~np.isnan(ref)
    step = 2.0 ** -8 * (1 + 2.0 ** -8) if got.dtype == torch.bfloat16 else U
    d, t = np.abs(full - ref)[cover], (tol + step * np.abs(ref))[cover]
    print(f"      {name}: largest error over its tolerance {float((d / np.maximum(t, 1e-300)).max() if d.size else 0):.3f}", flush=True)
    assert (d <= t).all(), name


def cut(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


def check_pass(x, cu, blend, full=True, od=None, dhd=None):
    t = {n: a.cuda() for n, a in x.items()}
    B, T, D = x["x"].shape
    h0, dhT = (x["h0"], x["dhT"]) if full else (None, None)
    th0, tdhT = (t["h0"], t["dhT"]) if full else (None, None)
    h = torch.full((B, T, D), 7.0, device="cuda", dtype=od or x["x"].dtype)
    _, hT, car = gb.gdn_scan_fwd(t["x"], t["g"], th0, cut(cu), blend=blend, h=h, keep_carries=True)
    rh, rT, eh, eT = SC.forward(x["x"], x["g"], h0, cu, blend)
    inside(h, rh, eh, "h")
    inside(hT, rT, eT, "hT")
    dh = x["dh"].to(dhd or x["x"].dtype)
    dx, dg, dh0 = gb.gdn_scan_bwd(t["x"], t["g"], dh.cuda(), car, tdhT, cut(cu), blend=blend)
    rx, rg, r0, ex, eg, e0 = SC.backward(x["x"], x["g"], h0, dh, dhT, cu, blend)
    inside(dx, rx, ex, "dx")
    inside(dg, rg, eg, "dg")
    inside(dh0, r0, e0, "dh0")
    return h, hT, car, dx, dg, dh0


SHAPES = [
    # B, T, cu, D
    (1, 1, None, 8), (2, 7, None, 72), (3, 256, None, 64), (2, 0, None, 64), (2, 257, None, 136), (1, 3000, None, 40), (5, 600, None, 64),
    (1, 90, [0, 1, 1, 3, 20, 36, 37, 52, 90], 72), (1, 256, [0, 0, 0, 256], 64), (1, 1100, [0, 0, 256, 513, 513, 514, 1026, 1090, 1090], 72),
    (1, 5000, [0, 4700, 4701, 5000], 24), (4, 32, None, 72), (4, 33, None, 72), (3, 20, None, 136), (65, 70, None, 24),
    # two tiles walked by one work-group, and up to four of 32 tokens
    (3, 512, None, 72), (1, 510, [0, 7, 510], 72), (1, 500, [0, 0, 490], 40), (1, 420, [0, 130, 390], 24), (1, 400, [0, 400], 136), (48, 127, None, 40),
    (1, 900, [0, 700, 900], 40), (1, 1024, [0, 0, 3, 1000], 72), (1, 600, [*range(0, 600, 60), 600], 3336), (1, 1000, [0, 30, 31, 500, 510, 520, 530, 540, 980], 72),
    # tiles of 32 tokens, one long sequence among short ones
    (1, 1050, [0, 0, 31, 63, 96, 97, 97, 300, 332, 333, 365, 370, 380, 390, 400, 1040], 72),
    (1, 900, [0, 0, 31, 63, 96, 97, 97, 300, 332, 333, 365, 370, 380, 390, 400, 890], 72),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,cu,D", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("blend", [False, True])
def test_against_oracle(B, T, cu, D, dtype, blend):
    print(f"[gpu] scan B={B} T={T} cu={cu} D={D} {dtype} blend={blend}", flush=True)
    N = B if cu is None else len(cu) - 1
    x = make(T + D, B, T, N, D, dtype)
    outs = check_pass(x, cu, blend)
    if cu is not None and cu[-1] < T:   # rows that no sequence covers
        assert (outs[0][:, cu[-1]:] == 7).all()
    check_pass(x, cu, blend, full=False, od=torch.float32, dhd=torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("blend", [False, True])
@pytest.mark.parametrize("rate", [0.0, 1e-4, 30.0])
def test_decays_from_none_to_strong(blend, rate):
    """No decay at all (a running sum; blended: the state stays), hardly any, and one that forgets within a token."""
    print(f"[gpu] scan rate={rate} blend={blend}", flush=True)
    check_pass(make(11, 1, 900, 1, 16, "f32", rate), None, blend)


@pytest.mark.gpu
def test_many_tiles_at_once():
    """More tiles than the device holds at once: 48 channel blocks of 2 x 33 tiles; sampled channels against the oracle."""
    B, T, D = 2, 8200, 3064
    print(f"[gpu] scan B={B} T={T} D={D}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    t = dict(x=r(B, T, D).bfloat16(), g=-0.3 * r(B, T, D).square() * torch.rand(D, generator=gen, device="cuda").square(), h0=r(B, D),
             dh=r(B, T, D).bfloat16(), dhT=r(B, D))
    h, hT, car = gb.gdn_scan_fwd(t["x"], t["g"], t["h0"], keep_carries=True)
    dx, dg, dh0 = gb.gdn_scan_bwd(t["x"], t["g"], t["dh"], car, t["dhT"])
    for _ in range(3):   # the same bits, whatever order the tiles ran in
        again = gb.gdn_scan_fwd(t["x"], t["g"], t["h0"], keep_carries=True)
        back = gb.gdn_scan_bwd(t["x"], t["g"], t["dh"], car, t["dhT"])
        assert all(torch.equal(a, b) for a, b in zip((*again, *back), (h, hT, car, dx, dg, dh0)))
    at = [0, 63, 64, 1000, 3063]
    s = {n: a[..., at].cpu() for n, a in t.items()}
    rh, rT, eh, eT = SC.forward(s["x"], s["g"], s["h0"], None, False)
    inside(h[..., at], rh, eh, "h")
    inside(hT[..., at], rT, eT, "hT")
    rx, rg, r0, ex, eg, e0 = SC.backward(s["x"], s["g"], s["h0"], s["dh"], s["dhT"], None, False)
    inside(dx[..., at], rx, ex, "dx")
    inside(dg[..., at], rg, eg, "dg")
    inside(dh0[..., at], r0, e0, "dh0")


@pytest.mark.gpu
@pytest.mark.parametrize("blend", [False, True])
def test_many_short_sequences(blend):
    """Tiles of 32 tokens, more than the device holds at once, some sequences of many tiles; sampled channels against the oracle."""
    gen = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 40, (400,), generator=gen).tolist() + [1500] + torch.randint(0, 40, (300,), generator=gen).tolist() + [64, 65, 63, 700]
    cu, D = np.concatenate([[0], np.cumsum(lens)]).tolist(), 1032
    print(f"[gpu] scan {len(lens)} sequences, {cu[-1]} tokens, D={D} blend={blend}", flush=True)
    x = make(9, 1, cu[-1] + 3, len(lens), D, "bf16")
    t = {n: a.cuda() for n, a in x.items()}
    h, hT, car = gb.gdn_scan_fwd(t["x"], t["g"], t["h0"], cut(cu), blend=blend, keep_carries=True)
    dx, dg, dh0 = gb.gdn_scan_bwd(t["x"], t["g"], t["dh"], car, t["dhT"], cut(cu), blend=blend)
    at = [0, 63, 64, 1031]
    s = {n: a[..., at] for n, a in x.items()}
    rh, rT, eh, eT = SC.forward(s["x"], s["g"], s["h0"], cu, blend)
    inside(h[..., at], rh, eh, "h")
    inside(hT[..., at], rT, eT, "hT")
    rx, rg, r0, ex, eg, e0 = SC.backward(s["x"], s["g"], s["h0"], s["dh"], s["dhT"], cu, blend)
    inside(dx[..., at], rx, ex, "dx")
    inside(dg[..., at], rg, eg, "dg")
    inside(dh0[..., at], r0, e0, "dh0")


@pytest.mark.gpu
def test_thousands_of_sequences():
    """More sequences than one step of the tiles' layout takes, many of them empty, one of many tiles behind the first thousands."""
    gen = torch.Generator().manual_seed(8)
    lens = torch.randint(0, 4, (9001,), generator=gen).tolist()
    lens[8000] = 300
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    print(f"[gpu] scan {len(lens)} sequences, {cu[-1]} tokens", flush=True)
    check_pass(make(13, 1, cu[-1], len(lens), 8, "f32"), cu, True)


@pytest.mark.gpu
def test_carries_are_the_states_between_tiles():
    x = make(21, 1, 700, 1, 64, "f32")
    t = {n: a.cuda() for n, a in x.items()}
    h, hT, car = gb.gdn_scan_fwd(t["x"], t["g"], t["h0"], keep_carries=True)
    rh, _, eh, _ = SC.forward(x["x"], x["g"], x["h0"], None, False)
    assert car.shape == (3, 64) and torch.equal(car[0], t["h0"][0])
    inside(car[1:], rh[0, [255, 511]], eh[0, [255, 511]], "carries")
    # resumed: the sequence in two calls
    a, mid, _ = gb.gdn_scan_fwd(t["x"][:, :300], t["g"][:, :300].contiguous(), t["h0"])
    b, end, _ = gb.gdn_scan_fwd(t["x"][:, 300:], t["g"][:, 300:].contiguous(), mid)
    inside(torch.cat([a, b], 1), rh, 2 * eh, "two calls")
    assert torch.equal(end, b[:, -1])


@pytest.mark.gpu
def test_strided_tokens():
    x = make(5, 2, 300, 2, 264, "bf16")
    t = {n: a.cuda() for n, a in x.items()}
    fused = torch.randn(2, 300, 400, device="cuda").bfloat16()
    fused[..., 64:328] = t["x"]
    xv = fused[..., 64:328]
    a = gb.gdn_scan_fwd(t["x"], t["g"], t["h0"], keep_carries=True)
    b = gb.gdn_scan_fwd(xv, t["g"], t["h0"], keep_carries=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a = gb.gdn_scan_bwd(t["x"], t["g"], t["dh"], a[2], t["dhT"])
    b = gb.gdn_scan_bwd(xv, t["g"], t["dh"], b[2], t["dhT"])
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("blend", [False, True])
def test_nan_and_infinite_gates(blend):
    """A gate of -infinity forgets the state; NaN stays with its sequence and channel, in gates, inputs and gradients, across tiles."""
    D, cu = 64, [0, 600, 610, 1200]
    x = make(14, 1, 1200, 3, D, "f32")
    t = {n: a.cuda() for n, a in x.items()}
    t["g"][0, 100] = t["g"][0, 700] = float("-inf")
    run = lambda: (*gb.gdn_scan_fwd(t["x"], t["g"], t["h0"], cut(cu), blend=blend, keep_carries=True),)  # noqa: E731
    h, hT, car = run()
    dx, dg, dh0 = gb.gdn_scan_bwd(t["x"], t["g"], t["dh"], car, t["dhT"], cut(cu), blend=blend)
    assert torch.isfinite(h).all() and torch.isfinite(dg).all() and torch.isfinite(dx).all()
    assert torch.equal(h[0, 100], t["x"][0, 100]) and (dg[0, 100] == 0).all()
    rh, rT, eh, eT = SC.forward(x["x"], t["g"].cpu(), x["h0"], cu, blend)
    inside(h, rh, eh, "h")
    rx, rg, r0, ex, eg, e0 = SC.backward(x["x"], t["g"].cpu(), x["h0"], x["dh"], x["dhT"], cu, blend)
    inside(dx, rx, ex, "dx")
    inside(dg, rg, eg, "dg")
    for what in ("g", "x"):
        for n in ("g", "x", "dh"):
            t[n].copy_(x[n])
        t[what][0, 300, 5] = float("nan")       # the first sequence, channel 5
        t["dh"][0, 900, 9] = float("nan")       # the third one's gradient, channel 9
        t["x"][0, 605] = t["g"][0, 605] = float("nan")
        h, hT, car = run()
        dx, dg, dh0 = gb.gdn_scan_bwd(t["x"], t["g"], t["dh"], car, t["dhT"], cut(cu), blend=blend)
        bad = torch.zeros(1200, D, dtype=torch.bool)
        bad[300:600, 5] = True
        bad[605:610] = True
        rh = SC.forward(x["x"], x["g"], x["h0"], cu, blend)[0][0]
        assert torch.equal(torch.isnan(h[0]).cpu(), bad)
        ok = ~bad.numpy()
        assert np.abs(h[0].cpu().double().numpy() - rh)[ok].max() <= 1e-4 * np.abs(rh).max()
        assert torch.isnan(hT[0, 5]) and torch.isnan(hT[1]).all() and torch.isfinite(hT[2]).all() and torch.isfinite(hT[0, :5]).all()
        assert torch.isnan(dx[0, 610:901, 9]).all() and torch.isfinite(dx[0, 901:]).all() and torch.isfinite(dx[0, 610:, :9]).all()
        assert torch.isfinite(dx[0, 301:600]).all() and torch.isfinite(dg[0, 901:, 9]).all() and torch.isnan(dh0[2, 9])


@pytest.mark.gpu
@pytest.mark.parametrize("blend", [False, True])
def test_bad_offsets_stay_inside_and_end(blend, monkeypatch):
    """Offsets that fall or leave [0, T] are clamped, also where they count more tiles than there is room for."""
    x = make(6, 1, 1000, 5, 64, "bf16")
    t = {n: a.cuda() for n, a in x.items()}
    short = {n: a[:, :500].contiguous() if n in ("x", "g", "dh") else a for n, a in t.items()}   # walked
    for offsets in ([-5, 600, 3, 500], [0, 500, 0, 500], [500, 0, 0, 700]):
        h = torch.zeros_like(short["x"])
        _, hT, car = gb.gdn_scan_fwd(short["x"], short["g"], torch.ones(3, 64, device="cuda"), cut(offsets), blend=blend, h=h, keep_carries=True)
        car = torch.nan_to_num(car, 0.0, 0.0, 0.0)
        gb.gdn_scan_bwd(short["x"], short["g"], short["dh"], car, torch.ones(3, 64, device="cuda"), cut(offsets), blend=blend)
        torch.cuda.synchronize()
        assert torch.isfinite(h.float()).all()
    for T in (1000, 1500):   # walked; passed on between work-groups
        u = {n: a.cuda() for n, a in make(6, 1, T, 5, 64, "bf16").items()}
        for offsets in ([-5, 600, 3, 2000000000, 0, T], [0, T, 0, T, 0, T], [T, 0, 0, 0, 0, 0], [0, T] * 10):
            n = len(offsets) - 1   # 19 of them: tiles of 32
            h0 = torch.ones(n, 64, device="cuda")
            h = torch.zeros_like(u["x"])
            _, hT, car = gb.gdn_scan_fwd(u["x"], u["g"], h0, cut(offsets), blend=blend, h=h, keep_carries=True)
            car = torch.nan_to_num(car, 0.0, 0.0, 0.0)   # rows past the last tile hold anything
            gb.gdn_scan_bwd(u["x"], u["g"], u["dh"], car, h0, cut(offsets), blend=blend)
            torch.cuda.synchronize()
            assert torch.isfinite(h.float()).all()
    t["h0"] = x["h0"].cuda()
    slots = torch.arange(5, dtype=torch.int32, device="cuda")
    gb.gdn_scan_update(t["x"][0], t["g"][0], t["h0"].clone(), slots, cut([-5, 600, 3, 2000000000, 0, 1000]), blend=blend)
    monkeypatch.setenv("GDN_CHECK", "1")
    gb.gdn_scan_fwd(t["x"], t["g"], t["h0"], cut([0, 3, 3, 500, 600, 999]))
    bad = cut([0, 600, 3, 700, 800, 1000])
    for f in (lambda: gb.gdn_scan_fwd(t["x"], t["g"], t["h0"], bad), lambda: gb.gdn_scan_bwd(t["x"], t["g"], t["dh"], torch.zeros(8, 64, device="cuda"), None, bad),
              lambda: gb.gdn_scan_update(t["x"][0], t["g"][0], t["h0"], slots, bad)):
        with pytest.raises(gb.GDNError):
            f()


@pytest.mark.gpu
def test_graph_replay_streams_and_repeats():
    """Captured scans replayed between eager ones, their workspaces full of what earlier calls left; two streams at once."""
    cu = [0, 700, 703, 2100]
    x = make(12, 1, 2100, 3, 264, "bf16")
    t = {n: a.cuda() for n, a in x.items()}
    c = cut(cu)

    def both(stream=None):
        h, hT, car = gb.gdn_scan_fwd(t["x"], t["g"], t["h0"], c, blend=True, keep_carries=True, stream=stream)
        return h, hT, car[:12], *gb.gdn_scan_bwd(t["x"], t["g"], t["dh"], car, t["dhT"], c, blend=True, stream=stream)

    tiles = 3 + 1 + 6
    want = both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(5):
        for j in (0, 1, 3, 4, 5):
            out[j].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for j in (0, 1, 3, 4, 5):
            assert torch.equal(out[j], want[j]), (i, j)
        assert torch.equal(out[2][:tiles], want[2][:tiles])
        t["x"].mul_(1)
        again = both()
        assert all(torch.equal(again[j], want[j]) for j in (0, 1, 3, 4, 5))
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    got = [both(side[i % 2]) for i in range(6)]
    for s in side:
        s.synchronize()
    for g in got:
        assert all(torch.equal(g[j], want[j]) for j in (0, 1, 3, 4, 5))


RUNS = [
    # lens, D, dtype
    ([1], 8, "bf16"), ([1, 0, 3, 48, 0], 264, "bf16"), ([5] * 9, 136, "f32"), ([1] * 70, 520, "bf16"), ([2, 9, 0, 4], 2056, "f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,D,dtype", RUNS)
@pytest.mark.parametrize("mode", ["last", "every", "padded"])
@pytest.mark.parametrize("blend", [True, False])
def test_update_against_oracle(lens, D, dtype, mode, blend):
    print(f"[gpu] scan update lens={lens[:6]}x{len(lens)} D={D} {dtype} {mode} blend={blend}", flush=True)
    N, T = len(lens), sum(lens)
    ns = N + T + 3
    x = make(N * 31 + T, 1, T + 2, ns, D, dtype)   # two rows behind the last sequence
    order = torch.randperm(ns, generator=torch.Generator().manual_seed(T)).to(torch.int32)
    cu = torch.tensor([0, *lens]).cumsum(0).to(torch.int32)
    slots, out = order[:N].clone(), None
    if mode == "every":
        out = torch.cat([order[N:N + T], torch.tensor([-1, ns], dtype=torch.int32)])
        out[T // 2] = -1   # a state that is not kept
    if mode == "padded":
        slots[::2] = torch.tensor([-1, ns, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).repeat(N)[: len(slots[::2])]
    for od in (torch.float32, torch.bfloat16):
        if dtype == "f32" and od == torch.bfloat16:
            continue
        pool, h = x["h0"].cuda(), torch.full((T + 2, D), 7.0, dtype=od, device="cuda")
        gb.gdn_scan_update(x["x"][0].cuda(), x["g"][0].cuda(), pool, slots.cuda(), cu.cuda(), None if out is None else out.cuda(), h, blend=blend)
        rh, rp, eh, ep = SC.run(x["x"][0], x["g"][0], x["h0"], slots.numpy(), cu.numpy(), None if out is None else out.numpy(), blend)
        inside(h, rh, eh, "h")
        inside(pool, rp, ep, "pool")
        assert (h[T:] == 7).all()   # rows that no sequence covers
        untouched = np.setdiff1d(np.arange(ns), (slots if out is None else out).numpy())
        assert torch.equal(pool.cpu()[untouched], x["h0"][untouched])


@pytest.mark.gpu
def test_prompt_then_runs():
    """A prompt through gdn_scan_fwd, its state into the pool, then tokens one by one and in runs, drafts kept and one accepted."""
    D = 264
    x = make(31, 1, 400, 1, D, "f32")
    t = {n: a.cuda() for n, a in x.items()}
    rh, _, eh, _ = SC.forward(x["x"], x["g"], x["h0"], None, True)
    _, hT, _ = gb.gdn_scan_fwd(t["x"][:, :380], t["g"][:, :380].contiguous(), t["h0"], blend=True)
    pool = torch.randn(12, D, device="cuda")
    rest = pool.clone()
    pool[3] = hT[0]
    i32 = dict(dtype=torch.int32, device="cuda")
    xs, gs = t["x"][0], t["g"][0]
    step = lambda a, b, slot, out=None: gb.gdn_scan_update(xs[a:b], gs[a:b], pool, torch.tensor([slot], **i32), torch.tensor([0, b - a], **i32),  # noqa: E731
                                                           None if out is None else torch.tensor(out, **i32), blend=True)
    got = [step(380, 381, 3), step(381, 390, 3)]
    step(390, 394, 3, [5, 6, 7, 8])             # four draft tokens, of which two are accepted
    got += [rest[:0], step(392, 400, 6)]
    inside(torch.cat(got), np.concatenate([rh[0, 380:390], rh[0, 392:400]]), 2 * np.concatenate([eh[0, 380:390], eh[0, 392:400]]), "runs")
    inside(pool[[5, 7, 8]], rh[0, [390, 392, 393]], 2 * eh[0, [390, 392, 393]], "drafts")
    assert torch.equal(pool[[0, 1, 2, 4, 9, 10, 11]], rest[[0, 1, 2, 4, 9, 10, 11]])


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Tokens and slots whose elements start past 2^31."""
    x = make(8, 1, 500, 1, 64, "bf16")
    big = torch.zeros(1, 33000, 131072, device="cuda", dtype=torch.bfloat16)
    big[0, 32500:, 70000:70064] = x["x"][0].cuda()
    g = torch.zeros(1, 33000, 64, device="cuda")
    g[0, 32500:] = x["g"][0].cuda()
    h, hT, car = gb.gdn_scan_fwd(big[..., 70000:70064], g, keep_carries=True)
    rh, rT, eh, eT = SC.forward(x["x"], x["g"], None, None, False)
    inside(h[:, 32500:], rh, eh, "h")
    inside(hT, rT, eT, "hT")
    dh = torch.zeros(1, 33000, 64, device="cuda", dtype=torch.bfloat16)
    dh[0, 32500:] = x["dh"][0].cuda()
    dx, dg, _ = gb.gdn_scan_bwd(big[..., 70000:70064], g, dh, car)
    rx, rg, _, ex, eg, _ = SC.backward(x["x"], x["g"], None, x["dh"], None, None, False)
    inside(dx[:, 32500:], rx, ex, "dx")
    inside(dg[:, 32500:], rg, eg, "dg")
    del big
    pool = torch.zeros(300000, 8192, device="cuda")
    z = make(9, 1, 2, 1, 8192, "f32")
    pool[299999] = z["h0"][0].cuda()
    h = gb.gdn_scan_update(z["x"][0].cuda(), z["g"][0].cuda(), pool, torch.tensor([299999], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    rh, rT, eh, eT = SC.forward(z["x"], z["g"], z["h0"], None, False)
    inside(h[None], rh, eh, "h")
    inside(pool[299999][None], rT, eT, "state")
    assert not pool[:299999].any()
