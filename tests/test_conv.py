"""gdn_conv_fwd / gdn_conv_bwd / gdn_conv_update: the oracle against differences and the refusals (CPU), the kernels against the oracle
(GPU).

Tolerances (u = 2^-24, half a step of fp32). z is a sum of W + 1 <= 5 terms: off by 5 u Z, Z the sum of their magnitudes. The sigmoid's
exponent z log2 e is rounded once, the exponential and the reciprocal are good to 2 u each, a sum and a product follow: s is off by
(|z| + 8) u of itself; y = z s has a slope of at most 1.1. So y is off by at most u (8 Z + |y| (|z| + 8)), and dz, whose factor
s (1 + z (1 - s)) is at most 1.1 with a slope of at most 1/2, by K u |dy|, K = 5 Z + (|z| + 8)(1 + |z|) (without activation 0). dx adds
W products and a sum: sum |w| (K + 8) u |dy|. Weight gradients are sums over tokens of at most 128 terms in a row here, then
trees: 192 u of the sum of magnitudes, and dz's own error. A bf16 output adds half a step, 2^-8 of the value. Windows are copies.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_42_amd import binding as gb
from oracle import conv as CV

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
P = 1 << 12   # any aligned non-NULL pointer: the checks run before any launch


# ------------------------------------------------------------------------------------------ CPU
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_oracle_gradients_match_differences(silu, W):
    rng = np.random.default_rng(W)
    D, cu = 2, [0, 4, 4, 5, 7]
    ins = dict(x=rng.standard_normal((1, 7, D)), w=rng.standard_normal((D, W)), b=rng.standard_normal(D), w0=rng.standard_normal((4, W - 1, D)))
    dy, dl = rng.standard_normal((1, 7, D)), rng.standard_normal((4, W - 1, D))

    def f(x, w, b, w0):
        y, last = CV.forward(x, w, b, w0, cu, silu)
        return float((y * dy).sum() + (last * dl).sum())

    grads = dict(zip(("x", "w", "b", "w0"), CV.backward(**{"x": ins["x"], "w": ins["w"], "b": ins["b"], "window0": ins["w0"], "dy": dy,
                                                          "dlast": dl, "cu": cu, "silu": silu})))
    h = 1e-5   # central differences: error of order h^2 times third derivatives of order 1
    for n, a in ins.items():
        for i in range(a.size):
            e = np.zeros(a.size)
            e[i] = h
            e = e.reshape(a.shape)
            d = (f(**{**ins, n: a + e}) - f(**{**ins, n: a - e})) / (2 * h)
            assert abs(d - grads[n].reshape(-1)[i]) < 1e-7, n


def test_oracle_run_is_the_sequence():
    rng = np.random.default_rng(1)
    x, w, pool = rng.standard_normal((6, 3)), rng.standard_normal((3, 4)), rng.standard_normal((2, 3, 3))
    y, after = CV.run(x, w, None, pool, [1], [0, 6], None, True)
    y2, last = CV.forward(x[None], w, None, pool[1:], None, True)
    assert np.array_equal(y, y2[0]) and np.array_equal(after[1], last[0]) and np.array_equal(after[0], pool[0])
    a, mid = CV.run(x[:2], w, None, pool, [1], [0, 2], None, True)
    b, end = CV.run(x[2:], w, None, mid, [1], [0, 4], None, True)
    assert np.allclose(np.concatenate([a, b]), y) and np.array_equal(end, after)


def c_fwd(**kw):
    a = dict(x=P, w=P, b=None, w0=None, cu=None, y=P, wT=None, B=2, T=8, N=2, D=64, W=4, xs=64, act=1, dtype=1)
    a.update(kw)
    return gb.lib().gdn_conv_fwd(*a.values(), None)


def c_bwd(**kw):
    a = dict(x=P, w=P, b=None, w0=None, dy=P, dwT=None, cu=None, dx=P, dw=None, db=None, dw0=None, B=2, T=8, N=2, D=64, W=4, xs=64,
             dxs=64, act=1, dtype=1, ws=None, wb=0)
    a.update(kw)
    return gb.lib().gdn_conv_bwd(*a.values(), None)


def c_update(**kw):
    a = dict(x=P, w=P, b=None, win=P, slots=P, cu=P, out=None, y=P, T=8, N=2, D=64, W=4, ns=4, xs=64, act=1, dtype=1)
    a.update(kw)
    return gb.lib().gdn_conv_update(*a.values(), None)


KIND = [(dict(dtype=2), -3), (dict(W=1), -5), (dict(W=5), -5), (dict(act=2), -5), (dict(D=60), -5), (dict(D=0), -5), (dict(D=(1 << 20) + 8), -5),
        (dict(xs=-64), -2), (dict(xs=65), -4), (dict(x=P + 8), -4), (dict(w=P + 4), -4), (dict(b=P + 2), -4), (dict(x=None), -1),
        (dict(w=None), -1), (dict(T=-1), -2)]
SEQ = KIND + [(dict(B=0, N=0), -2), (dict(N=3), -2), (dict(cu=P), -2), (dict(B=1, N=0, cu=P), -2), (dict(T=1 << 28), -2),
              (dict(B=1, N=1, T=1 << 28, D=512), -2), (dict(B=1, N=(1 << 24) + 1, cu=P), -2), (dict(B=1, N=1 << 24, cu=P, D=256), -2),
              (dict(B=1, N=2, cu=P + 2), -4), (dict(w0=P + 8), -4)]


@pytest.mark.parametrize("kw,status", SEQ + [(dict(y=None), -1), (dict(y=P + 8), -4), (dict(wT=P + 8), -4)])
def test_fwd_refuses(kw, status):
    assert c_fwd(**kw) == status


@pytest.mark.parametrize("kw,status", SEQ + [
    (dict(dy=None), -1), (dict(dx=None), -1), (dict(dxs=56), -2), (dict(dxs=-64), -2), (dict(dxs=65), -4), (dict(dwT=P + 4), -4),
    (dict(dw0=P + 4), -4), (dict(dw=P + 2), -4), (dict(dw=P), -6), (dict(db=P, ws=P, wb=8), -6), (dict(dw=P, ws=P + 16, wb=1 << 20), -4)])
def test_bwd_refuses(kw, status):
    assert c_bwd(**kw) == status


@pytest.mark.parametrize("kw,status", KIND + [
    (dict(cu=None), -2), (dict(N=-1), -2), (dict(ns=-1), -2), (dict(N=1 << 22), -2), (dict(slots=None), -1), (dict(win=None), -1), (dict(y=None), -1),
    (dict(win=P + 4), -4), (dict(slots=P + 2), -4), (dict(out=P + 2), -4), (dict(cu=P + 1), -4), (dict(y=P + 8), -4)])
def test_update_refuses(kw, status):
    assert c_update(**kw) == status


def test_outputs_over_inputs_are_refused():
    q, r, s = P + 4096, P + 8192, P + 12288
    for kw in (dict(), dict(y=q, w0=r, wT=r)):
        assert c_fwd(**kw) == -2
    for kw in (dict(dy=q), dict(dx=q, dy=q), dict(dy=q, dx=r, w0=s, dw0=s), dict(dy=q, dx=r, dwT=s, dw0=s)):
        assert c_bwd(**kw) == -2


def test_nothing_to_do_is_ok():
    assert c_fwd(T=0, x=None, y=None) == 0
    assert c_update(T=0, x=None, y=None, win=None) == 0
    assert c_update(T=0, N=0, cu=None, x=None, y=None) == 0
    w = gb.gdn_conv_bwd_workspace_bytes
    assert w(2, 0, 64, 4) == 0 and w(2, 8, 60, 4) == 0 and w(2, 8, 64, 5) == 0 and w(2, 8, 64, 4) == 64 * 5 * 4


def test_binding_refuses_on_the_host():
    m = lambda *s, dt=torch.float32: torch.empty(*s, device="meta", dtype=dt)  # noqa: E731
    i32 = torch.int32
    x, w = m(2, 8, 64), m(64, 4)
    for args, kw, text in (((m(8, 64), w), {}, r"\[B, T, D\]"), ((x, m(32, 4)), {}, "weight has shape"), ((x, m(64)), {}, "weight must"),
                           ((x, w), dict(activation="relu"), "activation"), ((x, w, m(8)), {}, "bias has shape"),
                           ((x, w, None, m(2, 2, 64)), {}, "window0 has shape"), ((x, w, None, m(2, 3, 64, dt=torch.bfloat16)), {}, "window0 has dtype"),
                           ((x, w, None, None, m(3)), {}, "cu_seqlens must"), ((x, w), {}, "on a GPU")):
        with pytest.raises(ValueError, match=text):
            gb.gdn_conv_fwd(*args, **kw)
    with pytest.raises(ValueError, match="dy has dtype"):
        gb.gdn_conv_bwd(x, w, m(2, 8, 64, dt=torch.bfloat16))
    with pytest.raises(ValueError, match="exceeds"):
        gb.gdn_conv_fwd(m(1, (1 << 32) + 8, 64), w)
    with pytest.raises(ValueError, match="exceeds"):
        gb.gdn_conv_update(m(8, 64), w, None, m((1 << 32) + 5, 3, 64), m(8, dt=i32))
    good = dict(x=m(8, 64), weight=w, bias=None, windows=m(5, 3, 64), slots=m(8, dt=i32))
    for change, text in ((dict(x=m(1, 8, 64)), r"\[T, D\]"), (dict(windows=m(5, 2, 64)), "windows has shape"), (dict(windows=m(5, 64)), "windows must"),
                         (dict(slots=m(3, dt=i32)), "without cu_seqlens"), (dict(slots=m(8)), "slots must"),
                         (dict(out_slots=m(3, dt=i32)), "out_slots has"), (dict(), "on a GPU")):
        with pytest.raises(ValueError, match=text):
            gb.gdn_conv_update(**{**good, **change})


# ------------------------------------------------------------------------------------------ GPU
def make(seed, B, T, N, D, W, dtype):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    dt = DT[dtype]
    return dict(x=r(B, T, D).to(dt), w=r(D, W), b=r(D), w0=r(N, W - 1, D).to(dt), dy=r(B, T, D).to(dt), dwT=r(N, W - 1, D).to(dt))


def half(t):
    return 2.0 ** -8 * (1 + 2.0 ** -8) if t.dtype == torch.bfloat16 else U


def inside(got, ref, tol, name):
    """got within tol of ref, in the rows that ref has."""
    full = got.cpu().double().numpy()
    assert full.shape == ref.shape, name
    cover = ~np.isnan(ref)
    d, t = np.abs(full - ref)[cover], np.broadcast_to(tol, ref.shape)[cover]
    print(f"      {name}: largest error over its tolerance {float((d / np.maximum(t, 1e-300)).max() if d.size else 0):.3f}", flush=True)
    assert (d <= t).all(), name


def magnitudes(x, w, b, w0, cu):
    """Z of every token (see above), NaN where no sequence covers it."""
    absent = None if w0 is None else w0.abs()
    return CV.forward(x.abs(), w.abs(), None if b is None else b.abs(), absent, cu, False)[0]


def check_fwd(x, w, b, w0, cu, silu, y, wT):
    ref, last = CV.forward(x, w, b, w0, cu, silu)
    Z = magnitudes(x, w, b, w0, cu)
    z = np.abs(CV.forward(x, w, b, w0, cu, False)[0])
    inside(y, ref, U * (8 * Z + np.abs(ref) * (z + 8 if silu else 1)) + half(y) * np.abs(ref), "y")
    if wT is not None:
        assert np.array_equal(wT.cpu().double().numpy(), last), "windowT"


def check_bwd(x, w, b, w0, dy, dwT, cu, silu, dx, dw, db, dw0):
    rdx, rdw, rdb, rw0 = CV.backward(x, w, b, w0, dy, dwT, cu, silu)
    Z = np.nan_to_num(magnitudes(x, w, b, w0, cu))
    z = np.abs(np.nan_to_num(CV.forward(x, w, b, w0, cu, False)[0]))
    K = (5 * Z + (z + 8) * (1 + z)) if silu else np.zeros_like(Z)
    adz = np.abs(dy.double().numpy())
    kdz = torch.tensor((K + 8) * U * adz)
    # the same adjoint with |w| carries the bound of dz to dx, dw, db and the window
    ex, ew, eb, e0 = CV.backward(x.double().abs(), w.abs(), None, None if w0 is None else w0.double().abs(), kdz, None, cu, False)
    sx, sw, sb, _ = CV.backward(x.double().abs(), w.abs(), None, None if w0 is None else w0.double().abs(), torch.tensor(1.1 * adz), None, cu, False)
    more = np.zeros_like(rdx)
    inside(dx, rdx, ex + 4 * U * np.abs(rdx) + half(dx) * np.abs(rdx) + more, "dx")
    if dw is not None:
        inside(dw, rdw, ew + 192 * U * sw, "dw")
    if db is not None:
        inside(db, rdb, eb + 192 * U * sb, "db")
    if dw0 is not None:
        inside(dw0, rw0, e0 + 4 * U * np.abs(rw0) + half(dw0) * np.abs(rw0), "dwindow0")


SHAPES = [
    # B, T, cu, D
    (1, 1, None, 8), (2, 3, None, 264), (3, 40, None, 136), (1, 130, None, 520), (2, 0, None, 64),
    (1, 90, [0, 1, 1, 3, 20, 36, 37, 52, 90], 264), (1, 40, [0, 0, 0, 16, 32, 33, 38], 64), (1, 9, [0, 2, 4, 6, 6], 1032),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,cu,D", SHAPES)
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("silu", [True, False])
def test_against_oracle(B, T, cu, D, W, dtype, silu):
    print(f"[gpu] conv B={B} T={T} cu={cu} D={D} W={W} {dtype} silu={silu}", flush=True)
    N = B if cu is None else len(cu) - 1
    x = make(T + D + W, B, T, N, D, W, dtype)
    t = {n: a.cuda() for n, a in x.items()}
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    act = "silu" if silu else None
    for full in (True, False):
        b, w0, dwT = (x["b"], x["w0"], x["dwT"]) if full else (None, None, None)
        tb, tw0, tdwT = (t["b"], t["w0"], t["dwT"]) if full else (None, None, None)
        y = torch.full((B, T, D), 7.0, device="cuda", dtype=DT[dtype])
        _, wT = gb.gdn_conv_fwd(t["x"], t["w"], tb, tw0, cut, activation=act, y=y)
        check_fwd(x["x"], x["w"], b, w0, cu, silu, y, wT)
        dx = torch.full((B, T, D), 7.0, device="cuda", dtype=DT[dtype])
        _, dw, db, dw0 = gb.gdn_conv_bwd(t["x"], t["w"], t["dy"], tb, tw0, tdwT, cut, activation=act, dx=dx)
        assert (db is None) == (b is None)
        check_bwd(x["x"], x["w"], b, w0, x["dy"], dwT, cu, silu, dx, dw, db, dw0)
        if cu is not None and cu[-1] < T:   # rows that no sequence covers
            assert (y[:, cu[-1]:] == 7).all() and (dx[:, cu[-1]:] == 7).all()
    only, a, c, d = gb.gdn_conv_bwd(t["x"], t["w"], t["dy"], t["b"], t["w0"], t["dwT"], cut, activation=act, need_dw=False, need_dwindow0=False)
    assert a is None and c is None and d is None
    check_bwd(x["x"], x["w"], x["b"], x["w0"], x["dy"], x["dwT"], cu, silu, only, None, None, None)
    assert gb.gdn_conv_fwd(t["x"], t["w"], cu_seqlens=cut, output_final_window=False)[1] is None


@pytest.mark.gpu
@pytest.mark.parametrize("D,W", [(520, 4), (8200, 4), (8200, 2), (8200, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tiles(D, W, dtype):
    """More tiles than waves, or runs of so many tokens that what is known of them is looked up anew within a run; long sequences beside
    stretches of short ones, which begin and end at every place of a block."""
    gen = torch.Generator().manual_seed(D + W)
    lens = [700, 3, 0, 2197] + torch.randint(0, 40, (60,), generator=gen).tolist() + [101] + torch.randint(60, 70, (20,), generator=gen).tolist() + [1, 2500]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    T, N = cu[-1] + 2, len(lens)   # two rows behind the last sequence
    print(f"[gpu] conv packed {N} sequences, {T} tokens, D={D} W={W} {dtype}", flush=True)
    x = make(77, 1, T, N, D, W, dtype)
    t = {n: a.cuda() for n, a in x.items()}
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, wT = gb.gdn_conv_fwd(t["x"], t["w"], t["b"], t["w0"], cut, activation="silu")
    dx = torch.full_like(t["x"], 7.0)
    g = gb.gdn_conv_bwd(t["x"], t["w"], t["dy"], t["b"], t["w0"], t["dwT"], cut, activation="silu", dx=dx)
    assert (dx[:, cu[-1]:] == 7).all()
    only = gb.gdn_conv_bwd(t["x"], t["w"], t["dy"], t["b"], t["w0"], t["dwT"], cut, activation="silu", need_dw=False, dx=torch.full_like(dx, 7.0))
    assert torch.equal(only[0], dx) and torch.equal(only[3], g[3])
    for keep in (slice(0, 4), slice(256, 260), slice(D - 4, D)):   # channels are independent of each other
        s = {n: (a[keep] if n in ("w", "b") else a[..., keep]) for n, a in x.items()}
        check_fwd(s["x"], s["w"], s["b"], s["w0"], cu, True, y[..., keep], wT[..., keep])
        check_bwd(s["x"], s["w"], s["b"], s["w0"], s["dy"], s["dwT"], cu, True, g[0][..., keep], g[1][keep], g[2][keep], g[3][..., keep])


@pytest.mark.gpu
def test_strided_tokens():
    """x as a part of a fused projection, dx into a part of its gradient."""
    x = make(5, 2, 50, 2, 264, 4, "bf16")
    t = {n: a.cuda() for n, a in x.items()}
    y0, w0 = gb.gdn_conv_fwd(t["x"], t["w"], t["b"], t["w0"], activation="silu")
    g0 = gb.gdn_conv_bwd(t["x"], t["w"], t["dy"], t["b"], t["w0"], activation="silu")
    fused, dfused = torch.randn(2, 50, 400, device="cuda").bfloat16(), torch.full((2, 50, 400), 7.0, device="cuda").bfloat16()
    fused[..., 64:328] = t["x"]
    y, wT = gb.gdn_conv_fwd(fused[..., 64:328], t["w"], t["b"], t["w0"], activation="silu")
    g = gb.gdn_conv_bwd(fused[..., 64:328], t["w"], t["dy"], t["b"], t["w0"], activation="silu", dx=dfused[..., 64:328])
    assert torch.equal(y, y0) and torch.equal(wT, w0) and all(torch.equal(a, b) for a, b in zip(g, g0))
    assert (dfused[..., :64] == 7).all() and (dfused[..., 328:] == 7).all()
    with pytest.raises(ValueError, match="one token dimension"):
        gb.gdn_conv_fwd(torch.zeros(2, 60, 264, device="cuda", dtype=torch.bfloat16)[:, :50], t["w"])


@pytest.mark.gpu
def test_nan_stays_with_its_sequence():
    """NaN in one sequence and its window leaves its neighbours' outputs and gradients as they were, whatever tile they share."""
    D, W, cu = 64, 4, [0, 5, 9, 30]
    x = make(15, 1, 30, 3, D, W, "f32")
    t = {n: a.cuda() for n, a in x.items()}
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y0, w0 = gb.gdn_conv_fwd(t["x"], t["w"], t["b"], t["w0"], cut, activation="silu")
    dx0, *_, dw0 = gb.gdn_conv_bwd(t["x"], t["w"], t["dy"], t["b"], t["w0"], t["dwT"], cut, activation="silu")
    for n in ("x", "dy"):
        t[n][:, 5:9] = float("nan")
    t["w0"][1] = t["dwT"][1] = float("nan")
    y, wT = gb.gdn_conv_fwd(t["x"], t["w"], t["b"], t["w0"], cut, activation="silu")
    dx, *_, dw = gb.gdn_conv_bwd(t["x"], t["w"], t["dy"], t["b"], t["w0"], t["dwT"], cut, activation="silu")
    rest = [*range(5), *range(9, 30)]
    assert torch.equal(y[:, rest], y0[:, rest]) and torch.equal(dx[:, rest], dx0[:, rest])
    assert torch.equal(wT[[0, 2]], w0[[0, 2]]) and torch.equal(dw[[0, 2]], dw0[[0, 2]])
    assert torch.isnan(y[:, 5:9]).all() and torch.isnan(dx[:, 5:9]).all() and torch.isnan(dw[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("W", [2, 3, 4])
def test_infinite_gradients_count_once(W):
    """An infinite gradient makes its channel's sums infinite, wherever the token lies in a wave's run, and no NaN."""
    T, D = 64, 64
    x = make(25, 1, T, 1, D, W, "f32")
    t = {n: a.cuda() for n, a in x.items()}
    dy = t["dy"].clone()
    dy[0, torch.arange(T), torch.arange(T)] = float("inf")   # token t: channel t
    _, dw0, db0, _ = gb.gdn_conv_bwd(t["x"], t["w"], t["dy"], t["b"], t["w0"])
    dx, dw, db, _ = gb.gdn_conv_bwd(t["x"], t["w"], dy, t["b"], t["w0"])
    assert (db == float("inf")).all()
    u = torch.cat([t["w0"], t["x"]], 1)[0]
    for j in range(W):
        assert torch.equal(dw[:, j], torch.sign(u[torch.arange(T) + j, torch.arange(T)]) * float("inf"))
    assert torch.isinf(dx[0, torch.arange(T), torch.arange(T)]).all() and torch.isfinite(dw0).all() and torch.isfinite(db0).all()


@pytest.mark.gpu
def test_far_arguments_of_the_activation():
    """Sums of +-1e4: the activation is the sum itself or zero, its slope 1 or 0, with no NaN."""
    x = torch.tensor([1e4, -1e4, 100.0, -100.0, -88.0, 0.0], device="cuda").repeat_interleave(8).view(1, 6, 8)
    w = torch.zeros(8, 2, device="cuda")
    w[:, 1] = 1
    y, _ = gb.gdn_conv_fwd(x, w, activation="silu")
    assert torch.equal(y[0, [0, 2, 5]], x[0, [0, 2, 5]]) and (y[0, [1, 3, 4]].abs() <= 1e-30).all()
    dx, *_ = gb.gdn_conv_bwd(x, w, torch.ones_like(x), activation="silu")
    assert (dx[0, [0, 2]] == 1).all() and (dx[0, [1, 3, 4]].abs() <= 1e-30).all() and (dx[0, 5] == 0.5).all()


RUNS = [
    # lens, D, W, dtype
    ([1], 8, 4, "bf16"), ([1, 0, 3, 48, 0], 264, 4, "bf16"), ([5] * 9, 136, 3, "f32"), ([1] * 70, 520, 2, "bf16"), ([2, 9, 0, 4], 2056, 4, "f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,D,W,dtype", RUNS)
@pytest.mark.parametrize("mode", ["last", "every", "padded"])
@pytest.mark.parametrize("silu", [True, False])
def test_update_against_oracle(lens, D, W, dtype, mode, silu):
    print(f"[gpu] conv update lens={lens[:6]}x{len(lens)} D={D} W={W} {dtype} {mode} silu={silu}", flush=True)
    N, T = len(lens), sum(lens)
    ns = N + T + 3
    x = make(N * 31 + T, 1, T + 2, ns, D, W, dtype)   # two rows behind the last sequence
    gen = torch.Generator().manual_seed(T)
    order = torch.randperm(ns, generator=gen).to(torch.int32)
    cu = torch.tensor([0, *lens]).cumsum(0).to(torch.int32)
    slots, out = order[:N].clone(), None
    if mode == "every":
        out = torch.cat([order[N:N + T], torch.tensor([-1, ns], dtype=torch.int32)])
        out[T // 2] = -1   # a window that is not kept
    if mode == "padded":
        slots[::2] = torch.tensor([-1, ns, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).repeat(N)[: len(slots[::2])]
    bias = x["b"] if silu else None
    pool, y = x["w0"].cuda(), torch.full((T + 2, D), 7.0, dtype=DT[dtype], device="cuda")
    gb.gdn_conv_update(x["x"][0].cuda(), x["w"].cuda(), None if bias is None else bias.cuda(), pool, slots.cuda(), cu.cuda(),
                       None if out is None else out.cuda(), y, activation="silu" if silu else None)
    ref, after = CV.run(x["x"][0], x["w"], bias, x["w0"], slots.numpy(), cu.numpy(), None if out is None else out.numpy(), silu)
    Z = CV.run(x["x"][0].abs(), x["w"].abs(), None if bias is None else bias.abs(), x["w0"].abs(), slots.numpy(), cu.numpy(), None, False)[0]
    inside(y, ref, U * (8 * Z + np.abs(ref) * (Z + 8)) + half(y) * np.abs(ref), "y")
    assert np.array_equal(pool.cpu().double().numpy(), after)
    assert (y[T:] == 7).all()   # rows that no sequence covers


@pytest.mark.gpu
def test_prompt_then_runs():
    """A prompt through gdn_conv_fwd, its window into the pool, then tokens one by one and in runs: the whole sequence's bits."""
    D, W = 264, 4
    x = make(31, 1, 60, 1, D, W, "bf16")
    t = {n: a.cuda() for n, a in x.items()}
    whole, last = gb.gdn_conv_fwd(t["x"], t["w"], t["b"], activation="silu")
    head, win = gb.gdn_conv_fwd(t["x"][:, :41].contiguous(), t["w"], t["b"], activation="silu")
    pool = torch.randn(5, W - 1, D, device="cuda").bfloat16()
    rest = pool.clone()
    pool[3] = win[0]
    slot = torch.tensor([3], dtype=torch.int32, device="cuda")
    parts = [head[0]]
    for a, b in ((41, 42), (42, 43), (43, 50), (50, 60)):
        parts.append(gb.gdn_conv_update(t["x"][0, a:b], t["w"], t["b"], pool, slot, torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
                                        activation="silu"))
    assert torch.equal(torch.cat(parts), whole[0]) and torch.equal(pool[3], last[0])
    assert torch.equal(pool[[0, 1, 2, 4]], rest[[0, 1, 2, 4]])


@pytest.mark.gpu
def test_bad_offsets_stay_inside(monkeypatch):
    """Offsets that fall or leave [0, T] are clamped; GDN_CHECK=1 refuses them and accepts rows behind the last sequence."""
    x = make(6, 1, 40, 3, 64, 4, "bf16")
    t = {n: a.cuda() for n, a in x.items()}
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = torch.tensor([-5, 20, 3, 2000000000], **i32)
    slots = torch.tensor([0, 1, 2], **i32)
    y, wT = gb.gdn_conv_fwd(t["x"], t["w"], t["b"], t["w0"], cu, activation="silu", y=torch.zeros_like(t["x"]))
    gb.gdn_conv_bwd(t["x"], t["w"], t["dy"], t["b"], t["w0"], t["dwT"], cu, activation="silu", dx=torch.zeros_like(t["x"]))
    gb.gdn_conv_update(t["x"][0], t["w"], t["b"], t["w0"], slots, cu, y=torch.zeros_like(t["x"][0]))
    assert torch.isfinite(y.float()).all() and torch.isfinite(wT.float()).all()
    monkeypatch.setenv("GDN_CHECK", "1")
    good, bad = torch.tensor([0, 20, 20, 39], **i32), torch.tensor([0, 20, 3, 40], **i32)
    gb.gdn_conv_fwd(t["x"], t["w"], cu_seqlens=good)
    for f in (lambda: gb.gdn_conv_fwd(t["x"], t["w"], cu_seqlens=bad), lambda: gb.gdn_conv_bwd(t["x"], t["w"], t["dy"], cu_seqlens=bad),
              lambda: gb.gdn_conv_update(t["x"][0], t["w"], None, t["w0"], slots, bad)):
        with pytest.raises(gb.GDNError):
            f()


@pytest.mark.gpu
def test_graph_replay_streams_and_repeats():
    x = make(12, 1, 333, 3, 264, 4, "bf16")
    t = {n: a.cuda() for n, a in x.items()}
    cu = torch.tensor([0, 100, 103, 333], dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")

    def all_three(pool, stream=None):
        y, wT = gb.gdn_conv_fwd(t["x"], t["w"], t["b"], t["w0"], cu, activation="silu", stream=stream)
        g = gb.gdn_conv_bwd(t["x"], t["w"], t["dy"], t["b"], t["w0"], t["dwT"], cu, activation="silu", stream=stream)
        return y, wT, *g, gb.gdn_conv_update(t["x"][0], t["w"], t["b"], pool, slots, cu, activation="silu", stream=stream)

    pools = [t["w0"].clone() for _ in range(3)]
    first = all_three(pools[0])
    second = all_three(pools[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_three(pools[1])
    pools[1].copy_(t["w0"])
    for want in (first, second):
        for a in out:
            a.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        all_three(pools[2])
    assert torch.equal(pools[1], pools[0]) and torch.equal(pools[2], pools[0])
    side = torch.cuda.Stream()
    pools[2].copy_(t["w0"])
    side.wait_stream(torch.cuda.current_stream())
    got = all_three(pools[2], side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Tokens and slots whose elements start past 2^31."""
    D, W = 64, 4
    x = make(8, 1, 36, 1, D, W, "bf16")
    big = torch.zeros(1, 33000, 131072, device="cuda", dtype=torch.bfloat16)
    big[0, 32964:, 70000:70064] = x["x"][0].cuda()
    y, wT = gb.gdn_conv_fwd(big[..., 70000:70064], x["w"].cuda(), x["b"].cuda(), activation="silu")
    check_fwd(x["x"], x["w"], x["b"], None, None, True, y[:, 32964:], wT)
    dy = torch.zeros(1, 33000, D, device="cuda", dtype=torch.bfloat16)
    dy[0, 32964:] = x["dy"][0].cuda()
    gb.gdn_conv_bwd(big[..., 70000:70064], x["w"].cuda(), dy, x["b"].cuda(), activation="silu", dx=big[..., 8:72])
    rdx = CV.backward(x["x"], x["w"], x["b"], None, x["dy"], None, None, True)[0]
    inside(big[:, 32964:, 8:72], rdx, 1e-4 + 2.0 ** -8 * 1.01 * np.abs(rdx), "dx")   # fp32 sums of magnitudes below 100: 1e-4 is far above their u
    del big, dy
    pool = torch.zeros(90000, 3, 8192, device="cuda", dtype=torch.bfloat16)
    z = make(9, 1, 2, 1, 8192, W, "bf16")
    pool[89999] = z["w0"][0].cuda()
    y = gb.gdn_conv_update(z["x"][0].cuda(), z["w"].cuda(), None, pool, torch.tensor([89999], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    ref, after = CV.run(z["x"][0], z["w"], None, z["w0"], [0], [0, 2], None, False)
    assert np.abs(y.cpu().double().numpy() - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-5
    assert np.array_equal(pool[89999].cpu().double().numpy(), after[0]) and not pool[:89999].any()


@pytest.mark.gpu
def test_more_work_groups_than_one_row_of_the_grid():
    """Forward work-groups past 2^23, which go on in the grid's second row: 24 tokens each of 8 channels; a broadcast token, so that all
    rows behind the first W - 1 are alike, and a window behind the end."""
    T, D, W = 24 * (1 << 23) + 1000, 8, 4
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB")
    print(f"[gpu] conv T={T} D={D}", flush=True)
    x = make(3, 1, 1, 1, D, W, "bf16")
    t = {n: a.cuda() for n, a in x.items()}
    y = torch.zeros(1, T, D, device="cuda", dtype=torch.bfloat16)
    _, wT = gb.gdn_conv_fwd(t["x"].expand(1, T, D), t["w"], t["b"], t["w0"], activation="silu", y=y)
    n = W + 2
    want, _ = gb.gdn_conv_fwd(t["x"].expand(1, n, D).contiguous(), t["w"], t["b"], t["w0"], activation="silu")
    check_fwd(x["x"].expand(1, n, D), x["w"], x["b"], x["w0"], None, True, want, None)
    assert torch.equal(y[:, :W], want[:, :W]) and torch.equal(wT, t["x"].expand(1, W - 1, D))
    edge = 24 * (1 << 23)
    for lo, hi in ((W, 5000), (edge - 5000, edge + 1000), ((1 << 27) - 100, (1 << 27) + 100)):
        assert torch.equal(y[0, lo:hi], want[0, n - 1].expand(hi - lo, D)), lo
    assert torch.equal(y[0, W:].amin(0), want[0, n - 1]) and torch.equal(y[0, W:].amax(0), want[0, n - 1])
