"""gdn_layer_norm_fwd / gdn_layer_norm_bwd: the oracle against differences and the refusals (CPU), the kernels against the oracle (GPU).

Tolerances (u = 2^-24, half a step of fp32). A row's sum is at most 32 serial additions a lane, 6 tree levels and 8 waves: the mean is off by
at most 48 u of the row's largest magnitude A, a centred value by that and its own rounding; in units of the deviation, xh is off by
64 u (A rstd + |xh|), the variance's own rounding (the same sums, a root, a reciprocal) included. y takes a product and a sum more. In the
backward pass the two means of g and g xh take the same sums, so with m = max |g| dx is off by at most 256 u rstd m (1 + max |xh|) (1 + A
rstd + max |xh|). The gradients of weight and bias are sums of at most 64 rows a lane here, then trees: 128 u of
the sum of magnitudes, and xh's own error. A bf16 output adds half a step, 2^-8 of the value. The sum with the residual is
one fp32 addition and one rounding: exactly torch's.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_42_amd import binding as gb
from oracle import layernorm as LN

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
P = 1 << 12   # any aligned non-NULL pointer: the checks run before any launch


# ------------------------------------------------------------------------------------------ CPU
def test_oracle_gradients_match_differences():
    rng = np.random.default_rng(5)
    R, d = 3, 16
    s, dy, ds = rng.standard_normal((R, d)) + 0.5, rng.standard_normal((R, d)), rng.standard_normal((R, d))
    w, b = 1 + 0.3 * rng.standard_normal(d), rng.standard_normal(d)
    f = lambda s, w, b: float((LN.forward(s, w, b, 1e-3) * dy + s * ds).sum())  # noqa: E731
    dx, dw, db = LN.backward(s, dy, w, ds, 1e-3)
    h = 1e-5   # central differences: error of order h^2 times third derivatives of order 10
    for i in range(s.size):
        e = np.zeros(s.size)
        e[i] = h
        e = e.reshape(s.shape)
        assert abs((f(s + e, w, b) - f(s - e, w, b)) / (2 * h) - dx.reshape(-1)[i]) < 1e-7
    for i in range(d):
        e = np.zeros(d)
        e[i] = h
        assert abs((f(s, w + e, b) - f(s, w - e, b)) / (2 * h) - dw[i]) < 1e-7
        assert abs((f(s, w, b + e) - f(s, w, b - e)) / (2 * h) - db[i]) < 1e-7


def c_fwd(**kw):
    a = dict(x=P, r=None, w=None, b=None, y=P, s=None, rows=4, d=64, xs=64, rs=64, eps=1e-5, dtype=1, sd=1, od=1)
    a.update(kw)
    return gb.lib().gdn_layer_norm_fwd(*a.values(), None)


def c_bwd(**kw):
    a = dict(s=P, dy=P, ds=None, w=None, dx=P, dw=None, db=None, rows=4, d=64, ss=64, eps=1e-5, dtype=1, od=1, ws=None, wb=0)
    a.update(kw)
    return gb.lib().gdn_layer_norm_bwd(*a.values(), None)


SHARED = [(dict(dtype=2), -3), (dict(od=-1), -3), (dict(d=60), -5), (dict(d=0), -5), (dict(d=16392), -5), (dict(rows=-1), -2),
          (dict(rows=1 << 28), -2), (dict(rows=1 << 24, d=16384), -2), (dict(eps=0.0), -2), (dict(eps=float("nan")), -2),
          (dict(w=P + 4), -4)]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(r=P, s=P, sd=2), -3), (dict(r=P, s=P, sd=1, dtype=0), -3), (dict(xs=-64), -2), (dict(rs=-64), -2), (dict(x=None), -1),
    (dict(y=None), -1), (dict(r=P), -1), (dict(x=P + 8), -4), (dict(y=P + 8), -4), (dict(b=P + 4), -4), (dict(xs=65), -4),
    (dict(r=P, s=P, rs=68), -4), (dict(r=P, s=P + 4), -4), (dict(r=P, s=P), -2)])
def test_fwd_refuses(kw, status):
    assert c_fwd(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(ss=-64), -2), (dict(s=None), -1), (dict(dy=None), -1), (dict(dx=None), -1), (dict(s=P + 8), -4), (dict(ds=P + 2), -4),
    (dict(ss=65), -4), (dict(dw=P + 2), -4), (dict(dw=P), -6), (dict(db=P, ws=P, wb=16), -6), (dict(dw=P, ws=P + 16, wb=1 << 20), -4)])
def test_bwd_refuses(kw, status):
    assert c_bwd(**kw) == status


def test_nothing_to_do_is_ok():
    assert c_fwd(rows=0, x=None, y=None) == 0
    assert c_bwd(rows=0, s=None, dy=None, dx=None) == 0
    w = gb.gdn_layer_norm_bwd_workspace_bytes
    assert w(0, 64) == 0 and w(4, 60) == 0 and w(-1, 64) == 0 and w(4, 64) == 2 * 64 * 4


def test_binding_refuses_on_the_host():
    m = lambda *s, dt=torch.float32: torch.empty(*s, device="meta", dtype=dt)  # noqa: E731
    for args, kw, text in (
            ((m(2, 64, dt=torch.float16),), {}, "float32 or bfloat16"), ((m(2, 64), m(32)), {}, "weight has shape"),
            ((m(2, 64), m(64), m(64, dt=torch.bfloat16)), {}, "bias has dtype"), ((m(2, 64),), dict(residual=m(1, 64)), "residual has shape"),
            ((m(2, 64),), dict(residual=m(2, 64, dt=torch.bfloat16)), "residual has dtype"), ((m(2, 64),), dict(sum_out=m(2, 64)), "needs a residual"),
            ((m(2, 64),), {}, "on a GPU")):
        with pytest.raises(ValueError, match=text):
            gb.gdn_layer_norm_fwd(*args, **kw)
    with pytest.raises(ValueError, match="exceeds"):
        gb.gdn_layer_norm_fwd(m((1 << 32) + 8, 64))
    with pytest.raises(ValueError, match="exceeds"):
        gb.gdn_layer_norm_bwd(m((1 << 32) + 8, 64), m((1 << 32) + 8, 64))
    for args, kw, text in (((m(2, 64), m(2, 32)), {}, "dy has shape"), ((m(2, 64), m(2, 64)), dict(ds=m(2, 64, dt=torch.bfloat16)), "ds has dtype"),
                           ((m(2, 64), m(2, 64)), {}, "on a GPU")):
        with pytest.raises(ValueError, match=text):
            gb.gdn_layer_norm_bwd(*args, **kw)


# ------------------------------------------------------------------------------------------ GPU
def make(seed, rows, d, dtype, sum_dtype, offset=1.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(x=(r(rows, d) * 2 + offset * r(d)).to(DT[dtype]), r=(r(rows, d) * 3).to(DT[sum_dtype]), w=1 + 0.3 * r(d), b=r(d),
                dy=r(rows, d).to(DT[dtype]), ds=r(rows, d).to(DT[sum_dtype]))


def stats(s):
    s = s.double().numpy()
    xh, rstd = LN.normalise(s, 1e-5)
    return np.abs(s).max(-1, keepdims=True) if s.size else s[..., :1], xh, rstd


def half(t):
    return 2.0 ** -8 * (1 + 2.0 ** -8) if t.dtype == torch.bfloat16 else U


def inside(got, ref, tol, name):
    got = got.cpu().double().numpy()
    over = np.abs(got - ref) - tol
    print(f"      {name}: largest error over its tolerance {float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max() if got.size else 0):.3f}", flush=True)
    assert got.shape == ref.shape and (over <= 0).all(), name


def check_fwd(x, w, b, y):
    A, xh, rstd = stats(x)
    wa = 1.0 if w is None else np.abs(w.double().numpy())
    ref = LN.forward(x, w, b, 1e-5)
    tol = 64 * U * (A * rstd + np.abs(xh)) * wa + 4 * U * (np.abs(xh) * wa + (0 if b is None else np.abs(b.double().numpy())))
    inside(y, ref, tol + half(y) * np.abs(ref), "y")


def check_bwd(s, dy, w, ds, dx, dw, db):
    A, xh, rstd = stats(s)
    rdx, rdw, rdb = LN.backward(s, dy, w, ds, 1e-5)
    dyn = np.abs(dy.double().numpy())
    g = dyn if w is None else dyn * np.abs(w.double().numpy())
    big = np.abs(xh).max(-1, keepdims=True)
    tol = 256 * U * rstd * g.max(-1, keepdims=True) * (1 + big) * (1 + A * rstd + big) + (0 if ds is None else 2 * U * np.abs(ds.double().numpy()))
    inside(dx, rdx, tol + half(dx) * np.abs(rdx), "dx")
    if dw is not None:
        inside(dw, rdw, 128 * U * (dyn * (np.abs(xh) + A * rstd)).sum(0), "dw")
        inside(db, rdb, 128 * U * dyn.sum(0), "db")


# every number of lanes and pieces, and the edges between them
WIDTHS = [8, 64, 128, 136, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


@pytest.mark.gpu
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype,sum_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_against_oracle(d, dtype, sum_dtype):
    rows = 37 if d <= 512 else 9
    print(f"[gpu] layer norm rows={rows} d={d} {dtype} sum {sum_dtype}", flush=True)
    x = make(d + rows, rows, d, dtype, sum_dtype)
    t = {n: a.cuda() for n, a in x.items()}
    for od in (torch.float32, torch.bfloat16):
        y, s = gb.gdn_layer_norm_fwd(t["x"], t["w"], t["b"], residual=t["r"], out_dtype=od)
        want = (x["x"].float() + x["r"].float()).to(DT[sum_dtype])
        assert y.dtype == od and torch.equal(s.cpu(), want)
        check_fwd(want, x["w"], x["b"], y)
    y, none = gb.gdn_layer_norm_fwd(t["x"])
    assert none is None and y.dtype == DT[dtype]
    check_fwd(x["x"], None, None, y)
    y, _ = gb.gdn_layer_norm_fwd(t["x"], None, t["b"])
    check_fwd(x["x"], None, x["b"], y)
    s = (x["x"].float() + x["r"].float()).to(DT[sum_dtype])
    for od in (torch.float32, torch.bfloat16):
        dy = t["dy"].to(od)
        check_bwd(s, dy.cpu(), x["w"], x["ds"], *gb.gdn_layer_norm_bwd(s.cuda(), dy, t["w"], ds=t["ds"]))
    dx, dw, db = gb.gdn_layer_norm_bwd(s.cuda(), t["dy"])
    assert dw is None and db is None
    check_bwd(s, x["dy"], None, None, dx, None, None)
    check_bwd(s, x["dy"], None, None, *gb.gdn_layer_norm_bwd(s.cuda(), t["dy"], need_dw=True))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(1, 2048), (1, 64), (2, 8200), (1237, 200), (3000, 96), (2051, 1000), (700, 4096)])
def test_row_counts(rows, d):
    """More rows than work-groups take at once, and one."""
    print(f"[gpu] layer norm rows={rows} d={d}", flush=True)
    x = make(rows + d, rows, d, "bf16", "bf16")
    t = {n: a.cuda() for n, a in x.items()}
    y, s = gb.gdn_layer_norm_fwd(t["x"], t["w"], t["b"], residual=t["r"])
    check_fwd(s.cpu(), x["w"], x["b"], y)
    dx, dw, db = gb.gdn_layer_norm_bwd(s, t["dy"], t["w"], ds=t["ds"])
    keep = torch.randperm(rows, generator=torch.Generator().manual_seed(1))[:40]   # dx row by row; the sums over all rows
    check_bwd(s.cpu()[keep], x["dy"][keep], x["w"], x["ds"][keep], dx[keep.cuda()], None, None)
    xh, rstd = LN.normalise(s.cpu().double().numpy(), 1e-5)
    dyn, A = x["dy"].double().numpy(), np.abs(s.cpu().double().numpy()).max(-1, keepdims=True)
    inside(dw, (dyn * xh).sum(0), 128 * U * (np.abs(dyn) * (np.abs(xh) + A * rstd)).sum(0), "dw")
    inside(db, dyn.sum(0), 128 * U * np.abs(dyn).sum(0), "db")


@pytest.mark.gpu
def test_zero_rows():
    t = torch.zeros(0, 64, device="cuda")
    y, s = gb.gdn_layer_norm_fwd(t, residual=t)
    assert y.shape == s.shape == (0, 64)
    dx, dw, db = gb.gdn_layer_norm_bwd(t, t, torch.ones(64, device="cuda"))
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


@pytest.mark.gpu
def test_strides_leading_dimensions_and_places():
    """Views of a fused tensor, a broadcast row, leading dimensions, outputs over inputs."""
    x = make(3, 24, 128, "bf16", "bf16")
    t = {n: a.cuda() for n, a in x.items()}
    y0, s0 = gb.gdn_layer_norm_fwd(t["x"], t["w"], t["b"], residual=t["r"])
    fused = torch.randn(24, 384, device="cuda").bfloat16()
    fused[:, 128:256], fused[:, 256:] = t["x"], t["r"]
    xv, rv = fused[:, 128:256].view(4, 6, 128), fused[:, 256:].view(4, 6, 128)
    y, s = gb.gdn_layer_norm_fwd(xv, t["w"], t["b"], residual=rv)
    assert y.shape == (4, 6, 128) and torch.equal(y.flatten(0, 1), y0) and torch.equal(s.flatten(0, 1), s0)
    dx0, dw0, db0 = gb.gdn_layer_norm_bwd(t["x"], t["dy"], t["w"])
    dx, dw, db = gb.gdn_layer_norm_bwd(xv, t["dy"].view(4, 6, 128), t["w"])
    assert torch.equal(dx.flatten(0, 1), dx0) and torch.equal(dw, dw0) and torch.equal(db, db0)
    row = t["x"][:1].expand(24, 128)
    y, _ = gb.gdn_layer_norm_fwd(row, t["w"], t["b"])
    assert torch.equal(y, gb.gdn_layer_norm_fwd(t["x"][:1].contiguous(), t["w"], t["b"])[0].expand(24, 128))
    one, _ = gb.gdn_layer_norm_fwd(t["x"][0], t["w"], t["b"])   # a single row without leading dimensions
    assert torch.equal(one, y[0])
    a, b = t["x"].clone(), t["r"].clone()
    y, s = gb.gdn_layer_norm_fwd(a, t["w"], t["b"], residual=b, y=a, sum_out=b)
    assert y is a and s is b and torch.equal(a, y0) and torch.equal(b, s0)
    d = t["ds"].clone()
    want = gb.gdn_layer_norm_bwd(t["x"], t["dy"], t["w"], ds=t["ds"])
    got = gb.gdn_layer_norm_bwd(t["x"], t["dy"], t["w"], ds=d, dx=d)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    with pytest.raises(ValueError, match="last dimension"):
        gb.gdn_layer_norm_fwd(t["x"].t())
    with pytest.raises(gb.GDNError):
        gb.gdn_layer_norm_fwd(torch.zeros(600, device="cuda", dtype=torch.bfloat16)[4:516].view(4, 128))


@pytest.mark.gpu
def test_offsets_constants_and_special_values():
    """A mean far above the deviation, constant rows (variance 0), NaN and infinity that stay in their row."""
    x = make(9, 8, 640, "f32", "f32", offset=0.0)
    s = x["x"] * 0.01
    s[1] += 300.0
    s[2] = 7.0
    y, _ = gb.gdn_layer_norm_fwd(s.cuda(), x["w"].cuda(), x["b"].cuda())
    check_fwd(s, x["w"], x["b"], y)
    check_bwd(s, x["dy"], x["w"], x["ds"], *gb.gdn_layer_norm_bwd(s.cuda(), x["dy"].cuda(), x["w"].cuda(), ds=x["ds"].cuda()))
    clean = gb.gdn_layer_norm_bwd(s.cuda(), x["dy"].cuda(), x["w"].cuda())[0]
    s[3, 5], s[4, 600] = float("nan"), float("inf")
    y2, _ = gb.gdn_layer_norm_fwd(s.cuda(), x["w"].cuda(), x["b"].cuda())
    d2 = gb.gdn_layer_norm_bwd(s.cuda(), x["dy"].cuda(), x["w"].cuda())[0]
    good = [0, 1, 2, 5, 6, 7]
    assert torch.equal(y2[good], y[good]) and torch.equal(d2[good], clean[good])
    assert torch.isnan(y2[3:5]).all() and torch.isnan(d2[3:5]).all()


@pytest.mark.gpu
def test_graph_replay_streams_and_repeats():
    x = make(12, 300, 2048, "bf16", "f32")
    t = {n: a.cuda() for n, a in x.items()}
    y0, s0 = gb.gdn_layer_norm_fwd(t["x"], t["w"], t["b"], residual=t["r"])
    g0 = gb.gdn_layer_norm_bwd(s0, t["dy"], t["w"], ds=t["ds"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s = gb.gdn_layer_norm_fwd(t["x"], t["w"], t["b"], residual=t["r"])
        g = gb.gdn_layer_norm_bwd(s, t["dy"], t["w"], ds=t["ds"])
    for _ in range(4):
        for a in (y, s, *g):
            a.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(s, s0) and all(torch.equal(a, b) for a, b in zip(g, g0))
        again = gb.gdn_layer_norm_bwd(s0, t["dy"], t["w"], ds=t["ds"])
        assert all(torch.equal(a, b) for a, b in zip(again, g0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, s1 = gb.gdn_layer_norm_fwd(t["x"], t["w"], t["b"], residual=t["r"], stream=side)
    g1 = gb.gdn_layer_norm_bwd(s1, t["dy"], t["w"], ds=t["ds"], stream=side)
    side.synchronize()
    assert torch.equal(y1, y0) and all(torch.equal(a, b) for a, b in zip(g1, g0))


@pytest.mark.gpu
def test_more_lanes_than_32_bits():
    """2^32 lanes and more (32 for a row of 136 channels) of one broadcast row; without the weights' gradients backward."""
    rows, d = (1 << 27) + 40, 136
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 110 GiB")
    print(f"[gpu] layer norm {rows} x {d}", flush=True)
    x = torch.randn(1, d, device="cuda").bfloat16()
    one, _ = gb.gdn_layer_norm_fwd(x)
    y, _ = gb.gdn_layer_norm_fwd(x.expand(rows, d), y=torch.zeros(rows, d, device="cuda", dtype=torch.bfloat16))
    at = torch.tensor([0, 1, (1 << 26) - 1, 1 << 26, (1 << 27) - 1, 1 << 27, rows - 1], device="cuda")
    assert torch.equal(y[at], one.expand(len(at), d))
    dy = torch.randn(1, d, device="cuda").bfloat16()
    want, _, _ = gb.gdn_layer_norm_bwd(x, dy)
    y.copy_(dy.expand(rows, d))
    dx, _, _ = gb.gdn_layer_norm_bwd(x.expand(rows, d), y, dx=torch.zeros(rows, d, device="cuda", dtype=torch.bfloat16))
    assert torch.equal(dx[at], want.expand(len(at), d))


@pytest.mark.gpu
def test_rows_past_32_bits():
    """Rows whose elements start past 2^31 (a view of strided rows of 8.6 GB)."""
    big = torch.zeros(33000, 131072, device="cuda", dtype=torch.bfloat16)
    x = make(4, 3, 256, "bf16", "bf16")
    at = [0, 17000, 32999]
    big[at, :256] = x["x"].cuda()
    y, _ = gb.gdn_layer_norm_fwd(big[:, :256], x["w"].cuda(), x["b"].cuda())
    check_fwd(x["x"], x["w"], x["b"], y[at])
    dy = torch.zeros(33000, 256, device="cuda", dtype=torch.bfloat16)
    dy[at] = x["dy"].cuda()
    dx, dw, db = gb.gdn_layer_norm_bwd(big[:, :256], dy, x["w"].cuda())
    check_bwd(x["x"], x["dy"], x["w"], None, dx[at], None, None)
    xh, rstd = LN.normalise(x["x"], 1e-5)
    dyn, A = x["dy"].double().numpy(), np.abs(x["x"].double().numpy()).max(-1, keepdims=True)
    inside(dw, (dyn * xh).sum(0), 128 * U * (np.abs(dyn) * (np.abs(xh) + A * rstd)).sum(0), "dw")   # rows of zeros add nothing
