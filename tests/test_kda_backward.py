"""gdn_kda_chunk_bwd: the fp64 oracle against differences and the refusals (CPU), the kernels against the oracle (GPU).

Tolerance: all arithmetic is fp32 (u = 2^-24 = 6e-8) for both input types, so every gradient is held to 1e-4 of its
tensor's largest magnitude, the library's tolerance for fp32 inputs: a chunk's products sum at most 128 + 64 terms in
sequence (under 200 u = 1.2e-5 of the sum of magnitudes), dg adds the reverse sum over 64 rows of terms of that error, whose
signs are independent (another factor of about 8 at the worst row). bf16 gradients are those fp32 results
rounded, bit for bit.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_42_amd import binding as gb
from gated_delta_rule_42_amd import synthetic as SY
from oracle import kda as KD
from oracle import kda_backward as KB

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh0")
P = 1 << 12


# ------------------------------------------------------------------------------------------ CPU
def test_oracle_matches_differences():
    rng = np.random.default_rng(5)
    T, H, dk, dv = 7, 1, 4, 3
    cu = np.array([0, 3, 3, 7])
    x = dict(q=rng.standard_normal((1, T, H, dk)), k=rng.standard_normal((1, T, H, dk)) * 0.6,
             v=rng.standard_normal((1, T, H, dv)), g=-rng.random((1, T, H, dk)), beta=rng.random((1, T, H)) * 1.5,
             h0=rng.standard_normal((3, H, dv, dk)))
    do, dhT = rng.standard_normal((1, T, H, dv)), rng.standard_normal((3, H, dv, dk))

    def loss(y):
        o, hT = KD.forward(y["q"], y["k"], y["v"], y["g"], y["beta"], y["h0"], cu)
        return float((o * do).sum() + (hT * dhT).sum())

    grads = KB.backward(x["q"], x["k"], x["v"], x["g"], x["beta"], do, x["h0"], dhT, cu)
    h = 1e-5   # central differences: off by h^2 times third derivatives of order 10
    for name, gr in zip(("q", "k", "v", "g", "beta", "h0"), grads):
        for i in range(x[name].size):
            e = np.zeros(x[name].size)
            e[i] = h
            e = e.reshape(x[name].shape)
            d = (loss({**x, name: x[name] + e}) - loss({**x, name: x[name] - e})) / (2 * h)
            assert abs(d - gr.reshape(-1)[i]) < 1e-6 * max(1, abs(d)), (name, i)


def c_call(**kw):
    a = dict(q=P, k=P, v=P, g=P, beta=P, h0=None, do=P, dhT=None, dq=P, dk=P, dv=P, dg=P, db=P, dh0=None, cu=None, chunk=64, B=1,
             T=64, H=1, dkk=64, dvv=64, N=1, dtype=1, gd=1, ws=P, wb=1 << 30)
    a.update(kw)
    return gb.lib().gdn_kda_chunk_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -3), (dict(gd=2), -3), (dict(dtype=0, gd=1), -3), (dict(chunk=32), -5), (dict(dkk=96), -5), (dict(dvv=32), -5),
    (dict(B=0), -2), (dict(T=-1), -2), (dict(H=0), -2), (dict(N=2), -2), (dict(cu=P, B=2, N=3), -2), (dict(q=None), -1),
    (dict(g=None), -1), (dict(do=None), -1), (dict(dg=None), -1), (dict(db=None), -1), (dict(g=P + 4), -4), (dict(dg=P + 8), -4),
    (dict(dh0=P + 4), -4), (dict(beta=P + 2), -4), (dict(ws=None), -6), (dict(wb=100), -6), (dict(ws=P + 64), -4),
    (dict(N=1 << 21, cu=P), -2), (dict(T=1 << 30, H=1 << 14), -2),
])
def test_refuses(kw, status):
    assert c_call(**kw) == status


def test_workspace_matches_its_regions():
    f = gb.gdn_kda_chunk_bwd_workspace_bytes
    assert f(1, 64, 1, 96, 64, 1, False) == 0 and f(0, 64, 1, 64, 64, 0, False) == 0
    assert f(1, 0, 1, 64, 64, 1, False) == 0
    for B, T, H, dk, dv, N, var in ((2, 130, 3, 128, 64, 2, False), (1, 100, 2, 64, 128, 5, True)):
        nc = (T + 63 * N) // 64 if var else B * ((T + 63) // 64)
        al = lambda x: (x + 255) // 256 * 256  # noqa: E731
        u, w = nc * H, gb.gdn_kda_chunk_fwd_workspace_bytes(B, T, H, dk, dv, N, var, dtype=torch.float32)
        for n in (u * dv * dk, u * dv * dk, u * 64 * dv, u * 64 * dv):
            w = al(w) + 4 * n
        assert f(B, T, H, dk, dv, N, var) == w


def test_binding_refuses_on_the_host():
    m = lambda *s, dt=torch.float32: torch.empty(*s, device="meta", dtype=dt)  # noqa: E731
    good = dict(q=m(1, 8, 2, 64), k=m(1, 8, 2, 64), v=m(1, 8, 2, 64), g=m(1, 8, 2, 64), beta=m(1, 8, 2), do=m(1, 8, 2, 64))
    for change, text in ((dict(g=m(1, 8, 2)), "g has shape"), (dict(do=m(1, 8, 2, 128)), "do has shape"),
                         (dict(dhT=m(2, 2, 64, 64)), "hT has shape"), (dict(), "on a GPU")):
        with pytest.raises(ValueError, match=text):
            gb.gdn_kda_chunk_bwd(**{**good, **change})


# ------------------------------------------------------------------------------------------ GPU
def gpu_bwd(x, cot, **kw):
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    out = gb.gdn_kda_chunk_bwd(*(c(x[n]) for n in ("q", "k", "v", "g", "beta")), c(cot["do"]), c(x["h0"]), c(cot["dhT"]),
                               c(x["cu_seqlens"]), **kw)
    torch.cuda.synchronize()
    return out


def check(x, cot, heads=None):
    print(f"[gpu] kda_chunk_bwd {x['meta']} dhT={cot['dhT'] is not None}", flush=True)
    got = gpu_bwd(x, cot, grad_dtype=torch.float32)
    sl = (lambda t: t) if heads is None else (lambda t: None if t is None else t[:, :, heads].contiguous())
    slN = (lambda t: t) if heads is None else (lambda t: None if t is None else t[:, heads].contiguous())
    ref = KB.backward(*(sl(x[n]) for n in ("q", "k", "v", "g", "beta")), sl(cot["do"]), slN(x["h0"]), slN(cot["dhT"]),
                      x["cu_seqlens"])
    errs = {}
    for name, a, r in zip(NAMES, got, ref):
        a = a.cpu().double().numpy()
        if heads is not None:
            a = a[:, heads] if name == "dh0" else a[:, :, heads]
        assert np.isfinite(a).all(), name
        errs[name] = np.abs(a - r).max() / max(np.abs(r).max(), 1e-30) if r.size else 0.0
    print("      " + " ".join(f"{n}={e:.2e}" for n, e in errs.items()), flush=True)
    assert all(e <= 1e-4 for e in errs.values()), errs


def make(seed, B, T, H, dk, dv, dtype, h0, gs, lengths=None, beta_scale=1.0):
    w = SY.Workload(99, "kda_bwd", H=H, dk=dk, dv=dv, dtype=dtype, B=B, T=T, varlen=len(lengths or ()))
    x = SY.make_forward_inputs(w, seed=seed, gate_scale=1.0, h0=h0, lengths=lengths, beta_scale=beta_scale)
    return SY.channel_gates(x, seed + 1, gate_scale=gs)


SMALL = [
    # B, T, H, dk, dv, dtype, h0, dhT, gate_scale
    (1, 1, 1, 64, 64, "f32", True, True, 1.0),
    (1, 16, 1, 128, 128, "f32", False, False, 0.1),
    (1, 65, 2, 64, 64, "bf16", True, True, 0.02),
    (1, 200, 2, 64, 64, "f32", True, True, 1.0),
    (2, 130, 2, 128, 128, "f32", True, True, 0.01),
    (1, 100, 2, 64, 128, "f32", False, False, 1.0),
    (1, 190, 2, 128, 64, "f32", True, True, 0.05),
    (2, 150, 2, 128, 128, "bf16", True, True, 1.0),
    (1, 257, 3, 128, 128, "bf16", True, True, 0.01),
    (1, 190, 2, 128, 64, "bf16", True, False, 0.05),
    (2, 100, 2, 64, 128, "bf16", False, True, 0.3),
    (1, 190, 2, 128, 128, "f32", True, True, 5.0),      # decays up to e^-30 a token
    (1, 130, 1, 64, 64, "f32", True, True, 60.0),       # decays below fp32's smallest number
    (1, 130, 1, 128, 128, "f32", True, True, 0.0),      # no decay at all
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,H,dk,dv,dtype,h0,dhT,gs", SMALL)
def test_small(B, T, H, dk, dv, dtype, h0, dhT, gs):
    x = make(7000 + T + dk + dv, B, T, H, dk, dv, dtype, h0, gs)
    check(x, SY.make_cotangents(x, 8000 + T, dhT=dhT))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,dk,dv,dtype,packed", [
    (100, 66, 64, 64, "f32", False), (130, 34, 64, 128, "bf16", False), (130, 67, 128, 64, "bf16", False),
    (150, 33, 128, 128, "f32", False), (0, 70, 128, 128, "bf16", True)])
def test_many_heads(T, H, dk, dv, dtype, packed):
    """Enough (sequence, head) pairs for work-groups of 64 columns; not multiples of eight."""
    x = make(71, 1, T, H, dk, dv, dtype, True, 0.1, lengths=[65, 40] if packed else None)
    check(x, SY.make_cotangents(x, 72), heads=[0, H // 2, H - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,dk,dv,dtype,packed", [
    (130, 17, 64, 128, "f32", False), (150, 32, 128, 128, "bf16", False), (100, 35, 64, 64, "bf16", False),
    (130, 33, 128, 64, "f32", False), (0, 30, 128, 128, "bf16", True)])
def test_middling_heads(T, H, dk, dv, dtype, packed):
    """(sequence, head) pairs for work-groups of 32 columns."""
    x = make(73, 1, T, H, dk, dv, dtype, True, 0.1, lengths=[65, 40] if packed else None)
    check(x, SY.make_cotangents(x, 74), heads=[0, H // 2, H - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dk,dv", [("f32", 128, 128), ("bf16", 128, 128), ("bf16", 64, 128)])
def test_packed(dtype, dk, dv):
    """Packed sequences, some of them empty (their dh0 is dhT), single tokens, ends inside and at chunk borders."""
    x = make(41, 1, 0, 2, dk, dv, dtype, True, 0.05, lengths=[0, 70, 0, 1, 64, 129, 15, 0])
    cot = SY.make_cotangents(x, 42)
    check(x, cot)
    out = gpu_bwd(x, cot)
    for n in (0, 2, 7):
        assert torch.equal(out[5][n].cpu(), cot["dhT"][n])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dk,dhT", [("f32", 64, False), ("bf16", 128, False), ("bf16", 128, True)])
def test_single_tokens_from_nothing(dtype, dk, dhT):
    """A first token's decay acts on a state of zeros, so its gradient is zero, not the rounding of terms that cancel."""
    x = make(51, 1, 0, 3, dk, 64, dtype, False, 0.5, lengths=[1, 0, 1, 1])
    cot = SY.make_cotangents(x, 52, dhT=dhT)
    check(x, cot)
    assert not gpu_bwd(x, cot)[3].any()


@pytest.mark.gpu
def test_beta_to_2_and_mixed_decays():
    """Erasing strengths beyond 1, and channels of very different decays side by side (one of them stepwise)."""
    x = make(43, 1, 200, 2, 128, 128, "bf16", True, 0.01, beta_scale=2.0)
    x["g"][..., ::3] *= 3000.0
    x["g"][..., 5] = 0.0
    x["g"][:, 77, :, 7] = -1e4
    check(x, SY.make_cotangents(x, 44))


@pytest.mark.gpu
def test_bf16_gradients_are_rounded_fp32_and_repeat():
    x = make(45, 1, 150, 2, 64, 128, "bf16", True, 0.3)
    cot = SY.make_cotangents(x, 46)
    a, b, c = gpu_bwd(x, cot, grad_dtype=torch.float32), gpu_bwd(x, cot), gpu_bwd(x, cot, need_dh0=False)
    assert c[5] is None
    for i in range(6):
        want = a[i].to(torch.bfloat16) if i < 3 else a[i]
        assert torch.equal(want, b[i]) and (c[i] is None or torch.equal(b[i], c[i])), NAMES[i]


@pytest.mark.gpu
def test_train_workload_sampled_heads():
    """The training shape (B4 H16 T2048 d128, bf16) in full on the GPU; the oracle computes one of the heads."""
    x = SY.channel_gates(SY.make_forward_inputs(1), 5, gate_scale=0.1)
    check(x, SY.make_cotangents(x, 101), heads=[11])


@pytest.mark.gpu
def test_gradients_match_differences_of_the_forward_pass():
    """Directional differences of gdn_kda_chunk_fwd's own fp32 outputs. In fp32 the loss of ~ 2e4 terms is summed in fp64; the
    outputs carry about 1e-6 of relative error each, independent, so with a step of 1e-2 a difference is off by about
    1e-6 sqrt(2e4) / 1e-2 = 1.4e-2 plus the step's own h^2; gradients along random directions are of order 100."""
    x = make(51, 1, 130, 1, 64, 64, "f32", True, 0.1)
    cot = SY.make_cotangents(x, 52)
    grads = gpu_bwd(x, cot)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "g", "beta", "h0")}
    do, dhT = cot["do"].cuda().double(), cot["dhT"].cuda().double()

    def loss(y):
        o, hT = gb.gdn_kda_chunk_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["h0"])
        return float((o.double() * do).sum() + (hT.double() * dhT).sum())

    gen = torch.Generator(device="cuda").manual_seed(1)
    for name, gr in zip(("q", "k", "v", "g", "beta", "h0"), grads):
        e = torch.randn(d[name].shape, generator=gen, device="cuda")
        e = -e.abs() * 0.3 if name == "g" else e   # g stays below zero
        along = float((gr.double() * e.double()).sum())
        h = 1e-2
        # second differences bound the curvature that a one-sided step at g's border would see
        diff = (loss({**d, name: d[name] + h * e}) - loss({**d, name: d[name] - h * e})) / (2 * h)
        print(name, along, diff, flush=True)
        assert abs(along - diff) <= 0.02 * max(10.0, abs(along)), name


@pytest.mark.gpu
def test_graph_stream_and_shared_workspace():
    """A captured call replayed between eager calls, both on one workspace; another stream."""
    x = make(61, 1, 200, 2, 128, 128, "bf16", True, 0.2)
    cot = SY.make_cotangents(x, 62)
    d = [x[n].cuda() for n in ("q", "k", "v", "g", "beta")] + [cot["do"].cuda(), x["h0"].cuda(), cot["dhT"].cuda()]
    ws = torch.empty(gb.gdn_kda_chunk_bwd_workspace_bytes(1, 200, 2, 128, 128, 1, False), dtype=torch.uint8, device="cuda")
    want = gb.gdn_kda_chunk_bwd(*d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = gb.gdn_kda_chunk_bwd(*d, workspace=ws)
    for _ in range(3):
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))
        assert all(torch.equal(a, b) for a, b in zip(want, gb.gdn_kda_chunk_bwd(*d, workspace=ws)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gb.gdn_kda_chunk_bwd(*d, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.gpu
def test_empty_problem():
    z = torch.zeros(1, 0, 2, 64, device="cuda")
    h = torch.randn(1, 2, 64, 64, device="cuda")
    out = gb.gdn_kda_chunk_bwd(z, z, z, z, z[..., 0].contiguous(), z, None, h)
    assert torch.equal(out[5], h) and out[0].numel() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dk", [("f32", 128), ("f32", 64), ("bf16", 128), ("bf16", 64)])
def test_nan_gate_shows(dtype, dk):
    """A NaN gate reaches the gradients of its own sequence and head, as it reaches the forward pass's outputs, and no others."""
    x = make(85, 1, 0, 2, dk, 64, dtype, True, 0.1, lengths=[70, 90])
    cot = SY.make_cotangents(x, 86)
    want = gpu_bwd(x, cot)
    x["g"][0, 100, 1, 7] = float("nan")   # token 30 of the second sequence
    got = gpu_bwd(x, cot)
    assert torch.isnan(got[3][0, 100, 1, 7]) and torch.isnan(got[5][1, 1, :, 7]).all()
    for n in (0, 1, 4):   # dq, dk, dbeta of the token and of those behind it in its chunk, whose states are NaN
        rows = got[n][0, 100:134, 1]
        assert torch.isnan(rows).all(), NAMES[n]
    for n, (a, b) in enumerate(zip(want, got)):
        if n == 5:
            assert torch.equal(a[0], b[0]) and torch.equal(a[1, 0], b[1, 0])
        else:
            assert torch.equal(a[:, :70], b[:, :70]) and torch.equal(a[:, :, 0], b[:, :, 0])


STRONG = [   # the tokens of every chunk of 64 that decay strongly, and their log decay; the others' is between -0.02 and 0
    (range(0, 32), -20.0), (range(0, 48), -60.0), (range(0, 32), -104.0), (range(0, 40), -104.0),   # up to a block border, into a block
    ([r for r in range(64) if r % 16 < 12], -104.0),           # the first twelve of every block of 16
    ([r for r in range(64) if not 5 <= r % 16 < 11], -90.0),   # both ends of every block
    (range(3, 64, 8), -104.0), (range(0, 64, 21), -1e4), (range(1, 64, 9), float("-inf")),   # resets
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dk,dv", [("f32", 128, 64), ("bf16", 128, 128), ("bf16", 64, 64)])
@pytest.mark.parametrize("rows,g", STRONG)
def test_mild_tokens_among_strong_ones(rows, g, dtype, dk, dv):
    """What passes between two tokens depends on the decays between them alone, however large the sum before them is."""
    x = make(81, 1, 150, 2, dk, dv, dtype, True, 0.01)
    gen = torch.Generator().manual_seed(82)
    x["g"] = -0.02 * torch.rand(x["g"].shape, generator=gen)
    for r in rows:
        x["g"][:, r::64] = g
    check(x, SY.make_cotangents(x, 83))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [16, 31, 48])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype,dk,dv", [(t, dk, dv) for t in ("f32", "bf16") for dk in (64, 128) for dv in (64, 128)])
def test_part_of_a_chunk_in_every_instance(dtype, dk, dv, grad, T):
    """Chunks that end at or inside a block of 16 rows, through every instance of the chunk kernel; each of those keeps many sums in
    registers, and a build that spilled hundreds of them once had the last rows of such a chunk wrong."""
    if grad == torch.bfloat16 and dtype == "f32":
        with pytest.raises(gb.GDNError):
            gb.gdn_kda_chunk_bwd(*(torch.zeros(1, T, 1, d, device="cuda") for d in (dk, dk, dv, dk)), torch.zeros(1, T, 1, device="cuda"),
                                 torch.zeros(1, T, 1, dv, device="cuda"), grad_dtype=grad)
        return
    x = make(91 + T, 1, T, 2, dk, dv, dtype, True, 0.1)
    cot = SY.make_cotangents(x, 92)
    check(x, cot)
    a, b = gpu_bwd(x, cot, grad_dtype=torch.float32), gpu_bwd(x, cot, grad_dtype=grad)
    assert all(torch.equal(p.to(q.dtype), q) for p, q in zip(a, b))


@pytest.mark.gpu
def test_gradients_match_differences_below_zero_gates():
    """As test_gradients_match_differences_of_the_forward_pass, along the gates alone, from -0.05 - 0.1 softplus: a step of 1e-2
    times 0.3 |e|, |e| < 5, stays below zero on both sides. The same bound on the difference."""
    x = make(57, 1, 130, 1, 64, 64, "f32", True, 0.1)
    x["g"] = x["g"] - 0.05
    cot = SY.make_cotangents(x, 58)
    dg = gpu_bwd(x, cot)[3]
    d = {n: x[n].cuda() for n in ("q", "k", "v", "g", "beta", "h0")}
    do, dhT = cot["do"].cuda().double(), cot["dhT"].cuda().double()

    def loss(g):
        assert float(g.max()) < 0
        o, hT = gb.gdn_kda_chunk_fwd(d["q"], d["k"], d["v"], g, d["beta"], d["h0"])
        return float((o.double() * do).sum() + (hT.double() * dhT).sum())

    e = -0.3 * torch.randn(d["g"].shape, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").abs()
    h = 1e-2
    along, diff = float((dg.double() * e.double()).sum()), (loss(d["g"] + h * e) - loss(d["g"] - h * e)) / (2 * h)
    print(along, diff, flush=True)
    assert abs(along - diff) <= 0.02 * max(10.0, abs(along))
