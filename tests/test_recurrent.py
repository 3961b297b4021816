"""gdn_recurrent_fwd: refusals (CPU) and the kernel against the fp64 oracle (GPU).

Tolerance: all arithmetic is fp32 (u = 2^-24). Per token a state entry takes a decay (exp and product, about 4 u), the sum s . k of
dk terms (dk / 16 serial additions and 4 tree levels, at most 13 u of the sum of magnitudes) and the update (3 u); keys are unit
vectors and decays at most 1, so errors do not grow: T tokens leave at most about 24 T u of the largest magnitude, 7e-5
for the longest run here (48). The comparison takes 1e-4 of the largest reference magnitude, as the fp32 forward
pass does, and a bf16 o half a step, 2^-8 of its value, more.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_42_amd import binding as gb
from oracle import pool as PO

P = 1 << 12


def c_call(**kw):
    a = dict(q=P, k=P, v=P, g=P, beta=P, states=P, slots=P, cu=P, out=None, o=P, T=4, N=2, H=2, HV=4, dk=64, dv=64, ns=8, qs=128,
             ks=128, vs=256, cg=0, dtype=1, od=1)
    a.update(kw)
    return gb.lib().gdn_recurrent_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), -3), (dict(od=-1), -3), (dict(dk=32), -5), (dict(dv=96), -5), (dict(N=-1), -2), (dict(T=-1), -2),
    (dict(H=0), -2), (dict(HV=3), -2), (dict(HV=1), -2), (dict(ns=-1), -2), (dict(cu=None), -2), (dict(N=1 << 19), -2),
    (dict(qs=-8), -2), (dict(q=None), -1), (dict(v=None), -1), (dict(g=None), -1), (dict(beta=None), -1), (dict(states=None), -1),
    (dict(slots=None), -1), (dict(o=None), -1), (dict(q=P + 8), -4), (dict(states=P + 4), -4), (dict(g=P + 2), -4),
    (dict(g=P + 4, cg=1), -4), (dict(slots=P + 1), -4), (dict(out=P + 2), -4), (dict(ks=129), -4), (dict(vs=4), -4),
])
def test_refuses(kw, status):
    assert c_call(**kw) == status


def test_nothing_to_do_is_ok():
    assert c_call(T=0, q=None, o=None, states=None) == 0
    assert c_call(N=0, T=0, cu=None) == 0


def test_binding_refuses_on_the_host():
    m = lambda *s, dt=torch.float32: torch.empty(*s, device="meta", dtype=dt)  # noqa: E731
    i32 = torch.int32
    good = dict(q=m(4, 2, 64), k=m(4, 2, 64), v=m(4, 4, 64), g=m(4, 4), beta=m(4, 4), states=m(8, 4, 64, 64),
                slots=m(2, dt=i32), cu_seqlens=m(3, dt=i32))
    for change, text in ((dict(v=m(4, 3, 64)), "multiple"), (dict(k=m(4, 1, 64)), "k has shape"), (dict(g=m(4, 2)), "g has shape"),
                         (dict(states=m(8, 2, 64, 64)), "states has shape"), (dict(slots=m(2, dt=torch.int64)), "slots must"),
                         (dict(cu_seqlens=None), "without cu_seqlens"), (dict(cu_seqlens=m(4, dt=i32)), "cu_seqlens has"),
                         (dict(out_slots=m(3, dt=i32)), "out_slots has"), (dict(), "on a GPU")):
        with pytest.raises(ValueError, match=text):
            gb.gdn_recurrent_fwd(**{**good, **change})


def make(seed, lens, H, HV, dk, dv, dtype, channels, n_slots, extra=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T = sum(lens) + extra
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=unit(r(T, H, dk)).to(dt), k=unit(r(T, H, dk)).to(dt), v=r(T, HV, dv).to(dt),
             g=-torch.nn.functional.softplus(r(T, HV, dk) if channels else r(T, HV)) * torch.rand(1, generator=gen),
             beta=torch.sigmoid(r(T, HV)) * 1.5, states=r(n_slots, HV, dv, dk),
             cu=torch.tensor([0, *lens]).cumsum(0).to(torch.int32))
    x["order"] = torch.randperm(n_slots, generator=gen).to(torch.int32)
    return x


def check(o, states, o_ref, s_ref, what=""):
    o, s = o.cpu(), states.cpu().double().numpy()
    half = 2.0 ** -8 * (1 + 2.0 ** -8) if o.dtype == torch.bfloat16 else 0.0
    o = o.double().numpy()
    cover = ~np.isnan(o_ref)
    scale = max(1e-30, np.abs(o_ref[cover]).max()) if cover.any() else 0.0
    eo = (np.abs(o - o_ref) - half * np.abs(o_ref))[cover].max() if cover.any() else 0.0
    es = np.abs(s - s_ref).max() / np.abs(s_ref).max()
    print(f"      {what} err(o)={eo:.2e} of {scale:.2e}, err(states)={es:.2e}", flush=True)
    assert eo <= 1e-4 * scale and es <= 1e-4
    return o


CASES = [
    # lens, H, HV, dk, dv, dtype, channels
    ([1], 1, 1, 64, 64, "f32", False),
    ([1], 4, 8, 128, 128, "bf16", True),
    ([1, 0, 3, 48, 0], 2, 2, 128, 128, "bf16", False),
    ([0, 7, 2], 2, 6, 64, 128, "f32", True),
    ([5] * 9, 1, 3, 128, 64, "bf16", True),
    ([1] * 70, 4, 32, 128, 128, "bf16", False),
    ([3, 1] * 40, 16, 32, 64, 64, "bf16", True),
    ([17], 1, 2, 128, 128, "f32", False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,HV,dk,dv,dtype,channels", CASES)
@pytest.mark.parametrize("mode", ["last", "every", "padded"])
def test_against_oracle(lens, H, HV, dk, dv, dtype, channels, mode):
    print(f"[gpu] recurrent lens={lens[:6]}x{len(lens)} H={H} HV={HV} {dk}x{dv} {dtype} channels={channels} {mode}", flush=True)
    N, T = len(lens), sum(lens)
    ns = N + T + 3
    x = make(N * 31 + T, lens, H, HV, dk, dv, dtype, channels, ns, extra=2)   # two rows behind the last sequence
    slots = x["order"][:N].clone()
    out = None
    if mode == "every":
        out = torch.cat([x["order"][N:N + T], torch.tensor([-1, ns], dtype=torch.int32)])
        out[T // 2] = -1   # a state that is not kept
    if mode == "padded":
        slots[::2] = torch.tensor([-1, ns, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).repeat(N)[: len(slots[::2])]
    d = {n: t.cuda() for n, t in x.items()}
    for od in (torch.float32, torch.bfloat16):
        states = d["states"].clone()
        o = torch.full((T + 2, HV, dv), 7.0, dtype=od, device="cuda")
        gb.gdn_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], states, slots.cuda(), d["cu"],
                             None if out is None else out.cuda(), o)
        o_ref, s_ref = PO.run(x["q"], x["k"], x["v"], x["g"], x["beta"], x["states"], slots, x["cu"],
                              None if out is None else out.numpy())
        check(o, states, o_ref, s_ref, str(od))
        assert (o[T:] == 7).all()   # rows that no sequence covers
        untouched = np.setdiff1d(np.arange(ns), (slots if out is None else out).numpy())
        assert torch.equal(states.cpu()[untouched], x["states"][untouched])


@pytest.mark.gpu
def test_single_tokens_without_offsets_and_strided_views():
    """One token per sequence without cu_seqlens; q, k and v as views of one convolution output."""
    x = make(3, [1] * 6, 2, 4, 64, 128, "bf16", False, 10)
    d = {n: t.cuda() for n, t in x.items()}
    slots = d["order"][:6].contiguous()
    a, b = d["states"].clone(), d["states"].clone()
    o1 = gb.gdn_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], a, slots, d["cu"])
    f = torch.cat([d["q"].flatten(1), d["k"].flatten(1), d["v"].flatten(1), torch.zeros(6, 8, device="cuda", dtype=torch.bfloat16)], 1)
    q, k, v = f[:, :128].unflatten(1, (2, 64)), f[:, 128:256].unflatten(1, (2, 64)), f[:, 256:768].unflatten(1, (4, 128))
    o2 = gb.gdn_recurrent_fwd(q, k, v, d["g"], d["beta"], b, slots)
    assert torch.equal(o1, o2) and torch.equal(a, b)
    with pytest.raises(ValueError, match="follow each other"):
        gb.gdn_recurrent_fwd(d["q"], d["k"], torch.zeros(6, 4, 256, device="cuda", dtype=torch.bfloat16)[..., :128], d["g"], d["beta"], b, slots)


@pytest.mark.gpu
@pytest.mark.parametrize("channels", [False, True])
def test_matches_decode_step(channels):
    """A dense batch of single tokens is the decode step on the same states."""
    x = make(8, [1] * 5, 3, 3, 128, 128, "bf16", channels, 5)
    d = {n: t.cuda() for n, t in x.items()}
    a, b = d["states"].clone(), d["states"].clone()
    o1 = gb.gdn_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], a, torch.arange(5, dtype=torch.int32, device="cuda"))
    step = gb.gdn_kda_decode_step if channels else gb.gdn_decode_step
    o2 = step(d["q"], d["k"], d["v"], d["g"], d["beta"], b)
    # the two order the decay and the products differently: a few u of the largest magnitude
    assert (o1 - o2).abs().max() <= 64 * 2.0 ** -24 * o2.abs().max()
    assert (a - b).abs().max() <= 64 * 2.0 ** -24 * b.abs().max()


@pytest.mark.gpu
def test_split_runs_and_draft_rollback():
    """A run in one call equals the same run in two; a kept draft state continues like the run that ends there."""
    x = make(4, [9], 2, 4, 128, 128, "f32", True, 12)
    d = {n: t.cuda() for n, t in x.items()}
    i32 = dict(dtype=torch.int32, device="cuda")
    s0 = torch.zeros(1, **i32)
    args = lambda a, b: [d[n][a:b] for n in ("q", "k", "v", "g", "beta")]  # noqa: E731
    cu = lambda n: torch.tensor([0, n], **i32)  # noqa: E731
    a, b, c = (d["states"].clone() for _ in range(3))
    oa = gb.gdn_recurrent_fwd(*args(0, 9), a, s0, cu(9))
    ob = torch.cat([gb.gdn_recurrent_fwd(*args(0, 4), b, s0, cu(4)), gb.gdn_recurrent_fwd(*args(4, 9), b, s0, cu(5))])
    assert torch.equal(oa, ob) and torch.equal(a[0], b[0])
    out = torch.arange(2, 8, **i32)   # six draft tokens, each state kept; four are accepted
    gb.gdn_recurrent_fwd(*args(0, 6), c, s0, cu(6), out)
    assert torch.equal(c[0], d["states"][0])
    oc = gb.gdn_recurrent_fwd(*args(4, 9), c, out[3:4].contiguous(), cu(5))
    assert torch.equal(oc, oa[4:]) and torch.equal(c[5], a[0])
    own = torch.zeros(1, **i32)       # a sequence may name its own slot
    e, f = d["states"].clone(), d["states"].clone()
    gb.gdn_recurrent_fwd(*args(0, 1), e, s0, cu(1), own)
    gb.gdn_recurrent_fwd(*args(0, 1), f, s0, cu(1))
    assert torch.equal(e, f)


@pytest.mark.gpu
def test_bad_offsets_stay_inside():
    """Offsets that fall or leave [0, T] are clamped."""
    x = make(6, [4, 4], 1, 2, 64, 64, "bf16", False, 4)
    d = {n: t.cuda() for n, t in x.items()}
    states = d["states"].clone()
    cu = torch.tensor([-5, 6, 3, 2000000000], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    o = gb.gdn_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], states, slots, cu)
    o_ref, s_ref = PO.run(x["q"], x["k"], x["v"], x["g"], x["beta"], x["states"], [0, 2], [0, 6, 8])
    _, s_tail = PO.run(x["q"][3:], x["k"][3:], x["v"][3:], x["g"][3:], x["beta"][3:], x["states"], [2], [0, 5])
    s = states.cpu().double().numpy()
    assert np.abs(s[0] - s_ref[0]).max() <= 1e-4 * np.abs(s_ref[0]).max()
    assert np.abs(s[2] - s_tail[2]).max() <= 1e-4 * np.abs(s_tail[2]).max()
    assert torch.equal(states[1], d["states"][1]) and torch.equal(states[3], d["states"][3])
    assert torch.isfinite(o).all()


@pytest.mark.gpu
def test_graph_replay_streams_and_repeats():
    """A captured step replayed between eager ones on the same pool; another stream; the same bits every time."""
    x = make(12, [2, 1, 4], 2, 4, 128, 128, "bf16", True, 6)
    d = {n: t.cuda() for n, t in x.items()}
    slots = d["order"][:3].contiguous()
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    want = d["states"].clone()
    outs = [gb.gdn_recurrent_fwd(*args, want, slots, d["cu"]) for _ in range(6)]
    torch.cuda.synchronize()
    states = d["states"].clone()
    o = torch.empty_like(outs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gb.gdn_recurrent_fwd(*args, states, slots, d["cu"], o=o)
    states.copy_(d["states"])
    for i in range(6):
        if i % 2:
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, outs[i])
        else:
            assert torch.equal(gb.gdn_recurrent_fwd(*args, states, slots, d["cu"]), outs[i])
    assert torch.equal(states, want)
    side = torch.cuda.Stream()
    states.copy_(d["states"])
    side.wait_stream(torch.cuda.current_stream())
    got = gb.gdn_recurrent_fwd(*args, states, slots, d["cu"], stream=side)
    side.synchronize()
    assert torch.equal(got, outs[0])


@pytest.mark.gpu
def test_pool_past_32_bits():
    """A slot whose elements start past 2^31 (a pool of 8.8 GB)."""
    x = make(21, [2, 1], 16, 32, 128, 128, "bf16", False, 3)
    d = {n: t.cuda() for n, t in x.items()}
    pool = torch.zeros(4200, 32, 128, 128, device="cuda")
    slots, out = [4199, 4100], [4150, -1, 4198]
    pool[slots] = d["states"][:2]
    i32 = dict(dtype=torch.int32, device="cuda")
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    o = gb.gdn_recurrent_fwd(*args, pool, torch.tensor(slots, **i32), d["cu"], torch.tensor(out, **i32))
    o_ref, s_ref = PO.run(x["q"], x["k"], x["v"], x["g"], x["beta"], x["states"], [0, 1], x["cu"], [0, -1, 1])
    assert np.abs(o.cpu().double().numpy() - o_ref).max() <= 1e-4 * np.abs(o_ref).max()
    for slot, ref in ((4150, 0), (4198, 1)):
        assert np.abs(pool[slot].cpu().double().numpy() - s_ref[ref]).max() <= 1e-4 * np.abs(s_ref[ref]).max()
    assert torch.equal(pool[4199], d["states"][0]) and float(pool[:4100].abs().max()) == 0.0


@pytest.mark.gpu
def test_debug_check_allows_padding(monkeypatch):
    """GDN_CHECK=1 accepts tokens behind the last sequence and refuses falling offsets."""
    x = make(22, [2, 1], 1, 1, 64, 64, "f32", False, 3, extra=2)
    d = {n: t.cuda() for n, t in x.items()}
    monkeypatch.setenv("GDN_CHECK", "1")
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    slots = d["order"][:2].contiguous()
    gb.gdn_recurrent_fwd(*args, d["states"], slots, d["cu"])
    for cu in ([0, 3, 2], [0, 2, 6], [1, 2, 3]):
        with pytest.raises(gb.GDNError):
            gb.gdn_recurrent_fwd(*args, d["states"], slots, torch.tensor(cu, dtype=torch.int32, device="cuda"))


UNEVEN = [   # few more tokens than sequences: runs of several tokens on the single-token kernel
    ([1] * 30 + [9, 0] + [1] * 8, 2, 4, 128, 128, "bf16", False),
    ([1] * 5 + [4] + [1] * 25 + [2, 1, 3], 1, 3, 64, 128, "f32", True),
    ([1] * 80 + [17], 2, 2, 128, 64, "f32", False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,HV,dk,dv,dtype,channels", UNEVEN)
@pytest.mark.parametrize("mode", ["last", "every", "padded"])
def test_single_tokens_beside_a_run(lens, H, HV, dk, dv, dtype, channels, mode):
    assert sum(lens) + 2 <= len(lens) + len(lens) // 4   # (two rows behind the last sequence)
    test_against_oracle(lens, H, HV, dk, dv, dtype, channels, mode)


@pytest.mark.gpu
@pytest.mark.parametrize("N,H,HV,dk,dv,dtype,channels", [
    (128, 8, 32, 128, 128, "bf16", False), (128, 16, 32, 64, 128, "f32", True),       # four rows per lane group
    (129, 16, 64, 64, 64, "bf16", True), (130, 16, 64, 128, 64, "f32", False),
    (33, 8, 32, 128, 128, "f32", True), (70, 4, 32, 64, 64, "bf16", False)])          # two
def test_many_runs(N, H, HV, dk, dv, dtype, channels):
    """Batches for which a lane group takes several state rows."""
    print(f"[gpu] recurrent N={N} H={H} HV={HV} {dk}x{dv} {dtype} channels={channels}", flush=True)
    lens = [(2, 1, 3, 0, 4)[n % 5] for n in range(N)]
    x = make(N + dk, lens, H, HV, dk, dv, dtype, channels, N + 2)
    d = {n: t.cuda() for n, t in x.items()}
    slots = d["order"][:N].contiguous()
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    a, b = d["states"].clone(), d["states"].clone()
    o = gb.gdn_recurrent_fwd(*args, a, slots, d["cu"])
    check(o, a, *PO.run(*(x[n] for n in ("q", "k", "v", "g", "beta", "states")), slots.cpu(), x["cu"]))
    own = torch.full((sum(lens),), -1, dtype=torch.int32, device="cuda")   # the last token's state to the sequence's own slot
    for n in range(N):
        if lens[n]:
            own[int(x["cu"][n + 1]) - 1] = slots[n]
    assert torch.equal(gb.gdn_recurrent_fwd(*args, b, slots, d["cu"], own), o) and torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1, 1, 1, 1], [5, 20, 3, 2]])
@pytest.mark.parametrize("channels", [False, True])
def test_nan_and_infinite_gates(lens, channels):
    """A gate of -infinity forgets the state; NaN stays with its sequence and head; a padded entry reads nothing."""
    x = make(14, lens, 2, 4, 128, 128, "f32", channels, 6)
    cu = x["cu"].tolist()
    d = {n: t.cuda() for n, t in x.items()}
    slots = d["order"][:4].contiguous()
    run = lambda states, sl: gb.gdn_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], states, sl, d["cu"])  # noqa: E731
    s0 = d["states"].clone()
    want = run(s0, slots)
    d["g"][cu[0]] = float("-inf")
    a, b = d["states"].clone(), d["states"].clone()
    b[slots[0].item()] = 0
    oa, ob = run(a, slots), run(b, slots)
    assert torch.equal(oa, ob) and torch.equal(a, b) and torch.isfinite(oa).all()
    d["v"][cu[1], 1] = float("nan")   # one value head of sequence 1
    for t in (d["q"], d["k"], d["v"], d["g"], d["beta"]):
        t[cu[2]:cu[3]] = float("nan")   # all of sequence 2
    slots[2] = -1
    c = d["states"].clone()
    oc = run(c, slots)
    assert torch.isnan(oc[cu[1]:cu[2], 1]).all() and torch.isnan(c[slots[1].item(), 1]).all()
    assert (oc[cu[2]:cu[3]] == 0).all()
    others = [0, 2, 3]
    assert torch.equal(oc[cu[1]:cu[2]][:, others], want[cu[1]:cu[2]][:, others])
    assert torch.equal(c[slots[1].item()][others], s0[slots[1].item()][others])
    assert torch.equal(oc[cu[3]:], want[cu[3]:]) and torch.equal(oc[:cu[1]], oa[:cu[1]])
