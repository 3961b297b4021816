"""gdn_scan_fwd / gdn_scan_bwd on workspaces that hold what an earlier call could have left, and on inputs that change from call to call: what
passes between work-groups has to be this call's. The reference is the same call with a workspace of its own; bits do not depend on either.
Then the instances for large calls, against the oracle in sampled channels (tolerances: oracle/scan.py)."""
import numpy as np
import pytest
import torch

from gated_delta_rule_42_amd import binding as gb
from oracle import scan as SC

pytestmark = pytest.mark.gpu
SEQS = [
    # B, T, cu: tiles of 256 tokens, dense and packed, and of 32 (packed), all of them passed on between work-groups
    (2, 1500, None), (1, 3000, [0, 700, 703, 2990]), (1, 1300, [0] * 10 + [1, 1300]), (1, 2400, [*range(0, 1900, 50), 1900, 2380]),
]


def inputs(seed, B, T, N, D, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    rate = torch.exp(torch.empty(D, device="cuda").uniform_(-6.0, 0.5, generator=gen))
    return dict(x=r(B, T, D).to(dtype), g=-rate * torch.nn.functional.softplus(r(B, T, D)), h0=r(N, D), dh=r(B, T, D).to(dtype), dhT=r(N, D))


def cut(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


def covered(B, T, cu):
    return slice(0, T if cu is None else cu[-1])


def both(t, c, blend, ws=(None, None)):
    # a workspace given or the operator's own; outputs over a known ground, so that rows that no sequence covers compare too
    h = torch.zeros_like(t["x"])
    _, hT, car = gb.gdn_scan_fwd(t["x"], t["g"], t["h0"], c, blend=blend, h=h, keep_carries=True, workspace=ws[0])
    dx, dg, dh0 = gb.gdn_scan_bwd(t["x"], t["g"], t["dh"], car, t["dhT"], c, blend=blend, workspace=ws[1])
    return h, hT, dx, dg, dh0


def same(a, b, rows):
    return all(torch.equal(p[:, rows] if p.dim() == 3 else p, q[:, rows] if q.dim() == 3 else q) for p, q in zip(a, b))


@pytest.mark.parametrize("B,T,cu", SEQS)
@pytest.mark.parametrize("blend", [False, True])
def test_dirty_workspaces(B, T, cu, blend):
    """Workspaces full of numbers that would pass for maps and states, and of what a call on other inputs left."""
    D, N = 136, B if cu is None else len(cu) - 1
    print(f"[gpu] scan workspace B={B} T={T} N={N} blend={blend}", flush=True)
    c, rows = cut(cu), covered(B, T, cu)
    size = gb.gdn_scan_workspace_bytes(B, T, N, D, cu is not None)
    assert size > 0 and size % 4 == 0
    sets = [inputs(10 + i, B, T, N, D) for i in range(3)]
    want = [both(t, c, blend) for t in sets]
    assert not same(want[0], want[1], rows)
    for word in (0x3F800000, 0, 0x3E000000, -1):   # 1, 0, 1/8, and the mark itself
        ws = [torch.full((size // 4,), word, dtype=torch.int32, device="cuda") for _ in range(2)]
        assert same(both(sets[0], c, blend, ws), want[0], rows), hex(word)
        for i in (1, 2, 0, 0):   # the same workspaces, and for the backward pass the forward one's
            assert same(both(sets[i], c, blend, ws), want[i], rows), (hex(word), i)
            assert same(both(sets[i], c, blend, ws[::-1]), want[i], rows), (hex(word), i)


@pytest.mark.parametrize("B,T,cu", SEQS)
def test_replays_on_changed_inputs(B, T, cu):
    """A captured pass of both directions replayed on new inputs, with eager passes between the replays."""
    D, N = 136, B if cu is None else len(cu) - 1
    print(f"[gpu] scan replay B={B} T={T} N={N}", flush=True)
    c, rows = cut(cu), covered(B, T, cu)
    sets = [inputs(20 + i, B, T, N, D) for i in range(3)]
    want = [both(t, c, True) for t in sets]
    held = {n: a.clone() for n, a in sets[0].items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(held, c, True)
    for i in (0, 1, 2, 1, 0):
        for n in held:
            held[n].copy_(sets[i][n])
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want[i], rows), i
        assert same(both(sets[2 - i], c, True), want[2 - i], rows), i


def inside(got, ref, tol, name):
    full = got.cpu().double().numpy()
    step = 2.0 ** -8 * (1 + 2.0 ** -8) if got.dtype == torch.bfloat16 else 2.0 ** -24
    over = np.abs(full - ref) / (tol + step * np.abs(ref))
    print(f"      {name}: largest error over its tolerance {over.max():.3f}", flush=True)
    assert (over <= 1).all(), name


@pytest.mark.parametrize("dtype,h_dtype", [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "float32")])
@pytest.mark.parametrize("blend", [False, True])
@pytest.mark.parametrize("tiles", [256, 32])
def test_large_calls(dtype, h_dtype, blend, tiles):
    """Outputs past the caches, in every type and form, and tiles of 32 tokens of as large a call."""
    D = 3064
    B, T, cu = (2, 2100, None) if tiles == 256 else (1, 4000, [*range(0, 4000, 40), 4000])
    N = B if cu is None else len(cu) - 1
    print(f"[gpu] scan large tiles of {tiles} {dtype} h {h_dtype} blend={blend}", flush=True)
    hd = getattr(torch, h_dtype)
    t = inputs(7, B, T, N, D, getattr(torch, dtype))
    t["dh"] = t["dh"].to(hd)
    c = cut(cu)
    h, hT, car = gb.gdn_scan_fwd(t["x"], t["g"], t["h0"], c, blend=blend, out_dtype=hd, keep_carries=True)
    dx, dg, dh0 = gb.gdn_scan_bwd(t["x"], t["g"], t["dh"], car, t["dhT"], c, blend=blend)
    at = [0, 63, 64, 1000, 3063]
    s = {n: a[..., at].cpu() for n, a in t.items()}
    rh, rT, eh, eT = SC.forward(s["x"], s["g"], s["h0"], cu, blend)
    rx, rg, r0, ex, eg, e0 = SC.backward(s["x"], s["g"], s["h0"], s["dh"], s["dhT"], cu, blend)
    for got, ref, tol, name in ((h, rh, eh, "h"), (hT, rT, eT, "hT"), (dx, rx, ex, "dx"), (dg, rg, eg, "dg"), (dh0, r0, e0, "dh0")):
        inside(got[..., at], ref, tol, name)
