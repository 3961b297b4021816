"""gdn_scan_fwd / gdn_scan_bwd / gdn_scan_update over many tokens of slow gates: errors that may not grow with the length.

Tolerances (u = 2^-24, half a step of fp32). A map of many tokens, h -> h - K h + H, has K = 1 - exp(G) from the sum G of their gates: at most 20
additions one after another (4 tokens, 8 groups, 8 waves), then a series of nine steps: K is off by 32 u of itself, H (four steps of a gate
that is off by 16 u of itself, then maps as above) by 64 u K |x|.

A constant state (h0 = x = c, blended) is pulled back to c (1 + 96 u) at most by every map, and the rounding of a map's two
sums moves it by 2 u |c| at most on the way from one to the next; one never leaves the band in which the pull is below half a step, so at most 17 maps
(8 groups, 8 waves, the tile) add theirs to the band, and 4 tokens, whose factor is an exponential off by 2 u, 4 u each: |h - c| <=
(96 + 34 + 16) u |c|, whatever the length. On a pool there are no maps: 3 u more than
the band of one token's own errors, 12 u for k and 16 u for the input times k.

A decaying state (x = 0, h0 = 1) or gradient (dh = 0, dhT = 1) after n tiles with decay e^G: 2 u a tile for its sums, 32 u |G| for the tiles' K, 42 u inside the
tile: |h / e^G - 1| <= (2 n + 32 |G| + 42 + 4 * 3) u; dx = k D and dg = E h add 16 u for k and a product each.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_42_amd import binding as gb

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LONG = 32768


def cut(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


def gates(D, seed):
    """A gate per channel, from far below fp32's step at 1 to 1e-3, where the exponential's rounding goes either way."""
    gen = torch.Generator().manual_seed(seed)
    g = -torch.exp(torch.empty(D).uniform_(np.log(1e-8), np.log(1e-3), generator=gen))
    g[:4] = torch.tensor([-1e-6, -1e-7, -2e-8, -3e-6])
    return g


FORMS = [
    # T, cu: dense; packed; tiles of 32 tokens; walked by one work-group
    (LONG, None), (LONG, [0, 5, 5, LONG]), (LONG, [0] * 300 + [LONG]), (512, None),
]


@pytest.mark.parametrize("T,cu", FORMS)
def test_a_constant_stays(T, cu):
    print(f"[gpu] scan constant T={T} sequences {1 if cu is None else len(cu) - 1}", flush=True)
    D, N = 72, 1 if cu is None else len(cu) - 1
    gen = torch.Generator().manual_seed(T + N)
    c = (1 + torch.rand(D, generator=gen)) * torch.where(torch.rand(D, generator=gen) < 0.5, -1.0, 1.0)
    c[:4] = 1.0
    x, g = c.expand(1, T, D).contiguous().cuda(), gates(D, 1).expand(1, T, D).contiguous().cuda()
    h, hT, car = gb.gdn_scan_fwd(x, g, c.expand(N, D).contiguous().cuda(), cut(cu), blend=True, keep_carries=True)
    rel = lambda a: float(((a - c.cuda()) / c.cuda()).abs().max()) / U  # noqa: E731
    print(f"      off by {rel(h):.1f} u, final states {rel(hT):.1f} u", flush=True)
    assert rel(h) <= 146 and rel(hT) <= 146
    # the gradient of a gate is E (h - x), which is rounding alone here
    dx, dg, dh0 = gb.gdn_scan_bwd(x, g, torch.zeros_like(x), car, torch.ones(N, D, device="cuda"), cut(cu), blend=True)
    assert float(dg.abs().max()) <= 2 * 146 * U * 2


def test_a_constant_stays_on_a_pool():
    """5000 calls of one token, then runs."""
    D = 72
    c = 1 + torch.rand(D, generator=torch.Generator().manual_seed(3)).cuda()
    g = gates(D, 2).cuda()
    pool, slot = c[None].clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    x1, g1 = c[None].contiguous(), g[None].contiguous()
    for _ in range(5000):
        gb.gdn_scan_update(x1, g1, pool, slot, blend=True)
    T = 20000
    gb.gdn_scan_update(c.expand(T, D).contiguous(), g.expand(T, D).contiguous(), pool, slot, cut([0, T]), blend=True)
    off = float(((pool[0] - c) / c).abs().max()) / U
    print(f"      off by {off:.1f} u", flush=True)
    assert off <= 31


@pytest.mark.parametrize("T,cu", FORMS)
@pytest.mark.parametrize("blend", [False, True])
def test_slow_decays(T, cu, blend):
    print(f"[gpu] scan decays T={T} sequences {1 if cu is None else len(cu) - 1} blend={blend}", flush=True)
    D, N = 72, 1 if cu is None else len(cu) - 1
    g1 = gates(D, 4)
    x, g = torch.zeros(1, T, D, device="cuda"), g1.expand(1, T, D).contiguous().cuda()
    one = torch.ones(N, D, device="cuda")
    h, hT, car = gb.gdn_scan_fwd(x, g, one, cut(cu), blend=blend, keep_carries=True)
    dx, dg, dh0 = gb.gdn_scan_bwd(x, g, x, car, one, cut(cu), blend=blend)
    begin = 0 if cu is None else cu[-2]   # of the last sequence, the long one
    n = T - begin
    G1 = g1.double().numpy()
    t = np.arange(n)[:, None]
    tiles = np.ceil(n / (32 if N > 200 else 256))

    def near(got, ref, more, name):
        got = got.double().cpu().numpy()
        Gs = np.abs(np.log(np.abs(ref[0])))
        off = np.abs(got / ref[0] - 1) / U
        tol = 2 * tiles + 32 * Gs + 54 + more
        print(f"      {name}: off by {off.max():.1f} u, {float((off / tol).max()):.3f} of the tolerance", flush=True)
        assert (off <= tol).all(), name

    near(h[0, begin:], (np.exp(G1 * (t + 1)),), 0, "h")
    near(hT[-1], (np.exp(G1 * n),), 0, "hT")
    near(dh0[-1], (np.exp(G1 * n),), 0, "dh0")
    D_ = np.exp(G1 * (n - 1 - t))
    got = dx[0, begin:].double().cpu().numpy() / (-np.expm1(G1) if blend else 1.0)
    off = np.abs(got / D_ - 1) / U
    assert (off <= 2 * tiles + 32 * np.abs(G1 * (n - 1 - t)) + 54 + 16).all(), "dx"
    want = np.exp(G1 * n) * np.ones((n, 1))   # E_t h_{t-1}: the decay of the whole sequence, wherever it is cut
    off = np.abs(dg[0, begin:].double().cpu().numpy() / want - 1) / U
    print(f"      dg: off by {off.max():.1f} u", flush=True)
    assert (off <= 2 * (2 * tiles + 32 * np.abs(G1 * n) + 54 + 16)).all(), "dg"


@pytest.mark.parametrize("T,cu", [(1500, None), (2000, [0, 700, 1400, 2000]), (500, None)])
@pytest.mark.parametrize("blend", [False, True])
def test_infinities_stay_with_their_channel_and_sequence(T, cu, blend):
    """An infinite input leaves no finite state behind it in its sequence, an infinite gradient none before it; every other channel and
    sequence has the bits that it has without them."""
    print(f"[gpu] scan infinities T={T} cu={cu} blend={blend}", flush=True)
    D, N, t = 72, 1 if cu is None else len(cu) - 1, 450 if cu is None else 850
    gen = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, g, h0, dh, dhT = r(1, T, D), -r(1, T, D).square() * gates(D, 6).abs().cuda() * 300, r(N, D), r(1, T, D), r(N, D)

    def run():
        h, hT, car = gb.gdn_scan_fwd(x, g, h0, cut(cu), blend=blend, keep_carries=True)
        return h, hT, *gb.gdn_scan_bwd(x, g, dh, car, dhT, cut(cu), blend=blend)

    h, hT, dx, dg, dh0 = run()
    assert all(torch.isfinite(a).all() for a in (h, hT, dx, dg, dh0))
    x[0, t, 5], dh[0, t, 9] = float("inf"), -float("inf")
    h2, hT2, dx2, dg2, dh02 = run()
    n, lo, hi = (0, 0, T) if cu is None else (1, 700, 1400)
    bad, back = torch.zeros(T, D, dtype=torch.bool, device="cuda"), torch.zeros(T, D, dtype=torch.bool, device="cuda")
    bad[t:hi, 5], back[lo:t + 1, 9] = True, True
    assert torch.equal(~torch.isfinite(h2[0]), bad) and torch.equal(h2[0][~bad], h[0][~bad])
    assert torch.equal(~torch.isfinite(dx2[0]), back) and torch.equal(dx2[0][~back], dx[0][~back])
    last, first = torch.zeros(N, D, dtype=torch.bool, device="cuda"), torch.zeros(N, D, dtype=torch.bool, device="cuda")
    last[n, 5], first[n, 9] = True, True
    assert torch.equal(~torch.isfinite(hT2), last) and torch.equal(hT2[~last], hT[~last])
    assert torch.equal(~torch.isfinite(dh02), first) and torch.equal(dh02[~first], dh0[~first])
    assert not torch.isfinite(dg2[0][back]).any() and torch.equal(dg2[0, :, [4, 6, 8, 10]], dg[0, :, [4, 6, 8, 10]])
