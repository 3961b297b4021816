"""The operators around the channel-wise rule together, as a layer uses them: fused projection -> norm and rotation of q and k ->
chunked forward -> gradients back to the projection; and a prompt whose state goes into a pool, continued token by token.

The reference is the token recurrence in fp64 with torch's autograd (no formula of the library's or the oracles'). Inputs are
fp32, and each stage is within 1e-4 of its largest output (see the operators' own tests); the norm's backward divides by
row norms near 1, so a chain of three stages is held to 3e-4 of the largest gradient.
"""
import pytest
import torch

from gated_delta_rule_42_amd import binding as gb

pytestmark = pytest.mark.gpu


def project(seed, B, T, H, d, dtype):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(x=r(B, T, 3 * H * d).to(dtype), g=-torch.nn.functional.softplus(r(B, T, H, d)) * 0.2,
                beta=torch.sigmoid(r(B, T, H)), h0=0.1 * r(B, H, d, d), qw=1 + 0.2 * r(d), kw=1 + 0.2 * r(d),
                pos=torch.randint(0, 100000, (B, 1), generator=gen, dtype=torch.int32) + torch.arange(T, dtype=torch.int32),
                freq=(1000.0 ** (-torch.arange(d // 4, dtype=torch.float64) / (d // 4))).float(),
                do=r(B, T, H, d).to(dtype), dhT=r(B, H, d, d))


def split(x, H, d):
    return [t.unflatten(-1, (H, d)) for t in x.split(H * d, -1)]


def reference(p, H, d):
    """Outputs and gradients of the loss sum(o do) + sum(hT dhT) in fp64 by autograd."""
    y = {n: t.double().clone().requires_grad_(n not in ("pos", "freq", "do", "dhT")) for n, t in p.items()}
    q, k, v = split(y["x"], H, d)
    ang = y["pos"][..., None, None] * y["freq"]
    cos, sin = torch.cos(ang), torch.sin(ang)

    def norm(t, w, scale):
        t = t * torch.rsqrt(t.square().sum(-1, keepdim=True) + 1e-6) * w
        h = d // 4
        a, b = t[..., :h], t[..., h:2 * h]
        return scale * torch.cat([a * cos - b * sin, b * cos + a * sin, t[..., 2 * h:]], -1)

    q, k = norm(q, y["qw"], d ** -0.5), norm(k, y["kw"], 1.0)
    S, o = y["h0"], []
    for t in range(q.shape[1]):
        Sa = S * y["g"][:, t].exp()[:, :, None, :]
        u = y["beta"][:, t][..., None] * (v[:, t] - (Sa @ k[:, t][..., None])[..., 0])
        S = Sa + u[..., None] * k[:, t][..., None, :]
        o.append((S @ q[:, t][..., None])[..., 0])
    o = torch.stack(o, 1)
    ((o * y["do"]).sum() + (S * y["dhT"]).sum()).backward()
    return o.detach(), S.detach(), {n: t.grad for n, t in y.items() if t.requires_grad}


def near(a, b, tol, name):
    err = float((a.cpu().double() - b).abs().max() / b.abs().max())
    print(f"      {name}: {err:.2e}", flush=True)
    assert err <= tol, name


def test_training_step():
    """Gradients land in one fused tensor, without a copy of q, k or v between the stages."""
    B, T, H, d = 2, 130, 2, 64
    p = project(1, B, T, H, d, torch.float32)
    o_ref, S_ref, g_ref = reference(p, H, d)
    t = {n: x.cuda() for n, x in p.items()}
    q, k, v = split(t["x"], H, d)
    kw = dict(positions=t["pos"], inv_freq=t["freq"], norm="l2", q_scale=d ** -0.5)
    qn, kn = gb.gdn_qk_norm_fwd(q, k, t["qw"], t["kw"], **kw)
    v = v.contiguous()
    o, hT = gb.gdn_kda_chunk_fwd(qn, kn, v, t["g"], t["beta"], t["h0"])
    near(o, o_ref, 1e-4, "o")
    near(hT, S_ref, 1e-4, "hT")
    dqn, dkn, dv, dg, db, dh0 = gb.gdn_kda_chunk_bwd(qn, kn, v, t["g"], t["beta"], t["do"], t["h0"], t["dhT"])
    dx = torch.empty_like(t["x"])
    dq, dk, dvx = split(dx, H, d)
    _, _, dqw, dkw = gb.gdn_qk_norm_bwd(q, k, dqn, dkn, t["qw"], t["kw"], dq=dq, dk=dk, **kw)
    dvx.copy_(dv)
    for name, a in (("x", dx), ("g", dg), ("beta", db), ("h0", dh0), ("qw", dqw), ("kw", dkw)):
        near(a, g_ref[name], 3e-4, "d" + name)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_then_tokens_on_a_pool(dtype):
    """Prompts through the chunked pass into slots of a pool, then draft tokens of unequal numbers (their states kept),
    then one more token from an accepted one: the outputs are those of the whole sequences in one chunked pass."""
    H, d, prompts, drafts = 2, 64, [70, 33], [4, 2]
    p = [project(10 + i, 1, n + m + 1, H, d, dtype) for i, (n, m) in enumerate(zip(prompts, drafts))]
    pool = torch.randn(12, H, d, d, device="cuda")
    before = pool.clone()
    slots = torch.tensor([7, 3], dtype=torch.int32, device="cuda")
    whole, parts = [], []
    for i, y in enumerate(p):
        t = {n: x.cuda() for n, x in y.items()}
        q, k, v = split(t["x"], H, d)
        q, k = gb.gdn_qk_norm_fwd(q, k, t["qw"], t["kw"], positions=t["pos"], inv_freq=t["freq"], q_scale=d ** -0.5)
        v = v.contiguous()
        full, _ = gb.gdn_kda_chunk_fwd(q, k, v, t["g"], t["beta"], t["h0"], o_dtype=torch.float32)
        whole.append(full)
        n = prompts[i]
        s = [x[:, :n].contiguous() for x in (q, k, v, t["g"], t["beta"])]
        _, hT = gb.gdn_kda_chunk_fwd(*s, t["h0"])
        pool[slots[i]] = hT[0]
        parts.append([x[0, n:] for x in (q, k, v, t["g"], t["beta"])])
    # the draft tokens of both sequences in one call, every state kept (slots 0, 1, 2, 4 and 5, 6)
    cu = torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda")
    keep = torch.tensor([0, 1, 2, 4, 5, 6], dtype=torch.int32, device="cuda")
    x = [torch.cat([a[:4], b[:2]]) for a, b in zip(*parts)]
    o = gb.gdn_recurrent_fwd(*x, pool, slots, cu, keep)
    # the first sequence goes on from its third draft token, the second from its last
    x = [torch.stack([a[3], b[2]]) for a, b in zip(*parts)]
    o2 = gb.gdn_recurrent_fwd(*x, pool, torch.tensor([2, 6], dtype=torch.int32, device="cuda"))
    # the recurrent form is fp32; the chunked pass is within 1e-4 of the largest output (fp32) or 2e-2 of the RMS (bf16)
    for got, ref in ((o[:4], whole[0][0, 70:74]), (o[4:], whole[1][0, 33:35]), (o2[0], whole[0][0, 73]), (o2[1], whole[1][0, 35])):
        err = float((got - ref).abs().max() / (ref.abs().max() if dtype == torch.float32 else ref.square().mean().sqrt()))
        print(f"      {err:.2e}", flush=True)
        assert err <= (2e-4 if dtype == torch.float32 else 4e-2)
    for i in (8, 9, 10, 11):
        assert torch.equal(pool[i], before[i])
