"""A token-mixing block from the library's own operators, as a model runs it: the residual
stream's norm, projections (torch), the L2 norm of q and k, a mixer (Gated DeltaNet, or the
gated linear recurrence), the heads' norm under its gate, the output projection, and the
residual scale with the next norm.  Prefill and decoding agree, and the recurrence block's
gradients agree with differentiating its float64 formula.
"""
import pytest
import torch

import deltanet_chunkwise_delta_b200 as dn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32
H, D = 4, 512                     # 4 heads x 128


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dn.load()


def weights(seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)
    p = {n: (r(D, D) / D ** 0.5).to(DEV, BF) for n in ("q", "k", "v", "z", "o")}
    p["ab"] = (r(D, 2 * H) / D ** 0.5).to(DEV, BF)
    p["decay"] = (r(D, D) / D ** 0.5).to(DEV, BF)
    for n, d in (("pre", D), ("next", D), ("head", 128), ("scale", D)):
        p[n] = (1 + 0.1 * r(d)).to(DEV)
    p["l2"] = torch.full((128,), 128 ** -0.5, device=DEV)
    return p


def gdn_block(p, x, mix):
    """x [B, T, D] (fp32 residual stream) -> (next block's input, residual stream); mix runs
    the recurrence."""
    n, _ = dn.deltanet_norm_fwd(x.to(BF), p["pre"])
    heads = lambda t: t.view(*t.shape[:2], H, 128)
    q, k, v, z = (heads(n @ p[w]) for w in "qkvz")
    q, _ = dn.deltanet_norm_fwd(q, p["l2"], eps=1e-6 / 128)
    k, _ = dn.deltanet_norm_fwd(k, p["l2"], eps=1e-6 / 128)
    ab = (n @ p["ab"]).float()
    g, beta = torch.nn.functional.logsigmoid(ab[..., :H] + 3), torch.sigmoid(ab[..., H:])
    o = mix(q, k, v, beta.contiguous(), g.contiguous())
    o, _ = dn.deltanet_norm_fwd(o, p["head"], z)
    y = o.reshape(*x.shape) @ p["o"]
    return dn.deltanet_norm_fwd(y, residual=x, scale=p["scale"], next_weight=p["next"])


def test_prefill_then_decoding_is_one_prefill():
    """200 tokens at once == 190 at once and 10 decoded one by one, through a cache with the
    requests in other rows (bf16 products: 2e-2 of the largest value, the forward pass's own
    bar of 1e-2 on each side)."""
    p = weights()
    x = torch.randn((3, 200, D), generator=torch.Generator().manual_seed(1)).to(DEV)
    full_state = []

    def prefill(q, k, v, beta, g):
        o, s = dn.gated_deltanet_fwd(q, k, v, beta, g)
        full_state.append(s)
        return o

    want_n, want_r = gdn_block(p, x, prefill)
    n0, r0 = gdn_block(p, x[:, :190].contiguous(), prefill)
    cache = torch.full((8, H, 128, 128), float("nan"), device=DEV)
    slots = torch.tensor([6, 1, 3], dtype=torch.int32, device=DEV)
    cache[slots.long()] = full_state[1]
    ns, rs = [n0], [r0]
    for t in range(190, 200):
        n, r = gdn_block(p, x[:, t:t + 1].contiguous(),
                         lambda q, k, v, beta, g: dn.deltanet_step(q, k, v, beta, cache, g, slot_idx=slots))
        ns.append(n), rs.append(r)
    rel = lambda a, b: ((a.float() - b.float()).abs().max() / b.float().abs().max()).item()
    assert rel(torch.cat(ns, 1), want_n) <= 2e-2 and rel(torch.cat(rs, 1), want_r) <= 2e-2
    assert rel(cache[slots.long()], full_state[0]) <= 2e-2
    assert torch.isnan(cache[[0, 2, 4, 5, 7]]).all()
    assert dn.get_error() == 0


def rec_forward(x, w, cu):
    """The recurrence block in fp32 from the library's operators; what its backward needs."""
    n, _ = dn.deltanet_norm_fwd(x, w["pre"])
    u, g = n @ w["v"], torch.nn.functional.logsigmoid(n @ w["decay"] + 2)
    h, _ = dn.deltanet_scan_fwd(u, g, None, cu)
    z = n @ w["z"]
    o, _ = dn.deltanet_norm_fwd(h, w["mid"], z)
    y = o @ w["o"]
    out, r = dn.deltanet_norm_fwd(y, residual=x, scale=w["scale"], next_weight=w["next"])
    return out, r, (n, g, h, z, o, y)


def rec_backward(x, w, cu, saved, d_out, d_r):
    n, g, h, z, o, y = saved
    top = dn.deltanet_norm_bwd(y, d_out, residual=x, scale=w["scale"], next_weight=w["next"], d_residual_out=d_r)
    d_o = top.d_y @ w["o"].T
    mid = dn.deltanet_norm_bwd(h, d_o, w["mid"], z)
    du, dg, _ = dn.deltanet_scan_bwd(g, h, mid.d_y, None, cu)
    # g = logsigmoid(t): dg/dt = 1 - sigmoid(t) = 1 - e^g
    dt = dg * (1 - g.exp())
    dn_ = du @ w["v"].T + dt @ w["decay"].T + mid.d_gate @ w["z"].T
    pre = dn.deltanet_norm_bwd(x, dn_, w["pre"])
    flat = lambda t: t.reshape(-1, t.shape[-1])
    return dict(x=top.d_residual + pre.d_y, pre=pre.d_weight, mid=mid.d_weight, scale=top.d_scale,
                next=top.d_next_weight, v=flat(n).T @ flat(du), decay=flat(n).T @ flat(dt),
                z=flat(n).T @ flat(mid.d_gate), o=flat(o).T @ flat(top.d_y))


def rec_reference(x, w, cu):
    """The same block, token by token in float64, for autograd."""
    rms = lambda t, v: t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * v
    n = rms(x, w["pre"])
    u, a, z = n @ w["v"], torch.sigmoid(n @ w["decay"] + 2), n @ w["z"]
    hs, starts = [], set(cu)
    for t in range(x.shape[1]):
        hs.append(u[:, t] if t in starts else a[:, t] * hs[-1] + u[:, t])
    h = torch.stack(hs, 1)
    y = (rms(h, w["mid"]) * torch.nn.functional.silu(z)) @ w["o"]
    r = x + w["scale"] * y
    return rms(r, w["next"]), r


def test_recurrence_block_gradients():
    """Outputs and every gradient of the block against float64 autograd, packed sequences.
    fp32 throughout with torch's fp32 products: 1e-4 of each tensor's largest value (sums of
    up to 150 x 96 terms of mixed sign at 2^-24 each)."""
    torch.backends.cuda.matmul.allow_tf32 = False
    d, cu = 96, [0, 60, 61, 61, 150]
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen)
    w = {n: r(d, d) / d ** 0.5 for n in ("v", "decay", "z", "o")}
    w.update({n: 1 + 0.1 * r(d) for n in ("pre", "mid", "scale", "next")})
    x, d_out, d_r = r(1, 150, d), r(1, 150, d), r(1, 150, d)
    on = lambda t: t.to(DEV)
    gw = {k: on(t) for k, t in w.items()}
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    out, res, saved = rec_forward(on(x), gw, c)
    got = rec_backward(on(x), gw, c, saved, on(d_out), on(d_r))
    w64 = {k: t.double().requires_grad_() for k, t in w.items()}
    x64 = x.double().requires_grad_()
    o64, r64 = rec_reference(x64, w64, cu)
    ((o64 * d_out).sum() + (r64 * d_r).sum()).backward()
    rel = lambda a, b: ((a.double().cpu() - b).abs().max() / b.abs().max()).item()
    assert rel(out, o64.detach()) <= 1e-4 and rel(res, r64.detach()) <= 1e-4
    assert rel(got["x"], x64.grad) <= 1e-4
    for k in w:
        assert rel(got[k], w64[k].grad) <= 1e-4, k
    assert dn.get_error() == 0


def test_backward_in_a_graph_beside_an_eager_one():
    """The block's forward and backward captured and replayed while the results of an eager
    run on the same tensors live."""
    d = 128
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen).to(DEV)
    w = {n: r(d, d) / d ** 0.5 for n in ("v", "decay", "z", "o")}
    w.update({n: 1 + 0.1 * r(d) for n in ("pre", "mid", "scale", "next")})
    x, d_out, d_r = r(2, 90, d), r(2, 90, d), r(2, 90, d)

    def step():
        out, res, saved = rec_forward(x, w, None)
        return [out, res, *rec_backward(x, w, None, saved, d_out, d_r).values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = step()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=side):
        captured = step()
    for _ in range(2):
        gr.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, eager):
        assert torch.equal(a, b)
