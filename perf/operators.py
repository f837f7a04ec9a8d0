"""What is measured of the operators around the delta-rule kernels: the gated linear
recurrence (``deltanet_scan_*``), the norms before and after a block (``deltanet_norm_*``)
and the single-token form of the delta rule on a cache of states (``deltanet_step``).

``run`` computes each operator in its plain form (elementary torch operations in 32 bits,
rounded once at the end), or, with ``own`` true, through the library.  ``exact`` computes
it in 64 bits from its definition.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # the recurrence as the mixer of one training layer: 8 rows of 2048 tokens, the
        # 1.3B layer's width (16 heads x 128)
        dict(name="scan_fwd_layer", op="scan_fwd", B=8, T=2048, D=2048, N=0, x="bf16", g="f32",
             init=False, fused=False),
        # a packed batch of 32 sequences with their start states, gates in bf16 beside the
        # input in one projection's output: the packed workload's number of tokens
        dict(name="scan_fwd_packed", op="scan_fwd", B=1, T=222459, D=2048, N=32, x="bf16", g="bf16",
             init=True, fused=True),
        # training on one long sequence
        dict(name="scan_bwd_long", op="scan_bwd", B=1, T=65536, D=2048, N=0, x="bf16", g="f32",
             init=False, fused=False),
        # odd sizes in 32 bits with the state's gradients, as a parity run of a small model
        dict(name="scan_bwd_odd", op="scan_bwd", B=3, T=1000, D=1111, N=0, x="f32", g="f32",
             init=True, fused=False),
        # one decoded token for each of 256 requests, states in a larger cache
        dict(name="scan_step_256", op="scan_step", N=256, T=1, D=2048, slots=320, x="bf16", g="f32"),
        # between two blocks of a training layer: residual scale, sum and the next norm
        dict(name="norm_fwd_residual", op="norm_fwd", B=8, T=2048, H=0, d=2048, y="bf16", r="f32",
             weight=False, gate="none", scale=True, next=True),
        # a mixer's heads under their norm and gate, ahead of the output projection
        dict(name="norm_fwd_heads", op="norm_fwd", B=8, T=2048, H=16, d=128, y="bf16", r="none",
             weight=True, gate="silu", scale=False, next=False),
        # the whole chain's gradients: norm after the block, gate, scale, residual, next norm
        dict(name="norm_bwd_block", op="norm_bwd", B=8, T=2048, H=0, d=2048, y="bf16", r="bf16",
             weight=True, gate="sigmoid", scale=True, next=True),
        # gradients of the heads' norm and gate
        dict(name="norm_bwd_heads", op="norm_bwd", B=8, T=2048, H=16, d=128, y="bf16", r="none",
             weight=True, gate="silu", scale=False, next=False),
        # one decoded token for 256 requests of a Gated DeltaNet layer (16 heads, 128 x 128)
        dict(name="step_gdn_256", op="step", N=256, T=1, H=16, dk=128, dv=128, nh=1, rule="gdn",
             x="bf16", slots=320),
        # one request alone, where latency counts
        dict(name="step_single", op="step", N=1, T=1, H=16, dk=128, dv=128, nh=1, rule="delta",
             x="bf16", slots=1),
        # a few drafted tokens per request in 32 bits, a decay per key channel, d_k != d_v
        dict(name="step_kda_draft", op="step", N=33, T=4, H=8, dk=64, dv=128, nh=1, rule="kda",
             x="f32", slots=40),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the listed ranges: sizes spread over their logarithm, odd ones among them,
    the work bounded by the largest listed case of the kind."""
    op = rng.choice(["scan_fwd", "scan_bwd", "scan_step", "norm_fwd", "norm_bwd", "step"])
    if op in ("scan_fwd", "scan_bwd"):
        D = _log(rng, 16, 4096)
        if rng.random() < 0.6:
            D = max(16, D // 16 * 16)
        x = rng.choice(["bf16", "bf16", "f32"])
        g = "f32" if x == "f32" else rng.choice(["f32", "bf16"])
        packed = rng.random() < 0.4
        most = 100_000_000 // D
        T = _log(rng, 1, min(131072, most))
        B = 1 if packed else rng.randint(1, max(1, min(8, most // T)))
        return dict(op=op, B=B, T=T, D=D, N=_log(rng, 1, 64) if packed else 0, x=x, g=g,
                    init=rng.random() < 0.5, fused=x == g and rng.random() < 0.5)
    if op == "scan_step":
        N = _log(rng, 1, 512)
        return dict(op=op, N=N, T=rng.choice([1, 1, 1, 2, 4]), D=_log(rng, 32, 4096),
                    slots=N + rng.randint(0, 64), x=rng.choice(["bf16", "f32"]), g="f32")
    if op in ("norm_fwd", "norm_bwd"):
        heads = rng.random() < 0.4
        y = rng.choice(["bf16", "bf16", "f32"])
        d = rng.choice([32, 64, 80, 128, 256]) if heads else _log(rng, 64, 8192)
        if not heads and rng.random() < 0.6:
            d = max(64, d // 64 * 64)
        H = rng.randint(1, 32) if heads else 0
        T = _log(rng, 1, min(32768, 30_000_000 // (d * max(H, 1))))
        B = rng.randint(1, max(1, min(4, 30_000_000 // (d * max(H, 1) * T))))
        r = "none" if heads else rng.choice(["none", y, "f32"])
        weight = heads or r == "none" or rng.random() < 0.5
        return dict(op=op, B=B, T=T, H=H, d=d, y=y, r=r, weight=weight,
                    gate=rng.choice(["none", "silu", "sigmoid"]),
                    scale=r != "none" and rng.random() < 0.5,
                    next=r != "none" and rng.random() < 0.7)
    H, N, rule = rng.choice([1, 2, 3, 4, 8, 16, 32]), _log(rng, 1, 256), rng.choice(["delta", "gdn", "gdp", "kda"])
    while N * H > 4096:
        N //= 2
    return dict(op=op, N=N, T=rng.choice([1, 1, 1, 2, 3, 5, 8]), H=H, dk=rng.choice([64, 128]),
                dv=rng.choice([64, 128]), nh=rng.choice([2, 3]) if rule == "gdp" else 1, rule=rule,
                x=rng.choice(["bf16", "bf16", "f32"]), slots=N + rng.randint(0, 32))


# ---- inputs ------------------------------------------------------------------

def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _log_decay(gen, *shape):
    """ln a = logsigmoid(z + 4), z ~ N(0, 1): a has median 0.982 (the gated workloads' recipe)."""
    return torch.nn.functional.logsigmoid(_randn(gen, *shape) + 4.0)


def _offsets(T, N, seed):
    """Packed sequence starts: lengths in log-uniform proportions (a factor of 256), every
    seventh sequence without tokens."""
    rng = np.random.default_rng(seed)
    p = np.exp(rng.uniform(0.0, math.log(256.0), N))
    p[6::7] = 0.0
    cu = np.zeros(N + 1, dtype=np.int64)
    cu[1:] = np.floor(np.cumsum(p) / p.sum() * T + 0.5)
    cu[N] = T
    return torch.tensor(np.minimum(cu, T), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    s = dict(case=dict(case))
    op = case["op"]
    if op in ("scan_fwd", "scan_bwd"):
        B, T, D, N = case["B"], case["T"], case["D"], case["N"]
        xt, gt = DT[case["x"]], DT[case["g"]]
        if case["fused"]:
            # one projection's output holds x and g side by side
            both = torch.empty((B, T, 2 * D), dtype=xt, device="cuda")
            both[..., :D] = _randn(gen, B, T, D)
            both[..., D:] = _log_decay(gen, B, T, D)
            x, g = both[..., :D], both[..., D:]
        else:
            x = _randn(gen, B, T, D).to(xt)
            g = _log_decay(gen, B, T, D).to(gt)
        s["cu"] = _offsets(T, N, seed) if N else None
        n = N or B
        s["init"] = _randn(gen, n, D) * 0.5 if case["init"] else None
        s["x"], s["g"] = x, g
        if op == "scan_bwd":
            s["h"], _ = _plain_scan(x, g, s["init"], s["cu"])
            del s["x"]
            s["dh"] = _randn(gen, B, T, D).to(xt)
            s["dfinal"] = _randn(gen, n, D) if case["init"] else None
    elif op == "scan_step":
        N, T, D, M = case["N"], case["T"], case["D"], case["slots"]
        s["x"] = _randn(gen, N, T, D).to(DT[case["x"]])
        s["g"] = _log_decay(gen, N, T, D).to(DT[case["g"]])
        s["state"] = _randn(gen, M, D) * 0.5
        s["slots"] = torch.randperm(M, generator=gen, device="cuda")[:N].to(torch.int32)
    elif op in ("norm_fwd", "norm_bwd"):
        shape = (case["B"], case["T"], case["H"], case["d"]) if case["H"] else (case["B"], case["T"], case["d"])
        d, yt = case["d"], DT[case["y"]]
        s["y"] = _randn(gen, *shape).to(yt)
        s["weight"] = 1.0 + 0.1 * _randn(gen, d) if case["weight"] else None
        s["gate"] = _randn(gen, *shape).to(yt) if case["gate"] != "none" else None
        s["residual"] = _randn(gen, *shape).to(DT[case["r"]]) if case["r"] != "none" else None
        s["scale"] = 0.5 + 0.1 * _randn(gen, d) if case["scale"] else None
        s["next"] = 1.0 + 0.1 * _randn(gen, d) if case["next"] else None
        if op == "norm_bwd":
            has_out = case["next"] or case["r"] == "none"
            s["dout"] = _randn(gen, *shape).to(yt) if has_out else None
            s["dres"] = _randn(gen, *shape).to(DT[case["r"]]) if case["r"] != "none" else None
    else:
        N, T, H, dk, dv, M = (case[k] for k in ("N", "T", "H", "dk", "dv", "slots"))
        Tw, xt = T * case["nh"], DT[case["x"]]
        unit = torch.nn.functional.normalize
        s["q"] = unit(_randn(gen, N, T, H, dk), dim=-1).to(xt)
        s["k"] = unit(_randn(gen, N, Tw, H, dk), dim=-1).to(xt)
        s["v"] = _randn(gen, N, Tw, H, dv).to(xt)
        s["beta"] = torch.sigmoid(_randn(gen, N, Tw, H))
        s["g"] = {"delta": lambda: None, "gdn": lambda: _log_decay(gen, N, T, H),
                  "gdp": lambda: _log_decay(gen, N, T, H),
                  "kda": lambda: _log_decay(gen, N, T, H, dk)}[case["rule"]]()
        s["state"] = _randn(gen, M, H, dk, dv) * 0.1
        s["slots"] = torch.randperm(M, generator=gen, device="cuda")[:N].to(torch.int32)
    return s


# ---- plain forms -------------------------------------------------------------

def _ends(T, cu):
    """Of a packed batch: which tokens start a sequence and which end one [T]; for every
    sequence its first and last token (in range also without tokens) and whether it has any."""
    cu = cu.long()
    mark = torch.zeros((2, T + 1), dtype=torch.bool, device="cuda")
    mark[0].index_fill_(0, cu[:-1], True)
    mark[1].index_fill_(0, cu[1:], True)
    return mark[0, :T], mark[1, 1:], cu[:-1].clamp(max=T - 1), (cu[1:] - 1).clamp(min=0), (cu[1:] > cu[:-1])[:, None]


def _doubling(a, h):
    """The recurrence h_t += a_t h_{t-1} along dim 1 by doubling: after step j every token
    holds the map of the 2^j tokens up to it."""
    n, T = 1, a.shape[1]
    while n < T:
        h = torch.cat([h[:, :n], h[:, n:] + a[:, n:] * h[:, :-n]], dim=1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], dim=1)
        n *= 2
    return h


def _plain_scan(x, g, init, cu):
    a, h = torch.exp(g.float()), x.float().clone()
    if cu is None:
        if init is not None:
            h[:, 0] += a[:, 0] * init
        h = _doubling(a, h)
        return h.to(x.dtype), h[:, -1].clone()
    first, _, start, end, some = _ends(x.shape[1], cu)
    if init is not None:
        h[0].index_add_(0, start, torch.where(some, a[0, start] * init, 0.0))
    h = _doubling(a.masked_fill_(first[:, None], 0.0), h)
    return h.to(x.dtype), torch.where(some, h[0, end], 0.0 if init is None else init)


def _plain_scan_bwd(g, h, dh, init, dfinal, cu):
    a, e = torch.exp(g.float()), dh.float().clone()
    c = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], dim=1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], dim=1).float()
    if cu is None:
        if dfinal is not None:
            e[:, -1] += dfinal
        if init is not None:
            before[:, 0] = init
    else:
        first, last, start, end, some = _ends(h.shape[1], cu)
        if dfinal is not None:
            e[0].index_add_(0, end, torch.where(some, dfinal, 0.0))
        c.masked_fill_(last[:, None], 0.0)
        before.masked_fill_(first[:, None], 0.0)
        if init is not None:
            before[0].index_add_(0, start, torch.where(some, init, 0.0))
    delta = _doubling(c.flip(1), e.flip(1)).flip(1)
    out = [delta.to(h.dtype), (delta * a * before).to(g.dtype)]
    if init is not None and cu is None:
        out.append(delta[:, 0] * a[:, 0])
    elif init is not None:
        out.append(torch.where(some, delta[0, start] * a[0, start], 0.0 if dfinal is None else dfinal))
    return out


def _plain_scan_step(x, g, state, slots):
    at = slots.long()
    T = x.shape[1]
    first = torch.cat([state[at][:, None], x.float()], dim=1)
    a = torch.cat([torch.zeros_like(first[:, :1]), torch.exp(g.float())], dim=1)
    h = _doubling(a, first)
    state[at] = h[:, T]
    return h[:, 1:].to(x.dtype)


def _act(z, kind):
    sig = torch.sigmoid(z)
    return z * sig if kind == "silu" else sig


def _act_grad(z, kind):
    sig = torch.sigmoid(z)
    return sig * (1 + z * (1 - sig)) if kind == "silu" else sig * (1 - sig)


EPS = 1e-6


def _norm_parts(s):
    c = s["case"]
    y = s["y"].float()
    rstd1 = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    y1 = y * rstd1 * s["weight"] if s["weight"] is not None else y
    act = _act(s["gate"].float(), c["gate"]) if s["gate"] is not None else None
    y2 = y1 * act if act is not None else y1
    return y, rstd1, y1, act, y2


def _plain_norm(s):
    y2 = _norm_parts(s)[4]
    if s["residual"] is None:
        return [y2.to(s["y"].dtype)]
    r = s["residual"].float() + (y2 if s["scale"] is None else s["scale"] * y2)
    out = [r.to(s["residual"].dtype)]
    if s["next"] is not None:
        n = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["next"]
        out.append(n.to(s["y"].dtype))
    return out


def _plain_norm_bwd(s):
    c = s["case"]
    y, rstd1, y1, act, y2 = _norm_parts(s)
    rows = tuple(range(y.dim() - 1))
    out = {}
    if s["residual"] is None:
        dy2 = s["dout"].float()
    else:
        dr = s["dres"].float()
        if s["next"] is not None:
            r = s["residual"].float() + (y2 if s["scale"] is None else s["scale"] * y2)
            rstd2 = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
            dn = s["dout"].float()
            out["d_next"] = (dn * r * rstd2).sum(rows)
            t = dn * s["next"]
            dr = dr + rstd2 * (t - r * rstd2 * rstd2 * (t * r).mean(-1, keepdim=True))
        out["d_residual"] = dr.to(s["residual"].dtype)
        dy2 = dr
        if s["scale"] is not None:
            out["d_scale"] = (dr * y2).sum(rows)
            dy2 = dr * s["scale"]
    if act is not None:
        out["d_gate"] = (dy2 * y1 * _act_grad(s["gate"].float(), c["gate"])).to(s["gate"].dtype)
        dy2 = dy2 * act
    if s["weight"] is not None:
        out["d_weight"] = (dy2 * y * rstd1).sum(rows)
        t = dy2 * s["weight"]
        dy2 = rstd1 * (t - y * rstd1 * rstd1 * (t * y).mean(-1, keepdim=True))
    out["d_y"] = dy2.to(s["y"].dtype)
    return out


def _plain_step(s):
    c, at = s["case"], s["slots"].long()
    nh = c["nh"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    S, beta = s["state"][at], s["beta"]
    out = []
    for t in range(c["T"]):  # a token's write needs the state that the one before it left
        if s["g"] is not None:
            a = torch.exp(s["g"][:, t])
            S = S * (a[..., None] if c["rule"] == "kda" else a[..., None, None])
        for j in range(t * nh, (t + 1) * nh):
            u = beta[:, j, :, None] * (v[:, j] - (k[:, j, :, :, None] * S).sum(-2))
            S = S + k[:, j, :, :, None] * u[:, :, None, :]
        out.append((q[:, t, :, :, None] * S).sum(-2))
    s["state"][at] = S
    return [torch.stack(out, 1).to(s["q"].dtype), s["state"]]


# ---- one pass ----------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    op = s["case"]["op"]
    if op == "scan_fwd":
        return list(_plain_scan(s["x"], s["g"], s["init"], s["cu"]))
    if op == "scan_bwd":
        return _plain_scan_bwd(s["g"], s["h"], s["dh"], s["init"], s["dfinal"], s["cu"])
    if op == "scan_step":
        return [_plain_scan_step(s["x"], s["g"], s["state"], s["slots"]), s["state"]]
    if op == "norm_fwd":
        return _plain_norm(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    return _plain_step(s)


def _run_own(s):
    import deltanet_chunkwise_delta_b200 as dn

    c = s["case"]
    op = c["op"]
    if op == "scan_fwd":
        return list(dn.deltanet_scan_fwd(s["x"], s["g"], s["init"], s["cu"]))
    if op == "scan_bwd":
        dx, dg, dinit = dn.deltanet_scan_bwd(s["g"], s["h"], s["dh"], s["init"], s["cu"], s["dfinal"])
        return [dx, dg] if dinit is None else [dx, dg, dinit]
    if op == "scan_step":
        return [dn.deltanet_scan_step(s["x"], s["g"], s["state"], s["slots"]), s["state"]]
    act = c.get("gate", "none")
    act = "silu" if act == "none" else act
    if op == "norm_fwd":
        out, res = dn.deltanet_norm_fwd(s["y"], s["weight"], s["gate"], s["residual"], s["scale"], s["next"],
                                        activation=act, eps=EPS)
        return [x for x in (res, out) if x is not None]
    if op == "norm_bwd":
        gr = dn.deltanet_norm_bwd(s["y"], s["dout"], s["weight"], s["gate"], s["residual"], s["scale"],
                                  s["next"], s["dres"], activation=act, eps=EPS)
        got = dict(d_y=gr.d_y, d_weight=gr.d_weight, d_gate=gr.d_gate, d_residual=gr.d_residual,
                   d_scale=gr.d_scale, d_next=gr.d_next_weight)
        return {k: x for k, x in got.items() if x is not None}
    return [dn.deltanet_step(s["q"], s["k"], s["v"], s["beta"], s["state"], s["g"], c["nh"], s["slots"]),
            s["state"]]


# ---- bytes and operations ----------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("scan_fwd", "scan_bwd"):
        e, n = case["B"] * case["T"] * case["D"], (case["N"] or case["B"]) * case["D"]
        x, g = SIZE[case["x"]], SIZE[case["g"]]
        if op == "scan_fwd":
            return dict(bytes=e * (2 * x + g) + 4 * n * (2 if case["init"] else 1), flops=3 * e)
        return dict(bytes=e * (3 * x + 2 * g) + (12 * n if case["init"] else 0), flops=5 * e)
    if op == "scan_step":
        n = case["N"] * case["D"]
        return dict(bytes=n * (case["T"] * (2 * SIZE[case["x"]] + SIZE[case["g"]]) + 8), flops=3 * n * case["T"])
    if op in ("norm_fwd", "norm_bwd"):
        e = case["B"] * case["T"] * max(case["H"], 1) * case["d"]
        y, r = SIZE[case["y"]], SIZE.get(case["r"], 0)
        has_out = case["next"] or case["r"] == "none"
        gate, w = case["gate"] != "none", 4 * case["d"] * (case["weight"] + case["scale"] + case["next"])
        if op == "norm_fwd":
            return dict(bytes=e * (y * (1 + gate + has_out) + 2 * r) + w, flops=12 * e)
        return dict(bytes=e * (y * (2 + 2 * gate + has_out) + 3 * r) + 2 * w, flops=30 * e)
    N, T, H, dk, dv, nh, x = (case[k] for k in ("N", "T", "H", "dk", "dv", "nh", "x"))
    rows = N * T * H
    gate = {"delta": 0, "gdn": 4, "gdp": 4, "kda": 4 * dk}[case["rule"]]
    b = rows * (SIZE[x] * (dk + dv + nh * (dk + dv)) + 4 * nh + gate) + 8 * N * H * dk * dv
    return dict(bytes=b, flops=rows * dk * dv * (4 * nh + 2 + (case["rule"] != "delta")))


# ---- 64 bits -----------------------------------------------------------------

def _tokens(cu, B, T):
    """(row, state, first token, tokens) of every sequence."""
    if cu is None:
        return [(b, b, 0, T) for b in range(B)]
    c = cu.tolist()
    return [(0, n, c[n], c[n + 1] - c[n]) for n in range(len(c) - 1)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = lambda t: None if t is None else t.double()
    if op in ("scan_fwd", "scan_bwd"):
        B, T, D, cu = case["B"], case["T"], case["D"], s["cu"]
        seqs = _tokens(cu, B, T)
        a = torch.exp(f(s["g"]))
        n = case["N"] or B
        if op == "scan_fwd":
            h, final = f(s["x"]), torch.zeros((n, D), dtype=torch.float64, device="cuda")
            if case["init"]:
                final.copy_(s["init"])
            if cu is None:  # the rows side by side, token after token
                for t in range(T):
                    final = torch.addcmul(h[:, t], a[:, t], final)
                    h[:, t] = final
                return [h, final]
            for b, i, t0, L in seqs:
                st = final[i].clone()
                for t in range(t0, t0 + L):
                    st = torch.addcmul(h[b, t], a[b, t], st)
                    h[b, t] = st
                final[i] = st
            return [h, final]
        h, dx = f(s["h"]), f(s["dh"])
        carry = torch.zeros((n, D), dtype=torch.float64, device="cuda")
        if s["dfinal"] is not None:
            carry.copy_(s["dfinal"])
        if cu is None:
            for t in range(T - 1, -1, -1):
                dx[:, t] += carry
                carry = dx[:, t] * a[:, t]
        for b, i, t0, L in seqs if cu is not None else []:
            c = carry[i].clone()
            for t in range(t0 + L - 1, t0 - 1, -1):
                dx[b, t] += c
                c = dx[b, t] * a[b, t]
            carry[i] = c
        dg = a.mul_(dx)
        for b, i, t0, L in seqs:
            if L:
                dg[b, t0 + 1:t0 + L] *= h[b, t0:t0 + L - 1]
                dg[b, t0] *= s["init"][i].double() if case["init"] else 0.0
        return [dx, dg] + ([carry] if case["init"] else [])
    if op == "scan_step":
        at, state = s["slots"].long(), f(s["state"])
        out = []
        for t in range(case["T"]):
            state[at] = torch.exp(f(s["g"][:, t])) * state[at] + f(s["x"][:, t])
            out.append(state[at])
        return [torch.stack(out, 1), state]
    if op == "norm_fwd":
        return [x.detach() for x in _exact_norm(s, {})[::-1] if x is not None]
    if op == "norm_bwd":
        leaves = {}
        out, res = _exact_norm(s, leaves)
        pairs = [(o, f(g)) for o, g in ((out, s["dout"]), (res, s["dres"])) if o is not None]
        grads = torch.autograd.grad([o for o, _ in pairs], list(leaves.values()), [g for _, g in pairs])
        names = dict(y="d_y", weight="d_weight", gate="d_gate", residual="d_residual", scale="d_scale",
                     next="d_next")
        return {names[k]: g for k, g in zip(leaves, grads)}
    S, at, nh = f(s["state"]), s["slots"].long(), case["nh"]
    out = torch.zeros((case["N"], case["T"], case["H"], case["dv"]), dtype=torch.float64, device="cuda")
    cur = S[at]
    for m in range(case["T"] * nh):
        t = m // nh
        if m % nh == 0 and s["g"] is not None:
            a = torch.exp(f(s["g"][:, t]))
            cur = cur * a.reshape(a.shape + (1,) * (cur.dim() - a.dim()))
        k = f(s["k"][:, m])
        u = f(s["beta"][:, m])[..., None] * (f(s["v"][:, m]) - torch.einsum("nhk,nhkv->nhv", k, cur))
        cur = cur + torch.einsum("nhk,nhv->nhkv", k, u)
        if m % nh == nh - 1:
            out[:, t] = torch.einsum("nhk,nhkv->nhv", f(s["q"][:, t]), cur)
    S[at] = cur
    return [out, S]


def _exact_norm(s, leaves):
    """The chain in 64 bits; its inputs go into ``leaves`` for differentiation."""
    def leaf(name):
        if s[name] is None:
            return None
        leaves[name] = s[name].double().requires_grad_()
        return leaves[name]

    def rms(v, w):
        return w * v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)

    with torch.enable_grad():
        o, w, z, r, sc, nx = (leaf(k) for k in ("y", "weight", "gate", "residual", "scale", "next"))
        if w is not None:
            o = rms(o, w)
        if z is not None:
            o = o * (z if s["case"]["gate"] == "silu" else 1.0) / (1.0 + torch.exp(-z))
        if r is None:
            return o, None
        r = r + (o if sc is None else sc * o)
        return (None if nx is None else rms(r, nx)), r
