"""Cases and plain forms of the operators that stand around the SwiGLU layers: layer norm
(forward, backward), the clipping of a model's gradients by their global norm, and the routed
mixture-of-experts layer for a few tokens.

Each case names one operator (``"op"``) and its sizes; ``run`` performs one pass of it, in
elementary torch operations in 32 bits, or (``own``) through the library's entry points.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5          # layer norm
CLIP_EPS = 1e-6     # added to the norm before the division


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the norm before the block of a decode step: 16 sequences, one token each
        dict(name="norm_fwd_decode", op="norm_fwd", M=16, D=4096, type="bf16", wtype="bf16", add=True),
        # the target training block's norm with the residual stream's sum fused in
        dict(name="norm_fwd_target", op="norm_fwd", M=11136, D=3584, type="bf16", wtype="fp32", add=True),
        # a width that no vector divides, in fp32, without a residual
        dict(name="norm_fwd_odd", op="norm_fwd", M=4099, D=1021, type="fp32", wtype="fp32", add=False),
        # the smallest training block
        dict(name="norm_bwd_tiny", op="norm_bwd", M=128, D=256, type="fp16", wtype="fp16", add=False),
        # the target training block; the residual stream's gradient is added to the result
        dict(name="norm_bwd_target", op="norm_bwd", M=11136, D=3584, type="bf16", wtype="fp32", add=True),
        # an odd width and an odd number of rows
        dict(name="norm_bwd_odd", op="norm_bwd", M=1537, D=5003, type="bf16", wtype="bf16", add=False),
        # gradients of the smallest block and its norm: W1, W2, gamma, beta
        dict(name="clip_tiny", op="clip", kind="block", layers=1, D=256, H=512, type="bf16", wtype="bf16",
             max_norm=1.0),
        # many odd-sized gradients of mixed types, a few large ones among them
        dict(name="clip_mixed", op="clip", kind="mixed", count=48, largest=6000001, shape_seed=3, max_norm=0.5),
        # four target blocks with their norms, larger than the L2 cache many times over
        dict(name="clip_stack4", op="clip", kind="block", layers=4, D=3584, H=14336, type="bf16", wtype="fp32",
             max_norm=1.0),
        # one token through a layer of 64 small experts
        dict(name="moe_one_token", op="moe", T=1, E=64, D=2048, H=1408, Dout=2048, k=8, renorm=False, add=False),
        # 16 sequences' next tokens through 8 large experts
        dict(name="moe_batch16", op="moe", T=16, E=8, D=4096, H=14336, Dout=4096, k=2, renorm=True, add=True),
        # a ragged batch near the largest, widths that are only multiples of 8
        dict(name="moe_ragged61", op="moe", T=61, E=40, D=2056, H=1416, Dout=2040, k=7, renorm=True, add=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "clip", "moe"])
    if op in ("norm_fwd", "norm_bwd"):
        D = _log_int(rng, 64, 16384)
        how = rng.choice(["any", "odd", "eights", "eights"])
        D = D | 1 if how == "odd" else max(64, D // 8 * 8) if how == "eights" else D
        M = _log_int(rng, 1, max(1, min(16384, 11136 * 3584 // D)))
        t = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if t == "fp32":
            M = max(1, M // 2)
        return dict(op=op, M=M, D=D, type=t, wtype=rng.choice([t, "fp32"]), add=rng.random() < 0.5)
    if op == "clip":
        if rng.random() < 0.5:
            D = _log_int(rng, 128, 4096) // 8 * 8
            H = _log_int(rng, 256, 14336) // 8 * 8
            layers = rng.randint(1, 8)
            while layers * 3 * D * H > 4 * 3 * 3584 * 14336:
                layers -= 1
            t = rng.choice(["bf16", "bf16", "fp16"])
            return dict(op=op, kind="block", layers=layers, D=D, H=H, type=t, wtype=rng.choice([t, "fp32"]),
                        max_norm=rng.choice([0.1, 1.0, 10.0]))
        return dict(op=op, kind="mixed", count=rng.randint(1, 56), largest=_log_int(rng, 1000, 8000000),
                    shape_seed=rng.randint(0, 10 ** 6), max_norm=rng.choice([0.1, 1.0, 1e6]))
    E = _log_int(rng, 2, 128)
    D = max(64, _log_int(rng, 256, 4096) // 8 * 8)
    H = max(64, _log_int(rng, 256, 14336) // 8 * 8)
    Dout = D if rng.random() < 0.75 else max(64, _log_int(rng, 256, 4096) // 8 * 8)
    while E * H * (2 * D + Dout) > 8 * 14336 * 3 * 4096:
        H = max(64, H // 2 // 8 * 8)
    return dict(op=op, T=_log_int(rng, 1, 64), E=E, D=D, H=H, Dout=Dout, k=rng.randint(1, min(8, E)),
                renorm=rng.random() < 0.5, add=rng.random() < 0.5)


def _clip_shapes(case):
    """(element count, type name) of every gradient, in the model's order."""
    if case["kind"] == "block":
        D, H, t, w = case["D"], case["H"], case["type"], case["wtype"]
        return [(2 * H * D, t), (D * H, t), (D, w), (D, w)] * case["layers"]
    g = torch.Generator().manual_seed(case["shape_seed"])
    u = torch.rand(case["count"], generator=g)
    which = torch.randint(0, 3, (case["count"],), generator=g).tolist()
    sizes = [max(1, int(case["largest"] ** float(v))) for v in u]
    sizes[0] = case["largest"]
    return [(n, ["bf16", "fp32", "fp16"][w]) for n, w in zip(sizes, which)]


def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        M, D = case["M"], case["D"]
        size, wsize = (4 if case[n] == "fp32" else 2 for n in ("type", "wtype"))
        if op == "norm_fwd":        # x (, residual) -> y (, their sum), mean, rstd
            return {"bytes": M * D * size * (4 if case["add"] else 2) + 2 * D * wsize + 8 * M, "flops": 8 * M * D}
        return {"bytes": M * D * size * (4 if case["add"] else 3) + 3 * D * wsize + 8 * M, "flops": 14 * M * D}
    if op == "clip":
        shapes = _clip_shapes(case)
        return {"bytes": sum(2 * n * (4 if t == "fp32" else 2) for n, t in shapes) + 4,
                "flops": sum(3 * n for n, _ in shapes)}
    T, E, D, H, Dout, k = (case[n] for n in ("T", "E", "D", "H", "Dout", "k"))
    # the experts that at least one of T tokens picks, with picks spread evenly
    used = E * (1.0 - (1.0 - k / E) ** T)
    return {"bytes": int(used * (2 * H * D + Dout * H) * 2 + 2 * E * D + 2 * T * (D + Dout * (2 if case["add"] else 1)) +
                         8 * T * k),
            "flops": 2 * T * E * D + 2 * T * k * (2 * H * D + Dout * H)}


# ------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        t = torch.empty(shape, device="cuda", dtype=dtype).normal_(mean, std, generator=g)
        return t

    st = dict(case)
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        M, D = case["M"], case["D"]
        t, w = TYPES[case["type"]], TYPES[case["wtype"]]
        channel = normal(D, std=0.5).exp()      # a residual stream's channels differ in scale
        shift = normal(D, std=0.3)
        st["x"] = (normal(M, D) * channel + shift).to(t)
        st["gamma"] = normal(D, std=0.2, mean=1.0).to(w)
        st["beta"] = normal(D, std=0.2).to(w)
        st["r"] = (normal(M, D) * channel).to(t) if case["add"] else None
        if op == "norm_bwd":        # x is the saved sum; r the gradient that skips the norm
            xd = st["x"].double()
            mean = xd.sum(1) / D
            st["mean"] = mean.float()
            st["rstd"] = (((xd - mean[:, None]) ** 2).sum(1) / D + EPS).rsqrt().float()
            st["dy"] = normal(M, D).to(t)
            del st["beta"]
        return st
    if op == "clip":
        # gradients of a batch mean: small, of another scale in every tensor
        shapes = _clip_shapes(case)
        total = sum(n for n, _ in shapes)
        scales = torch.empty(len(shapes)).uniform_(-1, 1, generator=torch.Generator().manual_seed(seed)).exp().tolist()
        st["grads"] = [normal(n, std=4.0 * c / math.sqrt(total), dtype=TYPES[t]) for (n, t), c in zip(shapes, scales)]
        st["out"] = [torch.empty_like(v) for v in st["grads"]]
        return st
    T, E, D, H, Dout = (case[n] for n in ("T", "E", "D", "H", "Dout"))
    bf = torch.bfloat16
    st["x"] = normal(T, D).to(bf)
    st["Wr"] = normal(E, D, std=D ** -0.5).to(bf)
    st["W1"] = normal(E, 2 * H, D, std=D ** -0.5, dtype=bf)
    st["W2"] = normal(E, Dout, H, std=H ** -0.5, dtype=bf)
    st["r"] = normal(T, Dout).to(bf) if case["add"] else None
    return st


# ------------------------------------------------------------------------------ one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _norm_fwd_own(st):
    from bwd_gemm_epilogue_gb300 import binding as sm
    y, s, mean, rstd = sm.swiglu_mlp_layer_norm_fwd(st["x"], st["gamma"], st["beta"], EPS, residual=st["r"])
    return dict(y=y, mean=mean, rstd=rstd, **(dict(s=s) if st["add"] else {}))


def _norm_fwd_plain(st):
    t, D = st["x"].dtype, st["D"]
    s = st["x"].float()
    if st["add"]:
        s = s + st["r"].float()
    mean = s.sum(1, keepdim=True) / D
    c = s - mean
    rstd = ((c * c).sum(1, keepdim=True) / D + EPS).rsqrt()
    y = (c * rstd * st["gamma"].float() + st["beta"].float()).to(t)
    return dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0], **(dict(s=s.to(t)) if st["add"] else {}))


def _norm_bwd_own(st):
    from bwd_gemm_epilogue_gb300 import binding as sm
    dx, dgamma, dbeta = sm.swiglu_mlp_layer_norm_bwd(st["dy"], st["x"], st["gamma"], st["mean"], st["rstd"],
                                                     dskip=st["r"])
    return dict(dx=dx, dgamma=dgamma, dbeta=dbeta)


def _norm_bwd_plain(st):
    D = st["D"]
    dy, rstd = st["dy"].float(), st["rstd"][:, None]
    xh = (st["x"].float() - st["mean"][:, None]) * rstd
    g = dy * st["gamma"].float()
    dx = (g - g.sum(1, keepdim=True) / D - xh * ((g * xh).sum(1, keepdim=True) / D)) * rstd
    if st["add"]:
        dx = dx + st["r"].float()
    w = st["gamma"].dtype
    return dict(dx=dx.to(st["x"].dtype), dgamma=(dy * xh).sum(0).to(w), dbeta=dy.sum(0).to(w))


def _clip_own(st):
    from bwd_gemm_epilogue_gb300 import binding as sm
    norm, out = sm.swiglu_mlp_clip_grads(st["grads"], st["max_norm"], CLIP_EPS, out=st["out"])
    return dict(norm=norm, out=out)


def _clip_plain(st):
    squares = [(v * v).sum() for v in (t.float() for t in st["grads"])]
    norm = torch.stack(squares).sum().sqrt()
    scale = (st["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    return dict(norm=norm, out=[(t.float() * scale).to(t.dtype) for t in st["grads"]])


def _moe_own(st):
    from bwd_gemm_epilogue_gb300 import binding as sm
    y, ids, gates = sm.swiglu_moe_routed_fwd(st["x"], st["Wr"], st["W1"], st["W2"], st["k"],
                                             renormalize=st["renorm"], residual=st["r"])
    return dict(y=y, ids=ids, gates=gates)


def _moe_plain(st):
    T, E, H, k = st["T"], st["E"], st["H"], st["k"]
    x = st["x"].float()
    logits = x @ st["Wr"].float().T
    p = (logits - logits.max(1, keepdim=True).values).exp()
    p = p / p.sum(1, keepdim=True)
    gates, ids = torch.sort(p, dim=1, descending=True, stable=True)     # ties: the lowest index first
    gates, ids = gates[:, :k], ids[:, :k]
    if st["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    if T * k <= E:      # fewer picks than experts: only the picked experts' weights
        z = torch.matmul(st["W1"][ids.reshape(-1)].float(), x.repeat_interleave(k, 0)[:, :, None])[:, :, 0]
        h = z[:, :H] * (z[:, H:] / (1 + (-z[:, H:]).exp()))
        o = torch.matmul(st["W2"][ids.reshape(-1)].float(), h[:, :, None]).reshape(T, k, -1)
    else:               # every expert on every token, then the picked ones
        z = torch.matmul(x, st["W1"].float().transpose(1, 2))           # [E, T, 2H]
        h = z[..., :H] * (z[..., H:] / (1 + (-z[..., H:]).exp()))
        o = torch.matmul(h, st["W2"].float().transpose(1, 2))           # [E, T, Dout]
        o = o[ids, torch.arange(T, device=x.device)[:, None]]
    y = (o * gates[:, :, None]).sum(1)
    if st["add"]:
        y = y + st["r"].float()
    return dict(y=y.to(torch.bfloat16), ids=ids.int(), gates=gates)


_OWN = {"norm_fwd": _norm_fwd_own, "norm_bwd": _norm_bwd_own, "clip": _clip_own, "moe": _moe_own}
_PLAIN = {"norm_fwd": _norm_fwd_plain, "norm_bwd": _norm_bwd_plain, "clip": _clip_plain, "moe": _moe_plain}


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        s = st["x"].double() + (st["r"].double() if case["add"] else 0.0)
        var, mean = torch.var_mean(s, dim=1, correction=0, keepdim=True)
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = torch.addcmul(st["beta"].double(), (s - mean) / torch.sqrt(var + EPS), st["gamma"].double())
        return dict(y=y, mean=mean.squeeze(1), rstd=rstd.squeeze(1), **(dict(s=s) if case["add"] else {}))
    if op == "norm_bwd":
        # the Jacobian of the normalisation, with the given statistics held as the forward's:
        # D dx / rstd = D g - <1, g> 1 - <xh, g> xh
        D = case["D"]
        dy, x, gam = st["dy"].double(), st["x"].double(), st["gamma"].double()
        r = st["rstd"].double().unsqueeze(1)
        xh = x.sub(st["mean"].double().unsqueeze(1)).mul(r)
        dot1 = torch.mv(dy, gam).unsqueeze(1)
        dotx = torch.mv(dy * xh, gam).unsqueeze(1)
        dx = r / D * (D * (dy * gam) - dot1 - dotx * xh)
        if case["add"]:
            dx = dx + st["r"].double()
        return dict(dx=dx, dgamma=torch.einsum("md,md->d", dy, xh), dbeta=torch.ones_like(dy[:, 0]) @ dy)
    if op == "clip":
        total = 0.0
        for t in st["grads"]:
            total += torch.linalg.vector_norm(t, dtype=torch.float64).item() ** 2
        norm = math.sqrt(total)
        factor = min(1.0, case["max_norm"] / (norm + CLIP_EPS))
        return dict(norm=norm, out=[t.double().mul_(factor) for t in st["grads"]])
    H, k = case["H"], case["k"]
    x = st["x"].double()
    logits = torch.einsum("td,ed->te", x, st["Wr"].double())
    order = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
    picked = torch.gather(logits, 1, order)
    base = torch.logsumexp(picked if case["renorm"] else logits, dim=1, keepdim=True)
    gates = torch.exp(picked - base)
    y = st["r"].double() if case["add"] else torch.zeros(case["T"], case["Dout"], dtype=torch.float64, device=x.device)
    for e in sorted(set(order.reshape(-1).tolist())):
        t, j = torch.nonzero(order == e, as_tuple=True)
        z = x[t] @ st["W1"][e].double().T
        left, gate = z.split(H, dim=1)
        h = left * gate * torch.sigmoid(gate)
        y.index_add_(0, t, (h @ st["W2"][e].double().T) * gates[t, j].unsqueeze(1))
    return dict(y=y, ids=order.int(), gates=gates)
