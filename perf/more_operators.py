"""Cases and plain forms of the operators on a token's way through a mixture-of-experts layer in
training, and of dropout: the gate (top-k softmax of the router's logits), the rows sorted by expert
and back with the gates applied, each with its gradient, and dropout with a mask that is computed and
never stored.

Each case names one operator (``"op"``) and its sizes; ``run`` performs one pass of it, in
elementary torch operations in 32 bits, or (``own``) through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the gate of a few sequences' next tokens, fine-grained experts
        dict(name="gate_fwd_few", op="gate_fwd", T=64, E=64, k=6, type="fp32", renorm=True, masked=False),
        # the gate of a large training batch
        dict(name="gate_fwd_batch", op="gate_fwd", T=65536, E=128, k=8, type="fp32", renorm=True, masked=False),
        # its gradient where the gates are shares of all experts, some switched off, and a padded batch's
        # tokens choose none; odd sizes
        dict(name="gate_bwd_odd", op="gate_bwd", T=40961, E=61, k=7, type="bf16", renorm=False, masked=True),
        # the smallest batch's tokens to their experts: 16 sequences, one token each
        dict(name="dispatch_fwd_few", op="dispatch_fwd", T=16, E=8, k=2, D=4096, type="bf16", dropped=0.0),
        # 8192 tokens to two of 8 large experts each
        dict(name="dispatch_fwd_moe8", op="dispatch_fwd", T=8192, E=8, k=2, D=4096, type="bf16", dropped=0.0),
        # the gradient of an odd batch in fp32, a tenth of the choices held by other ranks
        dict(name="dispatch_bwd_odd", op="dispatch_bwd", T=4099, E=40, k=7, D=1021, type="fp32", add="fp32", dropped=0.1),
        # one token's experts added up
        dict(name="combine_fwd_one", op="combine_fwd", T=1, E=64, k=8, D=2048, type="bf16", add="same", dropped=0.0, p=0.0),
        # 4096 tokens, six of 64 fine-grained experts each, into the residual stream with dropout
        dict(name="combine_fwd_moe64", op="combine_fwd", T=4096, E=64, k=6, D=2048, type="bf16", add="same", dropped=0.0,
             p=0.1),
        # the gradient of 8192 tokens' two large experts
        dict(name="combine_bwd_moe8", op="combine_bwd", T=8192, E=8, k=2, D=4096, type="bf16", dropped=0.0, p=0.1),
        # the gradient at an odd width in fp16, a tenth of the choices held by other ranks
        dict(name="combine_bwd_odd", op="combine_bwd", T=4099, E=40, k=7, D=1021, type="fp16", dropped=0.1, p=0.0),
        # the smallest training block's output
        dict(name="dropout_tiny", op="dropout", M=128, D=256, type="fp16", add=False, p=0.5),
        # the target training block's branch into its residual stream
        dict(name="dropout_target", op="dropout", M=11136, D=3584, type="bf16", add=True, p=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate_fwd", "gate_bwd", "dispatch_fwd", "dispatch_bwd", "combine_fwd", "combine_bwd", "dropout"])
    t = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    E = _log_int(rng, 2, 512)
    if op in ("gate_fwd", "gate_bwd"):
        T = _log_int(rng, 1, min(65536, 65536 * 128 // E))
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), type=t, renorm=rng.random() < 0.5,
                    masked=rng.random() < 0.5)
    D = _log_int(rng, 64, 8192)
    how = rng.choice(["any", "odd", "eights", "eights", "eights"])
    D = D | 1 if how == "odd" else max(64, D // 8 * 8) if how == "eights" else D
    size = 4 if t == "fp32" else 2
    p = rng.choice([0.0, 0.1, 0.25])
    if op == "dropout":
        return dict(op=op, M=_log_int(rng, 1, max(1, min(65536, 11136 * 3584 * 2 // (D * size)))), D=D, type=t,
                    add=rng.random() < 0.5, p=rng.choice([0.05, 0.1, 0.25, 0.5]))
    k = rng.randint(1, min(8, E))
    T = _log_int(rng, 1, max(1, min(32768, 8192 * 2 * 4096 * 2 // (D * k * size))))
    c = dict(op=op, T=T, E=E, k=k, D=D, type=t, dropped=rng.choice([0.0, 0.0, 0.1, 0.5]) if T >= 32 else 0.0)
    if op == "dispatch_bwd":
        return dict(c, add=rng.choice(["none", "same", "fp32"]))
    if op == "combine_fwd":
        return dict(c, add=rng.choice(["none", "same"]), p=p)
    return dict(c, p=p) if op == "combine_bwd" else c


def work(case):
    op = case["op"]
    size = 4 if case["type"] == "fp32" else 2
    if op == "dropout":
        n = case["M"] * case["D"]
        return {"bytes": n * size * (3 if case["add"] else 2), "flops": 2 * n}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "gate_fwd":        # logits -> ids, gates
        return {"bytes": T * E * size + 8 * T * k, "flops": 4 * T * E}
    if op == "gate_bwd":        # ids, gates, their gradients (, logits) -> the logits' gradient
        return {"bytes": T * E * size * (1 if case["renorm"] else 2) + 12 * T * k, "flops": 4 * T * k + 4 * T * E}
    D, pairs = case["D"], T * k * (1 - case["dropped"])
    row = D * size
    if op == "dispatch_fwd":    # ids, x -> counts, pos, rows
        return {"bytes": int(8 * T * k + 4 * E + T * row + pairs * row), "flops": T * k}
    if op == "dispatch_bwd":    # pos, the rows' gradient (, add) -> dx
        more = {"none": 0, "same": size, "fp32": 4}[case["add"]]
        return {"bytes": int(4 * T * k + pairs * row + T * row + T * D * more), "flops": int(pairs * D)}
    if op == "combine_fwd":     # pos, gates, rows (, residual) -> y
        return {"bytes": int(8 * T * k + pairs * row + T * row * (2 if case["add"] != "none" else 1)), "flops": int(2 * pairs * D)}
    return {"bytes": int(12 * T * k + 2 * pairs * row + T * row), "flops": int(4 * pairs * D)}


# ------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=g)

    def choice(T, E, k):
        """k different experts for each token, by falling logit, some liked more than others."""
        return torch.sort(normal(T, E) + normal(E, std=0.5), dim=1, descending=True)[1][:, :k].contiguous()

    st = dict(case)
    op, t = case["op"], TYPES[case["type"]]
    if op == "dropout":
        M, D = case["M"], case["D"]
        st["x"] = normal(M, D).to(t)
        st["r"] = normal(M, D).to(t) if case["add"] else None
    elif op in ("gate_fwd", "gate_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        logits = normal(T, E, std=1.5) + normal(E, std=0.5)
        if case["masked"]:      # experts switched off, and tokens of a padded batch
            logits.masked_fill_(torch.rand(E, device="cuda", generator=g) < 0.1, -math.inf)
            logits.masked_fill_(torch.rand(T, 1, device="cuda", generator=g) < 0.1, -math.inf)
        st["logits"] = logits.to(t)
        if op == "gate_bwd":    # what the forward gave
            st["ids"], st["gates"] = _gate_plain(st["logits"], k, case["renorm"])
            st["dgates"] = normal(T, k)
    else:
        T, E, k, D = case["T"], case["E"], case["k"], case["D"]
        ids = choice(T, E, k).int()
        if case["dropped"]:     # choices of experts that are not here
            ids.view(-1)[torch.randperm(T * k, device="cuda", generator=g)[:int(T * k * case["dropped"])]] = -1
        st["N"] = N = int((ids >= 0).sum())
        if op == "dispatch_fwd":
            st["ids"], st["x"] = ids, normal(T, D).to(t)
            return st
        st["pos"] = _sort_plain(ids, E)[1]
        st["rows"] = normal(N, D).to(t)         # the experts' outputs, or (dispatch_bwd) their inputs' gradients
        st["gates"] = torch.rand(T, k, device="cuda", generator=g)
        st["gates"] /= st["gates"].sum(1, keepdim=True)
        if op == "combine_bwd":
            st["dy"] = normal(T, D).to(t)
        elif case["add"] == "none":
            st["add_to"] = None
        else:
            st["add_to"] = normal(T, D).to(torch.float32 if case["add"] == "fp32" else t)
    # a run's seed, and the step and the layer that a dropout belongs to
    st["seed"], st["offset"] = 0x9d2c5680 * (seed + 1) % 2 ** 63, 3
    st["step"] = torch.tensor(1000 + seed, dtype=torch.int64, device="cuda")
    return st


# ------------------------------------------------------------------------------ one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _gate_fwd_own(st):
    from bwd_gemm_epilogue_gb300 import binding as sm
    ids, gates = sm.swiglu_moe_gate_fwd(st["logits"], st["k"], renormalize=st["renorm"])
    return dict(ids=ids, gates=gates)


def _gate_bwd_own(st):
    from bwd_gemm_epilogue_gb300 import binding as sm
    return dict(dlogits=sm.swiglu_moe_gate_bwd(st["logits"], st["ids"], st["gates"], st["dgates"], renormalize=st["renorm"]))


def _dispatch_fwd_own(st):
    from bwd_gemm_epilogue_gb300 import binding as sm
    counts, pos = sm.swiglu_moe_sort(st["ids"], st["E"])
    return dict(counts=counts, pos=pos, rows=sm.swiglu_moe_dispatch_fwd(st["x"], pos, st["N"]))


def _dispatch_bwd_own(st):
    from bwd_gemm_epilogue_gb300 import binding as sm
    return dict(dx=sm.swiglu_moe_dispatch_bwd(st["rows"], st["pos"], add=st["add_to"]))


def _combine_fwd_own(st):
    from bwd_gemm_epilogue_gb300 import binding as sm
    return dict(y=sm.swiglu_moe_combine_fwd(st["rows"], st["pos"], st["gates"], residual=st["add_to"], p=st["p"],
                                            seed=st["seed"], offset=st["offset"], step=st["step"]))


def _combine_bwd_own(st):
    from bwd_gemm_epilogue_gb300 import binding as sm
    drows, dgates = sm.swiglu_moe_combine_bwd(st["dy"], st["rows"], st["pos"], st["gates"], p=st["p"], seed=st["seed"],
                                              offset=st["offset"], step=st["step"])
    return dict(drows=drows, dgates=dgates)


def _dropout_own(st):
    from bwd_gemm_epilogue_gb300 import binding as sm
    return dict(y=sm.swiglu_mlp_dropout(st["x"], st["p"], st["seed"], offset=st["offset"], step=st["step"], residual=st["r"]))


def _gate_plain(logits, k, renorm):
    """Top k of softmax(logits), ties to the lowest index; where no logit above -inf is left, id -1 and gate 0."""
    l = logits.float()
    top = l.max(1, keepdim=True).values
    p = (l - torch.where(top == -math.inf, 0.0, top)).exp()
    picked, ids = torch.sort(l, dim=1, descending=True, stable=True)
    none = picked[:, :k] == -math.inf
    ids = ids[:, :k]
    gates = torch.gather(p, 1, ids)
    total = gates.sum(1, keepdim=True) if renorm else p.sum(1, keepdim=True)
    gates = gates / torch.where(total == 0, 1.0, total)
    return ids.masked_fill(none, -1).int(), gates.masked_fill(none, 0.0)


def _gate_fwd_plain(st):
    ids, gates = _gate_plain(st["logits"], st["k"], st["renorm"])
    return dict(ids=ids, gates=gates)


def _gate_bwd_plain(st):
    l, ids, q, dq = st["logits"].float(), st["ids"].long(), st["gates"], st["dgates"]
    here = ids >= 0
    mean = (q * dq).sum(1, keepdim=True)
    d = torch.zeros(l.shape[0], l.shape[1] + 1, device=l.device)
    slot = torch.where(here, ids, l.shape[1])           # the last column takes what no expert has
    if st["renorm"]:
        d = d.scatter(1, slot, q * (dq - mean))[:, :-1]
    else:
        top = l.max(1, keepdim=True).values
        p = (l - torch.where(top == -math.inf, 0.0, top)).exp()
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total == 0, 1.0, total)
        d = p * (d.scatter(1, slot, dq)[:, :-1] - mean)
    return dict(dlogits=d.to(st["logits"].dtype))


def _sort_plain(ids, E):
    """(rows of each expert, the row of each (token, choice) pair by expert, then by token and choice)."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.argsort(key, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(flat.numel(), device=ids.device)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).index_add(0, key, torch.ones_like(key))[:E]
    return counts.int(), torch.where(flat < 0, -1, pos).int().reshape(ids.shape)


def _dispatch_fwd_plain(st):
    counts, pos = _sort_plain(st["ids"], st["E"])
    rows = torch.empty(st["N"] + 1, st["D"], dtype=st["x"].dtype, device=pos.device)
    to = torch.where(pos < 0, st["N"], pos).long().reshape(-1)      # the last row takes what no expert gets
    rows[to] = st["x"].repeat_interleave(st["k"], 0)
    return dict(counts=counts, pos=pos, rows=rows[:-1])


def _picked_rows(st):
    """[T, k, D] fp32: the pairs' rows, zeros where there is none."""
    if st["N"] == 0:
        return torch.zeros(*st["pos"].shape, st["D"], device=st["pos"].device)
    return st["rows"].float()[st["pos"].clamp(min=0).long()] * (st["pos"] >= 0)[:, :, None]


def _dispatch_bwd_plain(st):
    dx = _picked_rows(st).sum(1)
    if st["add_to"] is not None:
        dx = dx + st["add_to"].float()
    return dict(dx=dx.to(st["rows"].dtype))


def _low(v):
    return v & 0xffffffff


def _philox(c0, c1, c2, c3, seed):
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011) of 32-bit words held in int64 tensors."""
    k0, k1 = seed & 0xffffffff, seed >> 32

    def high(m, c):     # of the 64-bit product: in int64 it would be signed
        return (c * (m >> 16) + (c * (m & 0xffff) >> 16)) >> 16

    for i in range(10):
        a, b = (k0 + i * 0x9E3779B9) & 0xffffffff, (k1 + i * 0xBB67AE85) & 0xffffffff
        c0, c1, c2, c3 = (high(0xCD9E8D57, c2) ^ c1 ^ a, _low(c2 * 0xCD9E8D57),
                          high(0xD2511F53, c0) ^ c3 ^ b, _low(c0 * 0xD2511F53))
    return c0, c1, c2, c3


def _factor(st, M, D):
    """[M, D]: 65536 / K where the 16 bits of an element are below K = round((1 - p) 65536), else 0.  Columns
    8 b .. 8 b + 7 of row i take the low and the high half of each word of Philox(b, i, offset + step)."""
    keep = round((1 - st["p"]) * 65536)
    block = torch.arange((D + 7) // 8, device="cuda")[None]
    row = torch.arange(M, device="cuda")[:, None]
    counter = (st["offset"] + st["step"]).expand(M, block.shape[1])
    words = _philox(block.expand_as(counter), row.expand_as(counter), _low(counter), _low(counter >> 32), st["seed"])
    bits = torch.stack([h for w in words for h in (w & 0xffff, w >> 16)], dim=2).reshape(M, -1)[:, :D]
    return (bits < keep).float() * (65536 / keep if keep else 0.0)


def _combine_fwd_plain(st):
    y = (_picked_rows(st) * st["gates"][:, :, None]).sum(1)
    if st["p"]:
        y = y * _factor(st, st["T"], st["D"])
    if st["add_to"] is not None:
        y = y + st["add_to"].float()
    return dict(y=y.to(st["rows"].dtype))


def _combine_bwd_plain(st):
    dy = st["dy"].float()
    if st["p"]:
        dy = dy * _factor(st, st["T"], st["D"])
    rows = _picked_rows(st)
    dgates = (rows * dy[:, None]).sum(2)
    drows = torch.empty(st["N"] + 1, st["D"], dtype=st["dy"].dtype, device=dy.device)
    to = torch.where(st["pos"] < 0, st["N"], st["pos"]).long().reshape(-1)
    drows[to] = (dy[:, None] * st["gates"][:, :, None]).to(drows.dtype).reshape(-1, st["D"])
    return dict(drows=drows[:-1], dgates=dgates)


def _dropout_plain(st):
    y = st["x"].float() * _factor(st, st["M"], st["D"])
    if st["add"]:
        y = y + st["r"].float()
    return dict(y=y.to(st["x"].dtype))


_OWN = {"gate_fwd": _gate_fwd_own, "gate_bwd": _gate_bwd_own, "dispatch_fwd": _dispatch_fwd_own,
        "dispatch_bwd": _dispatch_bwd_own, "combine_fwd": _combine_fwd_own, "combine_bwd": _combine_bwd_own,
        "dropout": _dropout_own}
_PLAIN = {"gate_fwd": _gate_fwd_plain, "gate_bwd": _gate_bwd_plain, "dispatch_fwd": _dispatch_fwd_plain,
          "dispatch_bwd": _dispatch_bwd_plain, "combine_fwd": _combine_fwd_plain, "combine_bwd": _combine_bwd_plain,
          "dropout": _dropout_plain}


# ------------------------------------------------------------------------------ 64 bits

def _exact_factor(st, M, D):
    """The same mask by 64-bit unsigned arithmetic on the host, the blocks of all rows in one array."""
    u = np.uint64
    low, half = u(0xffffffff), u(32)
    blocks = -(-D // 8)
    at = np.arange(M * blocks, dtype=np.uint64)
    counter = u((st["offset"] + int(st["step"])) % 2 ** 64)
    x = [at % u(blocks), at // u(blocks), np.broadcast_to(counter & low, at.shape), np.broadcast_to(counter >> half, at.shape)]
    key = [st["seed"] % 2 ** 32, st["seed"] // 2 ** 32]
    for _ in range(10):
        first, second = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(second >> half) ^ x[1] ^ u(key[0]), second & low, (first >> half) ^ x[3] ^ u(key[1]), first & low]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    words = np.stack(x, axis=1).astype("<u4")
    bits = words.view("<u2").reshape(M, blocks * 8)[:, :D]
    keep = round((1 - st["p"]) * 65536)
    return torch.from_numpy(bits < keep).cuda().double() * (65536 / max(keep, 1))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        y = torch.mul(st["x"].double(), _exact_factor(st, case["M"], case["D"]))
        return dict(y=y if st["r"] is None else y.add_(st["r"].double()))
    if op in ("gate_fwd", "gate_bwd"):
        l, k, E = st["logits"].double(), case["k"], case["E"]
        # fill the k places one after the other with the largest logit that is left
        left, ids = l.clone(), []
        at = torch.arange(case["T"], device=l.device)
        index = torch.arange(E, device=l.device)
        for _ in range(k):
            best = left.amax(1)
            e = torch.where(left == best[:, None], index, E).amin(1)
            ids.append(torch.where(best == -math.inf, -1, e))
            left[at, e] = -math.inf
        ids = torch.stack(ids, 1)
        chosen = torch.where(ids >= 0, torch.gather(l, 1, ids.clamp(min=0)), -math.inf)
        norm = torch.logsumexp(chosen if case["renorm"] else l, 1, keepdim=True)
        norm = norm.masked_fill(norm == -math.inf, 0.0)
        gates = (chosen - norm).exp()
        if op == "gate_fwd":
            return dict(ids=ids.int(), gates=gates)
        # the Jacobian of softmax, on the chosen ones or on all experts
        pick = (ids[:, :, None] == index).double()                              # [T, k, E]
        q, dg = st["gates"].double(), st["dgates"].double()
        if case["renorm"]:
            d = torch.einsum("tk,tke->te", q * dg, pick) - torch.einsum("tk,tke->te", q, pick) * (q * dg).sum(1, keepdim=True)
        else:
            p = (l - norm).exp()
            up = torch.einsum("tk,tke->te", dg, pick)
            d = p * up - p * (p * up).sum(1, keepdim=True)
        return dict(dlogits=d)
    T, E, k, D, N = case["T"], case["E"], case["k"], case["D"], st["N"]
    if op == "dispatch_fwd":
        ids = st["ids"].reshape(-1).cpu().numpy()
        counts = np.array([(ids == e).sum() for e in range(E)])
        pairs = np.concatenate([np.nonzero(ids == e)[0] for e in range(E)])
        pos = np.full(T * k, -1)
        pos[pairs] = np.arange(N)
        rows = st["x"].double()[torch.from_numpy(pairs // k).cuda()]
        return dict(counts=torch.from_numpy(counts).int(), pos=torch.from_numpy(pos).int().reshape(T, k), rows=rows)
    pos = st["pos"]
    t, j = torch.nonzero(pos >= 0, as_tuple=True)
    at = pos[t, j].long()
    rows = st["rows"].double()
    zeros = torch.zeros(T, D, dtype=torch.float64, device=rows.device)
    factor = _exact_factor(st, T, D) if case.get("p") else torch.ones((), dtype=torch.float64, device=rows.device)
    if op == "combine_bwd":
        dy = st["dy"].double() * factor
        dgates = torch.zeros(T, k, dtype=torch.float64, device=rows.device)
        dgates[t, j] = torch.einsum("nd,nd->n", dy[t], rows[at])
        drows = torch.empty_like(rows)
        drows[at] = dy[t] * st["gates"].double()[t, j, None]
        return dict(drows=drows, dgates=dgates)
    weights = st["gates"].double()[t, j, None] if op == "combine_fwd" else 1.0
    out = zeros.index_add_(0, t, rows[at] * weights) * factor
    if st["add_to"] is not None:
        out = out + st["add_to"].double()
    return {"y" if op == "combine_fwd" else "dx": out}
