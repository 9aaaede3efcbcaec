"""Plain 64-bit forms of the operators of include/swiglu_tokens.h, for their tests."""
import numpy as np
import torch

U = 2.0 ** -24
UT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -24, torch.float32: 1e-37}    # below the normal range


def within(got, ref, scale, what):
    """|got - ref| <= scale + uT |ref| everywhere (ref, scale fp64), and NaN where ref is."""
    assert got.shape == ref.shape, what
    assert torch.equal(got.isnan(), ref.isnan()), f"{what}: NaN"
    bound = scale + UT[got.dtype] * (ref.abs() + scale) + TINY[got.dtype]
    over = ((got.double() - ref).abs() / bound).nan_to_num(nan=0.0)
    assert bool((over <= 1).all()), f"{what}: {over.max().item():.3g} times the bound"


def philox(counter, key):
    """Philox4x32-10 of [n, 4] uint32 counters -> [n, 4] uint32."""
    c = np.asarray(counter, dtype=np.uint64).reshape(-1, 4).T
    k = [int(v) for v in key]
    low = np.uint64(0xffffffff)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = np.stack([(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low])
        k = [(k[0] + 0x9E3779B9) & 0xffffffff, (k[1] + 0xBB67AE85) & 0xffffffff]
    return c.T.astype(np.uint32)


def keep_mask(M, D, p, seed, offset, row=0):
    """(bool [M, D] of rows row .. row + M - 1, kept elements' factor)."""
    keep = round((1 - p) * 65536)
    blocks = -(-D // 8)
    b, i = np.meshgrid(np.arange(blocks), np.arange(row, row + M))
    offset %= 1 << 64
    counter = np.stack([b.ravel(), i.ravel(), np.full(b.size, offset & 0xffffffff), np.full(b.size, offset >> 32)], axis=1)
    words = philox(counter, (seed & 0xffffffff, seed >> 32))
    bits = np.ascontiguousarray(words.astype("<u4")).view("<u2").reshape(M, 8 * blocks)[:, :D]
    return torch.from_numpy(bits.astype(np.int64) < keep).cuda(), 65536 / max(keep, 1)


def dropped(x64, p, seed, offset):
    if p == 0:
        return x64
    mask, f = keep_mask(*x64.shape, p, seed, offset)
    return torch.where(mask, x64 * f, 0.0)


def gate(logits, k, renormalize):
    """(ids, gates, p): ties to the lowest index, NaN lowest, minus infinity never."""
    l = logits.double()
    rank = l.nan_to_num(nan=-1e300, neginf=-np.inf, posinf=np.inf)
    ids = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :k]
    none = torch.gather(rank, 1, ids) == -np.inf
    top = rank.max(1, keepdim=True).values
    p = (l - torch.where(top == -np.inf, 0.0, top)).exp()
    gates = torch.gather(p, 1, ids)
    total = gates.masked_fill(none, 0.0).sum(1, keepdim=True) if renormalize else p.sum(1, keepdim=True)
    total = torch.where(p.isnan().any(1, keepdim=True), np.nan, total)
    total = torch.where(total == 0, 1.0, total)
    return ids.masked_fill(none, -1), (gates / total).masked_fill(none, 0.0), p / torch.where(p.sum(1, keepdim=True) == 0, 1.0, p.sum(1, keepdim=True))


def sort(ids, E):
    flat = ids.reshape(-1).cpu().numpy()
    pos = np.full(flat.size, -1)
    counts = np.zeros(E, dtype=np.int64)
    order = [np.nonzero(flat == e)[0] for e in range(E)]
    at = 0
    for e, o in enumerate(order):
        pos[o] = np.arange(at, at + o.size)
        counts[e] = o.size
        at += o.size
    return torch.from_numpy(counts).int(), torch.from_numpy(pos).int().reshape(ids.shape)


def picked(rows, pos):
    """[T, k, D] fp64 rows of the pairs, zeros where there is none, and which there are."""
    here = (pos >= 0) & (pos < rows.shape[0])
    if rows.shape[0] == 0:
        return torch.zeros(*pos.shape, rows.shape[1], dtype=torch.float64, device=rows.device), here
    return torch.where(here[:, :, None], rows.double()[torch.where(here, pos, 0).long()], 0.0), here
