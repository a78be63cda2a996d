"""Plain 64-bit forms of the calls that move rows between token order and expert order."""
import torch


def slot_map(T, K, E, drop, gen):
    """[T * K] int32 (CPU): the row of every slot among the rows sorted by expert, -1 for a
    share `drop` of the slots; and the number of rows in use."""
    R = T * K
    expert = torch.rand(T, E, generator=gen).topk(K, 1).indices.reshape(-1)
    gone = torch.randperm(R, generator=gen)[: int(R * drop)]
    expert[gone] = E
    row = torch.empty(R, dtype=torch.int64)
    row[torch.sort(expert, stable=True).indices] = torch.arange(R)
    row[gone] = -1
    return row.int(), R - len(gone)


def dispatch(x, row, K, xg):
    """xg (64 bits) with x's rows put in."""
    out = xg.double().clone()
    for slot, r in enumerate(row.tolist()):
        if 0 <= r < out.shape[0]:
            out[r] = x[slot // K].double()
    return out


def combine(z, row, w, residual=None):
    """(y, the sum of the absolute terms) in 64 bits; w [T, K] or the slots a token."""
    K = w if isinstance(w, int) else w.shape[1]
    row = row.long().view(-1, K)
    have = (row >= 0) & (row < z.shape[0])
    z = z.double()
    # a slot without a row adds nothing, whatever lies in row 0 or in its weight
    terms = torch.where(have[..., None], z[row.clamp(0, max(z.shape[0] - 1, 0))], 0.0) if z.shape[0] else \
        torch.zeros(*row.shape, z.shape[1], dtype=torch.float64)
    if not isinstance(w, int):
        terms = terms * torch.where(have, w.double(), 0.0)[..., None]
    y, size = terms.sum(1), terms.abs().sum(1)
    if residual is not None:
        y, size = y + residual.double(), size + residual.double().abs()
    return y, size


def combine_backward(dy, z, row, w, dz):
    """(dz, dw, the sum of dw's absolute terms) in 64 bits."""
    T, K = w.shape
    dz, z, dy = dz.double().clone(), z.double(), dy.double()
    dw, size = (torch.zeros(T, K, dtype=torch.float64) for _ in range(2))
    for slot, r in enumerate(row.tolist()):
        if 0 <= r < z.shape[0]:
            t, k = divmod(slot, K)
            dz[r] = w[t, k].double() * dy[t]
            dw[t, k] = (dy[t] * z[r]).sum()
            size[t, k] = (dy[t] * z[r]).abs().sum()
    return dz, dw, size
