"""Plain 64-bit definitions of the experts' row moves on CPU tensors, and the
bounds their tests use (error model: ffn_ref)."""
import torch

import ffn_ref as ref


def sort(ids, E):
    """(pos, offsets, order) by Python's stable sort."""
    T, k = ids.shape
    flat = ids.flatten().tolist()
    kept = sorted((s for s in range(T * k) if 0 <= flat[s] < E), key=lambda s: flat[s])
    pos = [-1] * (T * k)
    for i, s in enumerate(kept):
        pos[s] = i
    offsets, c = [0] * (E + 1), [0] * E
    for s in kept:
        c[flat[s]] += 1
    for e in range(E):
        offsets[e + 1] = offsets[e] + c[e]
    i32 = lambda v, *s: torch.tensor(v, dtype=torch.int32).view(*s)
    return i32(pos, T, k), i32(offsets, E + 1), i32(kept + [-1] * (T * k - len(kept)), T * k)


def _weights(w, pos):
    return torch.ones(pos.shape, dtype=torch.float64) if w is None else w.double()


def out(x, pos, w, before):
    """Rows of x, weighted, into `before`; and the tolerance: one FP32 product, then
    the rounding."""
    got, tol = before.double().clone(), torch.zeros(before.shape, dtype=torch.float64)
    ww = _weights(w, pos)
    for t, j in torch.nonzero(pos >= 0).tolist():
        r = x[t].double() * ww[t, j]
        got[pos[t, j]] = r
        e = r.abs() * ref.U32
        tol[pos[t, j]] = e + ref.rounding(r.abs() + e, before.dtype)
    return got, tol


def back(rows, pos, w, D):
    """The weighted sums; k fused steps, each off by a rounding of at most the sum
    of magnitudes, then the rounding."""
    T, k = pos.shape
    got, mag = torch.zeros(T, D, dtype=torch.float64), torch.zeros(T, D, dtype=torch.float64)
    ww = _weights(w, pos)
    for t, j in torch.nonzero(pos >= 0).tolist():
        r = rows[pos[t, j]].double() * ww[t, j]
        got[t] += r
        mag[t] += r.abs()
    e = mag * (k * ref.U32)
    return got, e + ref.rounding(got.abs() + e, rows.dtype)


def dots(x, rows, pos, dtype):
    """The weights' gradient: at least 32 threads share a row, so one adds up at
    most D / 32 products and a vector's worth (8) and an element behind the
    vectors; 5 steps join a warp's, 8 a CTA's."""
    T, k = pos.shape
    D = x.shape[1]
    got, mag = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for t, j in torch.nonzero(pos >= 0).tolist():
        r = x[t].double() * rows[pos[t, j]].double()
        got[t, j], mag[t, j] = r.sum(), r.abs().sum()
    e = mag * ((D / 32 + 22) * ref.U32)
    return got, e + ref.rounding(got.abs() + e, dtype)
