"""Plain 64-bit forms and error bounds for the operators on unquantized and
4-bit integer experts (not a test module).

Bounds: a sum of R exact products in fp32, added in any order with an error
of at most 2^-23 per addition, is off by at most R * 2^-23 * S, S the sum of
the products' magnitudes; a rounding to bf16 is off by at most 2^-8 of the
value (half a step)."""
import torch

F64 = torch.float64
U32 = 2.0 ** -23
BF16_HALF = 2.0 ** -8


def offsets_of(counts, first=0, device="cuda:0"):
    off = [first]
    for c in counts:
        off.append(off[-1] + c)
    return torch.tensor(off, dtype=torch.int32, device=device)


def experts_rows(offsets):
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def source_rows(x, slots, k, M):
    """The rows that the sorted rows read, in fp64 (zeros for slots outside)."""
    if slots is None:
        return x.to(F64)
    s = slots.long()
    ok = (s >= 0) & (s < x.shape[0] * k)
    return x.to(F64)[torch.where(ok, s // k, 0)] * ok[:, None]


def product(rows, w, offsets, transpose=True):
    """(sum, sum of magnitudes) per output of rows . w[e]^T (or rows . w[e])."""
    n = w.shape[1] if transpose else w.shape[2]
    y = torch.zeros((rows.shape[0], n), dtype=F64, device=rows.device)
    mag = torch.zeros_like(y)
    for e, lo, hi in experts_rows(offsets):
        we = w[e].to(F64)
        we = we.t().contiguous() if transpose else we
        y[lo:hi] = rows[lo:hi] @ we
        mag[lo:hi] = rows[lo:hi].abs() @ we.abs()
    return y, mag


def assert_within(got, ref, bound, what, rows=None):
    got = got.to(F64)
    if rows is not None:
        got, ref, bound = got[rows], ref[rows], bound[rows]
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - bound
    assert got.numel() == 0 or over.max().item() <= 0, \
        f"{what}: {(over > 0).sum().item()} of {got.numel()} values outside the bound, by {over.max().item():.3g}"


def rounded(ref, err):
    """Bound of a value that is off by err and then rounded to bf16."""
    return err + BF16_HALF * (ref.abs() + err) + 2.0 ** -133


def swiglu(a, b):
    return a * torch.sigmoid(a) * b


def swiglu_error(a, ea, b, eb):
    """|d silu| <= 1.1 |d a|; silu itself in fp32 from a fast exponential:
    relative error at most (|a| + 8) 2^-22."""
    silu = (a * torch.sigmoid(a)).abs()
    rel = (a.abs() + 8) * 2.0 ** -22
    return (1.1 * ea) * (b.abs() + eb) + silu * eb + rel * (silu + 1.1 * ea) * (b.abs() + eb)
