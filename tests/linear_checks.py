"""Comparisons of tensor-core linear attention with the fp64 oracle that see a
lost or stale chunk.

Bounds are relative L2 errors, u = 2^-24.
* Outputs and gradients carry two bf16 roundings, of the score (or state) operand
  and of the result, each at most half a step, 2^-8.  Terms and roundings are
  independent of one another, so both together stay within sqrt(2) 2^-8 over the
  128 tokens of a chunk and head.  (The sum of a few tokens over the heads of a group
  can cancel, so an end of less than 16 tokens counts with the chunk before it.)
* fp32 states: a chunk's sum is at most 24 accumulations of 16 products (three
  parts of 128 tokens), each off by u, with weights off by 2 u; carrying it over n
  chunks (segments) rounds twice at each, sqrt(2 n / 3) u, of which twice is allowed.
"""
import numpy as np

CHUNK = 128
U = 2.0 ** -24
OUT_BOUND = 2 ** 0.5 * 2.0 ** -8


def state_bound(chunks):
    return (26 + 2 * (2 * chunks / 3) ** 0.5) * U


def worst_chunk(x, ref, lens):
    """The largest relative L2 error of x [T,H,D] over the (chunk, head) of every sequence."""
    x, ref = np.asarray(x, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    worst, t = 0.0, 0
    for n in lens:
        assert n == 0 or n >= 16
        starts = list(range(t, t + n, CHUNK))
        if len(starts) > 1 and t + n - starts[-1] < 16:
            starts.pop()
        for t0, t1 in zip(starts, starts[1:] + [t + n]):
            a = slice(t0, t1)
            err = np.sqrt(((x[a] - ref[a]) ** 2).sum((0, 2)))
            worst = max(worst, float((err / np.sqrt((ref[a] ** 2).sum((0, 2)))).max()))
        t += n
    return worst


def worst_state(x, ref):
    """The largest relative L2 error of x [N,H,Dv,Dk] over (sequence, head)."""
    x, ref = np.asarray(x, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    return float((np.sqrt(((x - ref) ** 2).sum((2, 3))) / np.sqrt((ref ** 2).sum((2, 3)))).max())


def dw_bound(dy, n, additions=600):
    """What a norm weight's gradient, the sum over rows [T,H,D] of dy n in fp32, may be off
    by, per column.  A term is within 2 (D + 64) u of its row's largest (the turned
    gradient, the row's inverse root), and passes through at most `additions` partial
    sums, each rounded by u of what it holds.  Rows are independent, so all of it adds in
    quadrature; three times that is allowed."""
    D = dy.shape[-1]
    size = np.abs(dy).max(-1, keepdims=True) * np.abs(n)
    return 3 * (2 * (D + 64) + additions) * U * np.sqrt((size ** 2).sum((0, 1)))
