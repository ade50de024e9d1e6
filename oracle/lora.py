"""Low-rank adapters of many requests beside a projection (fp64).

Test infrastructure: only the tests use this module; the GPU path never does.
A row at a time: delta[t] = scale[l] B_l (A_l x_t), l = adapter[t]; zero
where l is no adapter.
"""

import numpy as np


def delta(x, a, b, adapter, scale):
    """(delta [T, N], bound [T, N]) in fp64. The bound covers float32 sums of exact products in any order (a relative
    2^-24 a term added, 2^-23 taken here), the product with the scale, and the second sum over three parts a value."""
    T, K = x.shape
    N, R = b.shape[1], b.shape[2]
    d, lim = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        l = int(adapter[t])
        if not 0 <= l < len(a):
            continue
        f = float(scale[l])
        h = a[l] @ x[t]
        eh = K * 2.0 ** -23 * (np.abs(a[l]) @ np.abs(x[t])) + 2.0 ** -24 * np.abs(h)
        d[t] = b[l] @ (f * h)
        lim[t] = np.abs(b[l]) @ (abs(f) * (eh + 3 * R * 2.0 ** -23 * (np.abs(h) + eh)))
    return d, lim
