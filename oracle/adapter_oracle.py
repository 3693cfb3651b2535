"""fp64 oracle of a shared head with low-rank adapters, one row at a time.
Test infrastructure only; shares nothing with the CUDA path."""
from __future__ import annotations

import numpy as np


def adapter_logits(H, W, A, B, scale, adapter_id):
    """(logits [N, V], magnitude [N, V], bad [N]).  Row i: W h_i + scale[a] B[a] (A[a] h_i);
    -1 is no adapter, any other id outside the arrays is reported and taken as
    none.  ``magnitude``: the sum of the absolute terms, for rounding bounds."""
    H, W, A, B = (np.asarray(x, dtype=np.float64) for x in (H, W, A, B))
    n = H.shape[0]
    out = np.empty((n, W.shape[0]))
    mag = np.empty_like(out)
    bad = np.zeros(n, dtype=bool)
    for i in range(n):
        out[i] = W @ H[i]
        mag[i] = np.abs(W) @ np.abs(H[i])
        a = int(adapter_id[i])
        if 0 <= a < A.shape[0]:
            s = float(scale[a])
            out[i] += s * (B[a] @ (A[a] @ H[i]))
            mag[i] += abs(s) * (np.abs(B[a]) @ (np.abs(A[a]) @ np.abs(H[i])))
        else:
            bad[i] = a != -1
    return out, mag, bad
