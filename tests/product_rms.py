"""How far an fp32 result of the block-FP8 product may be off in the root mean square, from the definition's block sums.

For long K the elementwise bound (layer_ref.gemm: every rounding at its worst and in one direction) leaves room for
block sums of far fewer bits.  Here a block's own error is still taken at its worst, 128 additions of up to 2^-23 of
the sum M of its products' magnitudes, and 2^-24 each for its scale's product and for the addition to the sum so far;
but the blocks' errors are taken as independent, operands of either sign given, so that their squares add up."""
import numpy as np

import layer_ref as ref


def block_sums(a, sa, b, sb):
    """Scaled sums of the blocks and of their products' magnitudes, [KB, M, N] each, in binary64."""
    A, B = ref.E4M3[a], ref.E4M3[b]
    K, row = A.shape[1], np.arange(B.shape[0]) // 128
    P, M = [], []
    for kb, k in enumerate(range(0, K, 128)):
        s = sa[:, kb, None].astype(np.float64) * sb[row, kb].astype(np.float64)[None]
        P.append(A[:, k:k + 128] @ B[:, k:k + 128].T * s)
        M.append(np.abs(A[:, k:k + 128]) @ np.abs(B[:, k:k + 128]).T * np.abs(s))
    return np.stack(P), np.stack(M)


def bound(P, M):
    acc = np.cumsum(P, 0)
    return np.sqrt(((128 * 2.0 ** -23 * M) ** 2 + (2.0 ** -24 * P) ** 2 + (2.0 ** -24 * acc) ** 2).sum(0).mean())


def rms(x):
    return np.sqrt((np.asarray(x, np.float64) ** 2).mean())
