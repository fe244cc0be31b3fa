"""Plain binary64 forms of the layer operators, for the tests: decoding of
block-scaled codes, the block-FP8 quantizer, the product and the
mixture-of-experts layer, each with a bound on what the kernels' roundings may
add.  Written from the definitions; shares no code with the library.

Roundings counted (u = half a step, relative): bf16 2^-8, f16 2^-11, fp32
2^-24.  A sum of n fp32 terms is off by at most n 2^-23 sum |term| (one
rounding or truncation an addition, and one for each product's scale)."""
import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e4m3_table():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if c & 127 == 127 else (-x if c & 128 else x)
    return v


E4M3 = e4m3_table()
GRID = E4M3[:127]           # magnitudes of the codes 0 .. 126, ascending


def e4m3_encode(y):
    """Nearest E4M3 code of each value (ties to the even code, saturating)."""
    a = np.abs(y.astype(np.float64))
    hi = np.clip(np.searchsorted(GRID, a), 1, 126)
    lo = hi - 1
    d = (GRID[hi] - a) - (a - GRID[lo])
    mag = np.where(d < 0, hi, np.where(d > 0, lo, np.where(lo % 2 == 0, lo, hi)))
    mag = np.where(a >= 448, 126, mag)
    return (mag | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantize_fp8(x, brows):
    """x: fp32 numpy [R, C] -> codes, scales by the definition."""
    R, C = x.shape
    nbr, nbc = -(-R // brows), -(-C // 128)
    codes, scales = np.zeros((R, C), np.uint8), np.zeros((nbr, nbc), np.float32)
    for i in range(nbr):
        for j in range(nbc):
            cut = np.s_[i * brows:(i + 1) * brows, j * 128:(j + 1) * 128]
            b = x[cut]
            s = np.float32(np.abs(b).max()) / np.float32(448)
            scales[i, j] = s
            if s > 0:
                codes[cut] = e4m3_encode(b / s)
    return codes, scales


def spread(s, brows, R, C):
    return np.repeat(np.repeat(s, brows, 0)[:R], 128, 1)[:, :C]


def decode(codes, scales, s2, fmt):
    """One expert's matrix in binary64 (numpy)."""
    if fmt in ("nvfp4", "mxfp4"):
        n = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
        v = E2M1[n & 7] * np.where(n & 8, -1.0, 1.0)
    else:
        v = E4M3[codes]
    if fmt == "fp8_block":
        return v * spread(scales.astype(np.float64), 128, *v.shape)
    if fmt == "nvfp4":
        d = E4M3[scales] * float(s2)
    else:
        d = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return v * np.repeat(d, v.shape[1] // d.shape[1], 1)


def moe(x, ids, w, gate_up, down, fmt):
    """(y, bound) in binary64: the layer's result and how far the kernels may be off."""
    to = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    x64, w = x.cpu().double().numpy(), to(w).astype(np.float64)
    ids = to(ids)
    gu = [to(gate_up["codes"]), to(gate_up["scales"]), to(gate_up.get("s2"))]
    dn = [to(down["codes"]), to(down["scales"]), to(down.get("s2"))]
    T, H = x64.shape
    y, err, mag = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    E = gu[0].shape[0]
    for e in sorted(set(ids.ravel().tolist())):
        if e < 0 or e >= E:
            continue
        G = decode(gu[0][e], gu[1][e], None if gu[2] is None else gu[2][e], fmt)
        D = decode(dn[0][e], dn[1][e], None if dn[2] is None else dn[2][e], fmt)
        I = D.shape[1]
        for t, j in zip(*np.nonzero(ids == e)):
            a = G @ x64[t]
            da = (H * 2.0 ** -23 * (np.abs(G) @ np.abs(x64[t])) + np.abs(G).sum(1) * np.abs(x64[t]).max() * 2.0 ** -39
                  + 2.0 ** -22 * np.abs(a))
            g, u = a[:I], a[I:]
            sig = np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))
            h = g * sig * u
            # |silu'| <= 1.1; expf, the division and the product: 2^-20 relative
            dh = 1.1 * np.abs(u) * da[:I] + np.abs(g * sig) * da[I:] + 1.1 * da[:I] * da[I:] + 2.0 ** -20 * np.abs(h)
            hm = (np.abs(h) + dh).max()
            dh = dh + 2.0 ** -11 * (np.abs(h) + dh) + hm * 2.0 ** -39          # rounded to f16
            z = D @ h
            y[t] += w[t, j] * z
            err[t] += abs(w[t, j]) * (np.abs(D) @ dh + I * 2.0 ** -23 * (np.abs(D) @ np.abs(h)) + 2.0 ** -22 * np.abs(z))
            mag[t] += abs(w[t, j]) * np.abs(z)
    err += ids.shape[1] * 2.0 ** -23 * mag                                     # the sum over the experts
    return y, err + 2.0 ** -8 * (np.abs(y) + err) + 2.0 ** -126                # rounded to bf16


def gemm(a, sa, b, sb, out):
    """(c, bound): a [M, K] codes with scales [M, ceil(K/128)], b [N, K] with [ceil(N/128), ceil(K/128)]."""
    A = E4M3[a] * spread(sa.astype(np.float64), 1, *a.shape)
    B = E4M3[b] * spread(sb.astype(np.float64), 128, *b.shape)
    c, mag = A @ B.T, np.abs(A) @ np.abs(B.T)
    err = (a.shape[1] + 4) * 2.0 ** -23 * mag
    return c, err + (2.0 ** -8 if out == "bf16" else 2.0 ** -24) * (np.abs(c) + err) + 2.0 ** -126


def close(got, want, bound):
    """Every element inside its bound; NaN where NaN is wanted."""
    got = got.double().cpu().numpy() if torch.is_tensor(got) else got
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    bad = np.abs(got - want)[~nan] > bound[~nan]
    assert not bad.any(), "%d of %d outside, worst %.3g of its bound" % (
        bad.sum(), bad.size, np.nanmax((np.abs(got - want) / bound)))
