"""Every 4-bit code of a layer's weights, one at a time, on the GPU: tokens with a
single element and matrices with a single element a row make each element of the
result depend on one code of the matrix under test, whose bytes are random.

Bound: silu in fp32 (2^-20 relative), its product with u rounded to f16 (2^-11),
the result to bf16 (2^-8)."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from mxfp_block_scaled_b200 import mxq

pytestmark = pytest.mark.gpu

REL = 2.0 ** -8 * (1 + 2.0 ** -11) + 2.0 ** -11 + 2.0 ** -19

# (tokens, experts a token, hidden, inter): y added up by the down kernel; half-size CTAs; rows of gate and up, of down
# shared by the warps of full-size CTAs; a warp a task; the shorter ring in either product
SIZES = [(5, 1, 256, 128), (3, 10, 512, 256), (12, 3, 1024, 128), (12, 3, 128, 1024), (64, 2, 1024, 256), (64, 1, 8192, 128),
         (64, 1, 128, 8192)]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def _stack(codes, fmt):
    """nibbles [E, R, C] -> a stack whose scales are all 1."""
    E, R, C = codes.shape
    q = {"codes": (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8).cuda()}
    q["scales"] = torch.full((E, R, C // (16 if fmt == "nvfp4" else 32)), 0x38 if fmt == "nvfp4" else 127, dtype=torch.uint8,
                             device="cuda")
    if fmt == "nvfp4":
        q["s2"] = torch.ones(E, device="cuda")
    return q


def _values(n):
    return ref.E2M1[n & 7] * np.where(n & 8, -1.0, 1.0)


def _run(cols, T, k, H, gu, dn, fmt, want):
    """One-hot tokens of the given channels, T at a time; expert j of each token; y against want[channel] a row."""
    for c0 in range(0, len(cols), T):
        c = cols[c0:c0 + T]
        x = torch.zeros((T, H), dtype=torch.bfloat16)
        x[range(len(c)), c] = 1.0
        ids = torch.arange(k, dtype=torch.int32).repeat(T, 1)
        y = mxq.moe_forward(x.cuda(), ids.cuda(), torch.ones((T, k), device="cuda"), gu, dn, fmt)
        assert int(y["status"].item()) == 0
        ref.close(y["y"][:len(c)], want[c], REL * np.abs(want[c]))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,k,H,I", SIZES)
def test_every_code_of_gate_and_up(T, k, H, I, fmt):
    """Down is a unit matrix of the last expert (0 for the others): y[i] = silu(g_i) u_i of that expert, i < I."""
    g = torch.Generator().manual_seed(H + I)
    n = torch.randint(0, 16, (k, 2 * I, H), generator=g)
    d = torch.zeros((k, H, I), dtype=torch.int64)
    m = min(H, I)
    d[-1, range(m), range(m)] = 2                                   # 1.0
    cols = list(range(H)) if H <= 1024 else list(range(0, H, 37)) + list(range(H - 128, H))
    cols = cols if I <= 512 else cols[:128]
    for half in (0, 1):                 # the other half constant, so that no product hides a code
        w = n.clone()
        w[:, :I] = w[:, :I] if half == 0 else 6                     # 4.0
        w[:, I:] = w[:, I:] if half == 1 else 4                     # 2.0
        a, b = _values(w[-1, :I].numpy()), _values(w[-1, I:].numpy())
        want = np.zeros((H, H))
        want[:, :m] = (a / (1 + np.exp(-a)) * b)[:m].T
        _run(cols, T, k, H, _stack(w, fmt), _stack(d, fmt), fmt, want)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,k,H,I", SIZES)
def test_every_code_of_down(T, k, H, I, fmt):
    """Channel c of a token goes to row c % I of gate and up alone: y is column c % I of down times silu(4) 2."""
    g = torch.Generator().manual_seed(H * I)
    n = torch.randint(0, 16, (k, H, I), generator=g)
    n[:-1] = 0
    w = torch.zeros((k, 2 * I, H), dtype=torch.int64)
    c = torch.arange(H)
    shift = I - H if H < I else 0                                   # the last channels of inter, where there are fewer tokens'
    w[-1, c % I + shift, c], w[-1, I + c % I + shift, c] = 6, 4
    h = 4 / (1 + np.exp(-4.0)) * 2
    want = np.zeros((H, H))
    want[:] = (h * _values(n[-1].numpy()))[:, np.arange(H) % I + shift].T
    _run(list(range(min(H, I))), T, k, H, _stack(w, fmt), _stack(n, fmt), fmt, want)
