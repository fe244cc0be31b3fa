"""Attention over an MXFP8 cache whose values are of very different sizes: what a token's large
block may take from other tokens and other columns, and sums over tokens without values.

Bounds as in test_gpu_attention_numerics.py.  One large block among ordinary tokens: where a
sequence has many rows, of the 64 tokens that are multiplied together with it values may be off
by 2^-36 of it (f16's step, 2^-25 of 57344, and a reference that may stand 2^4 above), and zeros
from 2^-27 of it on."""
import math

import pytest
import torch

import cache_ref as ref
from mxfp_block_scaled_b200 import mxq
from test_gpu_cache import dev32, gen
from test_gpu_attention_numerics import attend, largest_weight, one_sequence, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mxq.load()


def write(cache, k, v, ln, table):
    n = k.shape[0]
    assert mxq.cache_write(cache, k.bfloat16(), v.bfloat16(), dev32([0, n]), ln, table).item() == 0


@pytest.mark.parametrize("new", [1, 5, 80])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("far", [12, 20, 22, 24, 28, 34, 55])
def test_one_large_block_leaves_the_other_columns(far, dim, new):
    """One token's first 32 values are 2^far times as large as all others.  Its own block's
    columns are held to its size; the others to their own, but for its 64 neighbours.  (Heads
    enough that a warp, or a CTA, has most of a head's tokens.)"""
    n, at, heads, group = 4096, 1500, 200 if new <= 5 else 32, 1 if new <= 5 else 4
    cache, ln, table = one_sequence("mxfp8", n, dim, heads=heads)
    k, v = (torch.randn((n, 1, dim), generator=gen(3 + i), device="cuda") for i in range(2))
    v = v.abs() + 0.5           # outputs of the size of the values
    v[at, 0, :32] *= 2.0 ** far
    write(cache, k.expand(n, heads, dim).contiguous(), v.expand(n, heads, dim).contiguous(), ln, table)
    q = torch.randn((new, heads * group, dim), generator=gen(5), device="cuda").bfloat16()
    scale = dim ** -0.5
    r = attend(cache, q, ln, table, scale)
    k, v = (t[:, 0] for t in ref.sequence_values(cache, 0, ln, table))
    s = scale * torch.einsum("ihd,jd->ihj", q.double(), k)
    pos = n - new + torch.arange(new, device="cuda")
    s.masked_fill_((torch.arange(n, device="cuda")[None] > pos[:, None])[:, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    p = s.sub_(lse[..., None]).exp_()
    o, weight = p @ v, p @ v.abs()
    eps = 2 * (dim + 8) * 2.0 ** -23 * scale * (q.double().abs() @ k.abs().t()).amax(-1)
    out, size = v[at].abs().max(), v.abs().amax(0)
    near_keys = slice(at // 64 * 64, at // 64 * 64 + 64)
    largest = p.amax(-1)[..., None]
    bound = 1.01 * (o.abs() * 2.0 ** -8 + weight * (2.0 ** -11 + eps[..., None] + 2.0 ** -18) * (1 + 2.0 ** -8)) \
        + largest * n * 2.0 ** -32 * size + 1e-30
    if new > 5:
        for j in range(near_keys.start, near_keys.stop):
            lost = 2.0 ** -36 if far < 20 else 2.0 ** -26       # (scales are powers of two)
            bound += p[..., j:j + 1] * torch.minimum(v[j].abs(), lost * out)
    worst = ((r["o"].double() - o).abs() / bound)
    assert worst.max().item() <= 1, (worst[..., :32].max().item(), worst[..., 32:].max().item())
    assert ((r["lse"].double() - lse).abs() <= eps + 2.0 ** -18 + lse.abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("new", [1, 80])
@pytest.mark.parametrize("step", [0.0, 5.4, 10.3])
def test_scores_that_rise_over_tokens_without_values(step, new):
    """Values of zero, and scores of which every second 128 lie `step` above the others, as far
    as a running maximum may lag: lse counts every token."""
    n, dim = 3 << 20, 64
    cache, ln, table = one_sequence("mxfp8", n, dim, tokens=256)
    k = torch.zeros((n, 1, dim), dtype=torch.bfloat16, device="cuda")
    k[torch.arange(n, device="cuda") // 128 % 2 == 1] = 1.0
    write(cache, k, torch.zeros_like(k), ln, table)
    q = torch.zeros((new, 2, dim), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    r = attend(cache, q, ln, table, step)
    seen = torch.cumsum(k[:, 0, 0].double(), 0)[n - new:, None]
    want = torch.log(n - new + 1 + torch.arange(new, device="cuda")[:, None] - seen + seen * math.exp(step))
    assert (r["o"] == 0).all()
    assert ((r["lse"].double() - want).abs() <= 2.0 ** -17 + want * 2.0 ** -22).all(), (r["lse"][0], want[0])


@pytest.mark.parametrize("new", [1, 80])
@pytest.mark.parametrize("run", [32, 64, 640])
@pytest.mark.parametrize("far", [10, 50, 100])
def test_tokens_without_values_beside_large_ones_count(far, run, new):
    """Runs of tokens whose values are zeros, and runs of tokens whose values are 2^far: both
    are in the sum of the weights."""
    n, dim = 2560, 128
    cache, ln, table = one_sequence("mxfp8", n, dim)
    k = torch.randn((n, 1, dim), generator=gen(1), device="cuda")
    v = torch.full((n, 1, dim), 2.0 ** far, device="cuda")
    v[torch.arange(n, device="cuda") // run % 2 == 0] = 0
    write(cache, k, v, ln, table)
    q = torch.randn((new, 4, dim), generator=gen(5), device="cuda").bfloat16()
    scale = dim ** -0.5
    r = attend(cache, q, ln, table, scale)
    o, lse, weight, spread = ref.attention(cache, q, [0, new], ln.tolist(), table, scale)
    eps = 2 * (dim + 8) * 2.0 ** -23 * spread
    largest = largest_weight(cache, q, ln, table, scale, lse)
    bound = 1.01 * (o.abs() * 2.0 ** -8 + weight * (2.0 ** -11 + eps[..., None] + 2.0 ** -18) * (1 + 2.0 ** -8)) \
        + n * 2.0 ** -32 * largest[..., None] * 2.0 ** far
    assert ((r["o"].double() - o).abs() <= bound).all()
    assert ((r["lse"].double() - lse).abs() <= eps + 2.0 ** -18 + lse.abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 4, 2000])
def test_values_that_grow_and_fall(new, dim):
    """Sizes from 2^-25 to 2^25 and back along the sequence, blocks of a head out of step with one
    another; prompts whose rows end anywhere, with heads enough that a CTA passes many steps."""
    n, heads = 2000, 64 if new > 4 else 400
    cache, ln, table = one_sequence("mxfp8", n, dim, heads=heads)
    k, v = (torch.randn((n, 1, dim), generator=gen(3 + i), device="cuda") for i in range(2))
    at = torch.arange(n, device="cuda")[:, None, None]
    blocks = torch.arange(dim, device="cuda") // 32
    v = (v.abs() + 0.5) * torch.exp2(torch.round(25 * torch.sin(at * (2 * math.pi / 700)) + 4 * torch.sin(at / 40 + 2 * blocks)))
    write(cache, k.expand(n, heads, dim).contiguous(), v.expand(n, heads, dim).contiguous(), ln, table)
    q = torch.randn((new, heads, dim), generator=gen(5), device="cuda").bfloat16()
    scale = dim ** -0.5
    r = attend(cache, q, ln, table, scale)
    k, v = (t[:, 0] for t in ref.sequence_values(cache, 0, ln, table))
    near = torch.nn.functional.pad(v.abs().amax(1), (0, -n % 64)).view(-1, 64).amax(1).repeat_interleave(64)[:n, None]
    seen = torch.arange(n, device="cuda")[None] <= n - new + torch.arange(new, device="cuda")[:, None]
    for h in (0, 1, heads // 2, heads - 1):
        x = q[:, h].double()
        s = (scale * x @ k.t()).masked_fill(~seen, -math.inf)
        lse = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[:, None])
        eps = 2 * (dim + 8) * 2.0 ** -23 * scale * (x.abs() @ k.abs().t()).amax(-1)
        o = p @ v
        bound = 1.01 * o * (2.0 ** -8 + (2.0 ** -11 + eps[:, None] + 2.0 ** -18) * (1 + 2.0 ** -8)) \
            + 2.0 ** -36 * p @ near + 2.0 ** -32 * p.amax(-1, keepdim=True) * (seen.double() @ v) + 1e-30
        worst = ((r["o"][:, h].double() - o).abs() / bound).max().item()
        assert worst <= 1, (h, worst)
        assert ((r["lse"][:, h].double() - lse).abs() <= eps + 2.0 ** -18 + lse.abs() * 2.0 ** -22).all()
