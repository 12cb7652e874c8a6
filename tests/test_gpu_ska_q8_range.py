"""GPU tests of the 8-bit ring cache's decode over the range of its values: very
small ones, blocks and heads of zeros, a heavy token whose value is small (an
attention sink), blocks of unlike scales, in windows that one CTA takes and in
windows that are split.

Bound of an output element, with p the softmax weights and n the slots:
  2^-8 |o|                   half a bf16 step
  2^-15 sum_u p_u |v_u|      float32 arithmetic.  A weight's score (below 48 in
                             powers of two, and a sum of up to 64 products only
                             below 16) is off by at most 2^-16.5 of a power of two,
                             2^-17 of the weight; exponential, logarithm of the
                             scale and the split add 2^-22 each; the sum of the
                             weights as much again; and twice that.
  n 2^-50 max_u p_u amax_u   amax_u the largest magnitude of u's block: the parts of
                             a weight end 2^-51 below the heaviest weight times
                             scale, and a code is below the block's amax / scale.
It is relative to what the output is made of, so it does not grow with values
that have no weight."""
import math

import pytest
import torch

import gated_linear_attention_ddts_b200 as rdm
from tests import ska_q8_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
KINDS = [torch.float8_e4m3fn, torch.int8]


def resident(K, V, pos, block, kind):
    """One sequence's cache before the token at `pos` (at least one round on): slot u
    holds K[u], V[:, u], those of the unfinished block before `pos` in the tail."""
    H, w, dv = V.shape
    c = ref.Cache(H, K.shape[1], dv, w, block, kind)
    c.pos = pos
    assert pos >= w
    cur = pos % w
    for h, x in enumerate([K, *V]):
        for i, at in enumerate(range(0, w, block)):
            c.codes[h][at:at + block], c.scale[h][i] = ref.round_block(x[at:at + block], kind)
        at = cur // block * block
        c.tail[h][:cur - at] = x[at:cur].double()
    return c


def check(c, q, k, v, scale, what, **kw):
    """The token (k, v) after the cache `c`, on the GPU and in the reference."""
    cache = [t.float().to(ty).cuda() for t, ty in zip(ref.state([c]), (c.kind, c.kind, torch.float32, torch.float32, BF16, BF16, torch.int32))]
    o = rdm.rdm_ska_q8_decode(q[None].cuda(), k[None].cuda(), v[None].cuda(), *cache, scale=scale, **kw)[0].cpu().double()
    blocks = [torch.stack([(c.codes[h][a:a + c.R].abs().max() * c.scale[h][a // c.R]) for a in range(0, c.w, c.R)]) for h in range(1, c.H + 1)]
    held = c.add(k, v)
    p = torch.softmax(q.double() @ held[0].t() * scale, -1)
    want = torch.stack([p[h] @ held[1 + h] for h in range(c.H)])
    mean = torch.stack([p[h] @ held[1 + h].abs() for h in range(c.H)])
    heavy = torch.stack([(p[h] * blocks[h].repeat_interleave(c.R)[:p.shape[1]]).max() for h in range(c.H)])
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -15 * mean + c.w * 2.0 ** -50 * heavy[:, None]
    assert torch.isfinite(o).all(), what
    worst = ((o - want).abs() / bound.clamp(min=1e-300)).max().item()
    assert worst <= 1, f"{what}: {worst:.3g} of the bound"
    assert rdm.rdm_ddts_sync_status() == 0
    ref.assert_state(cache, [c], what)
    return o


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF16)


# a window that one CTA takes in one piece, one that is split, the same whole
WINDOWS = [(180, {}), (1500, {}), (1500, {"workspace": False})]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,kw", WINDOWS)
@pytest.mark.parametrize("sigma", [1e4, 1.0, 1e-2, 1e-4, 1e-6, 1e-20, 1e-30])
def test_values_of_every_size(cuda_ok, kind, window, kw, sigma):
    c = resident(normal(1, window, 64), normal(2, 3, window, 64) * sigma, 2 * window + 100, 64, kind)
    check(c, normal(3, 3, 64), normal(4, 64), normal(5, 3, 64) * sigma, 1 / 8, f"values of {sigma}", **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,kw", WINDOWS)
@pytest.mark.parametrize("sigma", [1e-4, 1e-20])
@pytest.mark.parametrize("zero", [0.0, -0.0])
def test_small_values_and_an_unfinished_block_of_zeros(cuda_ok, kind, window, kw, sigma, zero):
    V = normal(2, 2, window, 128) * sigma
    cur = (2 * window + 100) % window
    V[:, cur // 32 * 32:cur] = zero
    c = resident(normal(1, window, 64), V, 2 * window + 100, 32, kind)
    check(c, normal(3, 2, 64), normal(4, 64), torch.full((2, 128), zero, dtype=BF16), 1 / 8, "tail of zeros", **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,kw", WINDOWS)
@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("sigma", [1e-4, 1e-20])
@pytest.mark.parametrize("zero", [0.0, -0.0])
def test_small_values_beside_blocks_of_zeros(cuda_ok, kind, window, kw, block, sigma, zero):
    """A block of zeros has the scale 1, which says nothing of the others; the last,
    short block is one, and (window 1500) all the slots of some splits."""
    V = normal(6, 2, window, 64) * sigma
    V[:, 16:80] = zero
    V[0, window // block * block:] = zero
    V[1, window // 3:window // 3 * 2] = zero
    c = resident(normal(7, window, 128), V, 3 * window + 2, block, kind)
    check(c, normal(8, 2, 128), normal(9, 128), normal(10, 2, 64) * sigma, 1 / 11, "blocks of zeros", **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,kw", WINDOWS)
def test_head_of_zeros(cuda_ok, kind, window, kw):
    V = normal(11, 3, window, 64)
    V[1] = 0
    v = normal(14, 3, 64)
    c = resident(normal(12, window, 64), V, window + 40, 64, kind)
    o = check(c, normal(13, 3, 64), normal(15, 64), torch.stack([v[0], 0 * v[1], v[2]]), 1 / 8, "head of zeros", **kw)
    assert not o[1].any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", [{}, {"workspace": False}])
@pytest.mark.parametrize("nats", [10, 14, 17, 20, 24])
@pytest.mark.parametrize("where", ["block", "tail", "new"])
def test_heavy_token_with_a_small_value(cuda_ok, kind, kw, nats, where):
    """One token `nats` above 32767 others that are all alike in score: in a block
    beside values of the usual size, in the unfinished block, or the new one.  One
    dimension makes the scores, the others of q are zero.  Head 0's heavy value is
    zero, head 1's 2^-20."""
    w, scale = 32768, 1 / 8
    pos = w + 20000
    K, V = normal(16, w, 64), normal(17, 2, w, 64)
    V[1] = V[1].abs() + 1  # one sign: nothing averages out
    k, v = normal(18, 64), normal(19, 2, 64).abs()
    K[:, 0], k[0] = 0.0, 0.0
    q = torch.zeros(2, 64, dtype=BF16)
    q[:, 0] = 8.0
    at = {"block": 777, "tail": pos % w - 3, "new": None}[where]
    heavy = torch.tensor([0.0, 2.0 ** -20])
    if at is None:
        k[0], v[:] = float(nats), heavy[:, None].to(BF16)
    else:
        K[at, 0], V[:, at] = float(nats), heavy[:, None].to(BF16)
    c = resident(K, V, pos, 32, kind)
    check(c, q, k, v, scale, f"{nats} nats", **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("slot", [0, 33, 700, 1203, 2047])
@pytest.mark.parametrize("falling", [False, True])
def test_scales_that_rise_and_fall_over_the_window(cuda_ok, kind, slot, falling):
    """Values from 1e-25 to 1e5 along a window of four chunks that one CTA takes,
    scores that rise or fall against them, the unfinished block in each chunk."""
    w = 2048
    up = torch.linspace(-25, 5, w)
    V = (normal(20, 2, w, 64).float() * (10.0 ** (up.flip(0) if falling else up))[:, None]).to(BF16)
    K = normal(21, w, 64)
    K[:, 0] = (-up.flip(0) if falling else -up) / 2
    q = torch.zeros(2, 64, dtype=BF16)
    q[:, 0] = 2.0
    v = normal(24, 2, 64) * 1e-10
    check(resident(K, V, 2 * w + slot, 64, kind), q, normal(23, 64), v, 1.0, f"slot {slot}", workspace=False)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,kw", WINDOWS)
@pytest.mark.parametrize("half", [False, True])
def test_blocks_whose_scale_is_one(cuda_ok, kind, window, kw, half):
    """Blocks that begin with zeros and have the scale 1 for their largest value's
    sake, beside blocks of zeros or not."""
    V = normal(25, 2, window, 128).clamp(-3, 3)
    V[:, ::64, :64] = 0
    V[:, 5::64, 77] = 127.0 if kind == torch.int8 else 448.0
    if half:
        V[:, :window // 128 * 64] = 0
    c = resident(normal(26, window, 64), V, window + 90, 64, kind)
    assert c.scale[1][:window // 64].eq(1).all()
    check(c, normal(27, 2, 64), normal(28, 64), normal(29, 2, 128), 1 / 8, "scale 1", **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [1, 40, 64, 700])
@pytest.mark.parametrize("sigma", [1e-4, 1e-20])
def test_small_values_in_the_first_round(cuda_ok, kind, tokens, sigma):
    """Slots behind the last token hold codes of a large scale or zeros with the scale
    1; neither counts."""
    K, V = normal(30, 1000, 64), normal(31, 2, 1000, 64) * sigma
    V[:, 320:384] = 0
    c = ref.Cache(2, 64, 64, 1000, 64, kind)
    for t in range(tokens):
        c.add(K[t], V[:, t])
    for h in (1, 2):
        c.codes[h][-200:], c.scale[h][-3:] = 100.0 if kind == torch.int8 else 240.0, 2.0 ** 20
    check(c, normal(32, 2, 64), normal(33, 64), normal(34, 2, 64) * sigma, 1 / 8, f"{tokens} tokens")
