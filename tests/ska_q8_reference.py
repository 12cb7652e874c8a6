"""The 8-bit ring cache from its definition, one sequence and one token at a
time, in float64 on the CPU: rounding of blocks, the state that tokens leave,
and the attention over it.

Bound of an output element: half a bf16 step, 2^-8 |r|, plus float32 arithmetic.
Scores stay below 16 (in powers of two); a sum of d <= 128 products, each rounded
by 2^-24 of at most that, has with random signs an error of about 16 sqrt(128)
2^-24 = 2^-16.5, and the exponentials, the weights' split into halves and the sum
of the weights add 2^-21 each.  An output is a mean of the values under such
weights: 2^-15 of the largest value (twice the standard error and more)."""
import math

import torch


def round_block(rows, kind):
    """(codes, scale) of one block's rows [n,d], both float64."""
    x = rows.double()
    finite = torch.isfinite(x)
    most = torch.where(finite, x.abs(), torch.zeros_like(x)).max().item()
    if kind == torch.int8:
        scale = (torch.tensor(most, dtype=torch.float32) / torch.tensor(127.0)).item() if most else 1.0
        q = torch.round(rows.float() / torch.tensor(scale, dtype=torch.float32))  # float32 division: part of the format
        q = torch.where(torch.isnan(q), torch.zeros_like(q), q.clamp(-127, 127))
        return q.double(), scale
    scale = 1.0
    if most:
        e = math.frexp(most / 448)  # most / 448 = m 2^e, 1/2 <= m < 1: the power of two at or above it
        scale = 2.0 ** max(-126, e[1] - 1 if e[0] == 0.5 else e[1])
    v = x / scale
    grid = 2.0 ** (torch.clamp(torch.floor(torch.log2(v.abs().clamp(min=1e-300))), min=-6.0) - 3)
    q = torch.where(torch.isinf(v), torch.sign(v) * 448, torch.round(v / grid) * grid)
    return q, scale


class Cache:
    """One sequence's cache: H + 1 rows of heads, the first the shared key's."""

    def __init__(self, H, dk, dv, window, block, kind):
        self.H, self.w, self.R, self.kind, self.pos = H, window, block, kind, 0
        nb = -(-window // block)
        self.codes = [torch.zeros(window, d).double() for d in [dk] + [dv] * H]
        self.scale = [torch.ones(nb).double() for _ in range(H + 1)]
        self.tail = [torch.zeros(block, d).double() for d in [dk] + [dv] * H]

    def add(self, k, v):
        """One token's key [dk] and values [H,dv]; the rows to attend to, before the block is rounded."""
        slot = self.pos % self.w
        blk, i = divmod(slot, self.R)
        n = min(self.pos + 1, self.w)
        held = []
        for h, x in enumerate([k] + list(v)):
            self.tail[h][i] = x.double()
            rows = self.codes[h][:n] * self.scale[h].repeat_interleave(self.R)[:n, None]
            rows[blk * self.R:slot + 1] = self.tail[h][:i + 1]
            held.append(rows)
            if i == self.R - 1 or slot == self.w - 1:
                q, s = round_block(self.tail[h][:i + 1].to(torch.bfloat16), self.kind)
                self.codes[h][blk * self.R:slot + 1] = q
                self.scale[h][blk] = s
        self.pos += 1
        return held

    def attend(self, q, held, scale):
        p = torch.softmax(q.double() @ held[0].t() * scale, -1)
        return torch.stack([p[h] @ held[1 + h] for h in range(self.H)])


def state(caches):
    """k_cache, v_cache, k_scale, v_scale, k_tail, v_tail, pos of a batch, float64."""
    return (torch.stack([c.codes[0] for c in caches]), torch.stack([torch.stack(c.codes[1:]) for c in caches]),
            torch.stack([c.scale[0] for c in caches]), torch.stack([torch.stack(c.scale[1:]) for c in caches]),
            torch.stack([c.tail[0] for c in caches]), torch.stack([torch.stack(c.tail[1:]) for c in caches]),
            torch.tensor([c.pos for c in caches]).double())


def assert_state(cache, caches, what):
    """Bit by bit; of the tails, the rows that hold a token of an unfinished block
    (the others mean nothing)."""
    live = torch.zeros(len(caches), caches[0].R, 1)
    for b, c in enumerate(caches):
        slot = (c.pos - 1) % c.w
        if c.pos and slot % c.R != c.R - 1 and slot != c.w - 1:
            live[b, :slot % c.R + 1] = 1
    for name, got, want in zip(("k_cache", "v_cache", "k_scale", "v_scale", "k_tail", "v_tail", "pos"), cache, state(caches)):
        got = got.float().cpu().double()
        if "tail" in name:
            rows = (live if name == "k_tail" else live[:, None]) > 0
            got, want = torch.where(rows, got, torch.zeros_like(got)), torch.where(rows, want, torch.zeros_like(want))
        assert torch.equal(got, want), f"{what}: {name}"


def assert_out(o, want, largest, what):
    o = o.cpu().double()
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -15 * largest
    assert torch.isfinite(o).all(), what
    worst = ((o - want).abs() / bound).max().item()
    assert worst <= 1, f"{what}: {worst:.2f} of the bound"
