"""GPU tests of the 8-bit ring cache through the public entry points against the
float64 reference (tests/ska_q8_reference.py): the cache bit by bit, the outputs
within half a bf16 step and float32 arithmetic."""
import math

import pytest
import torch

import gated_linear_attention_ddts_b200 as rdm
from tests import ska_q8_reference as ref
from tests import ssm_reference

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
KINDS = [torch.float8_e4m3fn, torch.int8]


def tokens(B, H, T, dk, dv, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, H, T, dk, generator=g).to(BF16), torch.randn(B, T, dk, generator=g).to(BF16),
            torch.randn(B, H, T, dv, generator=g).to(BF16))


def filled(k, v, window, block, kind, lengths=None):
    """(the GPU's cache, the reference's caches) after a prompt."""
    B, H, T, dv = v.shape
    cache = rdm.rdm_ska_q8_cache(B, H, k.shape[2], dv, window, block=block, dtype=kind)
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda") if lengths else None
    rdm.rdm_ska_q8_fill(k.cuda(), v.cuda(), *cache, lengths=ln)
    caches = []
    for b in range(B):
        c = ref.Cache(H, k.shape[2], dv, window, block, kind)
        for t in range(lengths[b] if lengths else T):
            c.add(k[b, t], v[b, :, t])
        caches.append(c)
    return cache, caches


def step(q, k, v, cache, caches, scale=0.0, what="", **kw):
    """One token of each sequence on the GPU and in the reference."""
    largest = max(v.double().abs().max().item(),
                  *((c.codes[h] * c.scale[h].repeat_interleave(c.R)[:c.w, None])[:c.pos].abs().max().item() for c in caches if c.pos for h in range(1, c.H + 1)), 0.0)
    o = rdm.rdm_ska_q8_decode(q.contiguous().cuda(), k.contiguous().cuda(), v.contiguous().cuda(), *cache, scale=scale, **kw)
    want = torch.stack([c.attend(q[b], c.add(k[b], v[b]), scale or 1 / math.sqrt(q.shape[-1])) for b, c in enumerate(caches)])
    ref.assert_out(o, want, largest, what)
    return o


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,block,T", [(1, 16, 3), (5, 16, 1), (16, 16, 16), (40, 16, 39), (40, 16, 40), (40, 16, 47), (40, 16, 95), (64, 32, 130),
                                            (100, 64, 99), (130, 64, 400), (300, 32, 37)])
def test_fill(cuda_ok, kind, window, block, T):
    _, k, v = tokens(2, 3, T, 64, 128, seed=window + T)
    cache, caches = filled(k, v, window, block, kind)
    assert rdm.rdm_ddts_sync_status() == 0
    ref.assert_state(cache, caches, "after the prompt")


@pytest.mark.parametrize("kind", KINDS)
def test_fill_ragged(cuda_ok, kind):
    lengths = [90, 0, 1, 16, 33, 40, 41, 79]
    _, k, v = tokens(8, 2, 90, 128, 64, seed=2)
    ref.assert_state(*filled(k, v, 40, 16, kind, lengths), "ragged prompt")


@pytest.mark.parametrize("lengths,clamped", [([-1, 5], [0, 5]), ([20, 21], [20, 20])])
def test_fill_length_out_of_range(cuda_ok, lengths, clamped):
    _, k, v = tokens(2, 1, 20, 64, 64, seed=3)
    cache = rdm.rdm_ska_q8_cache(2, 1, 64, 64, 32, block=16)
    rdm.rdm_ska_q8_fill(k.cuda(), v.cuda(), *cache, lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    assert rdm.rdm_ddts_sync_status() == rdm.RDM_ERR_INVALID_ARG
    _, caches = filled(k, v, 32, 16, torch.float8_e4m3fn, clamped)
    ref.assert_state(cache, caches, "clamped")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("window,block", [(1, 16), (20, 16), (37, 32), (64, 64)])
def test_decode_from_nothing(cuda_ok, kind, dk, dv, window, block):
    """Token by token from an empty cache, around the ring more than twice."""
    T = min(2 * window + 3, 90)
    q, k, v = tokens(2, 3, T, dk, dv, seed=dk + dv + window)
    cache = rdm.rdm_ska_q8_cache(2, 3, dk, dv, window, block=block, dtype=kind)
    caches = [ref.Cache(3, dk, dv, window, block, kind) for _ in range(2)]
    for t in range(T):
        step(q[:, :, t], k[:, t], v[:, :, t], cache, caches, what=f"token {t}")
    assert rdm.rdm_ddts_sync_status() == 0
    ref.assert_state(cache, caches, "after the last token")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H", [1, 2, 3, 4, 7, 8, 12, 16, 24])
def test_heads_and_positions(cuda_ok, kind, H):
    """Sequences at different places of the ring, then twenty tokens."""
    lengths = [3, 150, 211, 64]
    q, k, v = tokens(4, H, 240, 64, 64, seed=H)
    cache, caches = filled(k[:, :211], v[:, :, :211], 150, 32, kind, lengths)
    for t in range(211, 231):
        step(q[:, :, t], k[:, t], v[:, :, t], cache, caches, what=f"token {t}")
    ref.assert_state(cache, caches, "after the last token")


@pytest.mark.parametrize("B,H,d", [(296, 2, 64), (296, 3, 64), (296, 4, 64), (296, 5, 64), (296, 6, 64), (296, 7, 64), (296, 8, 64),
                                   (148, 9, 64), (140, 11, 64), (148, 16, 64), (296, 8, 128)])
def test_large_batches(cuda_ok, B, H, d):
    """Batches so large that a block takes two to eight heads of a sequence, the last
    group of a sequence fewer; sequences at every place of the ring."""
    q, k, v = tokens(B, H, 44, d, d, seed=B + H)
    lengths = [b % 40 + 1 for b in range(B)]
    kind = KINDS[H % 2]
    cache, caches = filled(k[:, :40], v[:, :, :40], 25, 16, kind, lengths)
    for t in range(40, 44):
        step(q[:, :, t], k[:, t], v[:, :, t], cache, caches, what=f"token {t}")
    ref.assert_state(cache, caches, "after the last token")


@pytest.mark.parametrize("B,H", [(10, 16), (20, 16), (40, 12)])
def test_long_windows_of_batches(cuda_ok, B, H):
    """Split windows with groups of two, four and more heads."""
    q, k, v = tokens(B, H, 560, 64, 64, seed=B)
    cache, caches = filled(k[:, :557], v[:, :, :557], 550, 64, KINDS[B // 10 % 2], [557 - 30 * (b % 9) for b in range(B)])
    for t in range(557, 560):
        step(q[:, :, t], k[:, t], v[:, :, t], cache, caches, what=f"token {t}")
    ref.assert_state(cache, caches, "after the last token")


@pytest.mark.parametrize("H", [65, 67, 72])
def test_more_heads_than_a_cluster(cuda_ok, H):
    """More than eight groups of heads: the positions are advanced by a kernel of
    their own."""
    q, k, v = tokens(2, H, 70, 64, 64, seed=H)
    cache, caches = filled(k[:, :60], v[:, :, :60], 48, 16, torch.int8, [60, 31])
    for t in range(60, 64):
        step(q[:, :, t], k[:, t], v[:, :, t], cache, caches, what=f"token {t}")
    ref.assert_state(cache, caches, "after the last token")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,H,window,block,T", [(1, 4, 5000, 64, 5203), (2, 1, 3001, 16, 2900), (1, 16, 1500, 32, 1490), (1, 9, 2048, 64, 2048)])
def test_long_windows(cuda_ok, kind, B, H, window, block, T):
    """Windows that one CTA does not take alone, with and without a workspace."""
    q, k, v = tokens(B, H, T + 3, 128, 128, seed=window)
    cache, caches = filled(k[:, :T], v[:, :, :T], window, block, kind)
    for t in range(T, T + 3):
        step(q[:, :, t], k[:, t], v[:, :, t], cache, caches, what=f"token {t}", **({"workspace": False} if t == T + 1 else {}))
    ref.assert_state(cache, caches, "after the last token")


@pytest.mark.parametrize("kind", KINDS)
def test_largest_window(cuda_ok, kind):
    """32768 slots, rounded codes drawn at random; the last slot is the new one."""
    w, d = 32768, 64
    g = torch.Generator().manual_seed(4)
    c = ref.Cache(2, d, d, w, 64, kind)
    c.pos = 3 * w - 1
    for h in range(3):
        codes = torch.randint(-127, 128, (w, d), generator=g)
        c.codes[h] = codes.double() if kind == torch.int8 else (codes.float() / 16).to(kind).double()
        c.scale[h] = (0.01 + 0.02 * torch.rand(w // 64, generator=g)).double()
        c.tail[h] = torch.randn(64, d, generator=g).to(BF16).double()
    caches = [c]
    s = ref.state(caches)
    cache = [t.float().to(ty).cuda() for t, ty in zip(s, (kind, kind, torch.float32, torch.float32, BF16, BF16, torch.int32))]
    c.scale = [t.float().double() for t in c.scale]
    q, k, v = tokens(1, 2, 1, d, d, seed=6)
    step(q[:, :, 0], k[:, 0], v[:, :, 0], cache, caches, what="last slot")
    ref.assert_state(cache, caches, "last slot")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pos", [0, 5, 15, 16, 40])
def test_slots_never_written_are_not_read(cuda_ok, kind, pos):
    """Codes, scales and tails full of NaN (e4m3) or of the largest codes, where
    no token has been."""
    q, k, v = tokens(2, 3, 41, 64, 64, seed=pos)
    cache = [t for t in rdm.rdm_ska_q8_cache(2, 3, 64, 64, 150, block=16, dtype=kind)]
    for t in cache[:2]:
        t.view(torch.uint8).fill_(0x7f)
    for t in cache[2:6]:
        t.fill_(float("nan"))
    if pos:
        rdm.rdm_ska_q8_fill(k[:, :pos].contiguous().cuda(), v[:, :, :pos].contiguous().cuda(), *cache)
    _, caches = filled(k[:, :pos], v[:, :, :pos], 150, 16, kind) if pos else (None, [ref.Cache(3, 64, 64, 150, 16, kind) for _ in range(2)])
    step(q[:, :, pos], k[:, pos], v[:, :, pos], cache, caches, what=f"position {pos}")


@pytest.mark.parametrize("kind", KINDS)
def test_scales_far_apart_and_sharp_scores(cuda_ok, kind):
    """Blocks of values a million times larger than others, blocks of zeros,
    values near the ends of bf16; scores that leave one token and scores that
    leave all alike."""
    q, k, v = tokens(1, 4, 200, 64, 128, seed=12)
    v[:, :, 16:32] *= 1e6
    v[:, 1, 32:64] = 0
    v[:, 2, 64:80] *= 1e-38
    k[:, 48:64] = 0
    cache, caches = filled(k[:, :199], v[:, :, :199], 180, 16, kind)
    ref.assert_state(cache, caches, "prompt")
    kept = [t.clone() for t in cache]
    import copy
    for scale in (1e-6, 0.05, 0.5):
        cc = copy.deepcopy(caches)
        cache = [t.clone() for t in kept]
        step(q[:, :, 199], k[:, 199], v[:, :, 199], cache, cc, scale=scale, what=f"scale {scale}")


@pytest.mark.parametrize("kind", KINDS)
def test_small_values_beside_a_large_scale(cuda_ok, kind):
    """The block with the large values gets no weight: the others' outputs keep
    their accuracy (relative to their own values)."""
    q, k, v = tokens(1, 2, 100, 64, 64, seed=13)
    q[:] = 0
    q[..., 0] = 8
    k[:, :, 0] = 4.0
    k[:, 16:32, 0] = -60.0  # scores 2^-46 below the others'
    v[:, :, 16:32] *= 1e5
    cache, caches = filled(k[:, :99], v[:, :, :99], 128, 16, kind)
    o = rdm.rdm_ska_q8_decode(q[:, :, 99].contiguous().cuda(), k[:, 99].contiguous().cuda(), v[:, :, 99].contiguous().cuda(), *cache)
    want = torch.stack([c.attend(q[b, :, 99], c.add(k[b, 99], v[b, :, 99]), 1 / 8) for b, c in enumerate(caches)])
    ref.assert_out(o, want, 5.0, "small values")


@pytest.mark.parametrize("kind", KINDS)
def test_blocks_with_values_that_are_not_finite(cuda_ok, kind):
    _, k, v = tokens(1, 1, 16, 64, 64, seed=14)
    v[0, 0, 3, 5], v[0, 0, 4, 6], v[0, 0, 5, 7] = float("inf"), -float("inf"), float("nan")
    cache, caches = filled(k, v, 16, 16, kind)
    assert torch.equal(cache[3].cpu().double(), torch.stack(caches[0].scale[1:])[None])
    got, want = cache[1].float().cpu().double()[0, 0], caches[0].codes[1]
    assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(want, nan=1e9))


def test_negative_position_is_reported(cuda_ok):
    q, k, v = tokens(2, 3, 1, 64, 64, seed=15)
    cache, _ = filled(*tokens(2, 3, 50, 64, 64, seed=16)[1:], 40, 16, torch.int8)
    cache[6][0] = -1
    before = [t.clone() for t in cache]
    rdm.rdm_ska_q8_decode(q[:, :, 0].contiguous().cuda(), k[:, 0].contiguous().cuda(), v[:, :, 0].contiguous().cuda(), *cache)
    assert rdm.rdm_ddts_sync_status() == rdm.RDM_ERR_INVALID_ARG
    assert rdm.rdm_ddts_sync_status() == 0
    assert all(torch.equal(a[0], b[0]) for a, b in zip(cache, before))
    assert cache[6].tolist() == [-1, 51]


def test_without_advance_and_given_buffers(cuda_ok):
    q, k, v = tokens(2, 4, 31, 64, 64, seed=17)
    cache, caches = filled(k[:, :30], v[:, :, :30], 64, 16, torch.float8_e4m3fn)
    args = [t.contiguous().cuda() for t in (q[:, :, 30], k[:, 30], v[:, :, 30])]
    o = torch.empty(2, 4, 64, dtype=BF16, device="cuda")
    need = rdm.rdm_ska_q8_decode_workspace_size(*args, *cache)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    first = rdm.rdm_ska_q8_decode(*args, *cache, advance_pos=False, o=o, workspace=ws)
    assert first is o and cache[6].tolist() == [30, 30]
    again = rdm.rdm_ska_q8_decode(*args, *cache, advance_pos=False)
    assert torch.equal(o, again)
    step(q[:, :, 30], k[:, 30], v[:, :, 30], cache, caches, what="then for good")


@pytest.mark.parametrize("B,H,window", [(3, 8, 100), (1, 2, 3000)])
def test_graph_replayed_token_by_token(cuda_ok, B, H, window):
    """A captured step replayed over new tokens in the same buffers, on a side
    stream, across a full block."""
    T0 = window + 5
    q, k, v = tokens(B, H, T0 + 20, 64, 64, seed=18)
    cache, caches = filled(k[:, :T0], v[:, :, :T0], window, 16, torch.float8_e4m3fn)
    kept = [t.clone() for t in cache]
    io = [torch.empty(s, dtype=BF16, device="cuda") for s in ((B, H, 64), (B, 64), (B, H, 64))]
    for t in io:
        t.zero_()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        o = rdm.rdm_ska_q8_decode(*io, *cache)
    for t, was in zip(cache, kept):
        t.copy_(was)
    for t in range(T0, T0 + 20):
        for dst, src in zip(io, (q[:, :, t], k[:, t], v[:, :, t])):
            dst.copy_(src)
        largest = v.double().abs().max().item()
        graph.replay()
        torch.cuda.synchronize()
        want = torch.stack([c.attend(q[b, :, t], c.add(k[b, t], v[b, :, t]), 1 / 8) for b, c in enumerate(caches)])
        ref.assert_out(o, want, largest, f"token {t}")
    ref.assert_state(cache, caches, "after the last token")


def test_two_streams_at_once(cuda_ok):
    """Two caches decoded on two streams, split windows with a workspace each, equal
    the same calls one after the other."""
    q, k, v = tokens(2, 4, 2100, 64, 64, seed=30)
    made = [filled(k[b:b + 1, :2090].contiguous(), v[b:b + 1, :, :2090].contiguous(), 2050, 32, torch.int8)[0] for b in range(2)]
    args = [[t[b:b + 1].contiguous().cuda() for t in (q[:, :, 2090], k[:, 2090], v[:, :, 2090])] for b in range(2)]
    want = [rdm.rdm_ska_q8_decode(*a, *c, advance_pos=False).clone() for a, c in zip(args, made)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for b in range(2):
            got[b].append(rdm.rdm_ska_q8_decode(*args[b], *made[b], advance_pos=False, stream=streams[b]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[b]) for b in range(2) for o in got[b])


def test_same_bits_every_time(cuda_ok):
    q, k, v = tokens(2, 5, 901, 128, 64, seed=19)
    cache, _ = filled(k[:, :900], v[:, :, :900], 800, 64, torch.int8)
    args = [t.contiguous().cuda() for t in (q[:, :, 900], k[:, 900], v[:, :, 900])]
    outs = [rdm.rdm_ska_q8_decode(*args, *cache, advance_pos=False) for _ in range(4)]
    assert all(torch.equal(outs[0], t) for t in outs)


def test_prompt_attention_then_8_bit_tokens(cuda_ok):
    """The prompt through rdm_ska_fwd with its keys and values into the 8-bit
    cache, then tokens: as long as nothing has been rounded (the whole context in
    the tail), they equal the forward over the whole sequence."""
    q, k, v = tokens(2, 4, 60, 64, 64, seed=20)
    cache = rdm.rdm_ska_q8_cache(2, 4, 64, 64, 200, block=64)
    d = [t.cuda() for t in (q, k, v)]
    rdm.rdm_ska_q8_fill(d[1][:, :50].contiguous(), d[2][:, :, :50].contiguous(), *cache)
    whole = rdm.rdm_ska_fwd(*d, 200)
    for t in range(50, 60):
        o = rdm.rdm_ska_q8_decode(*(x.contiguous() for x in (d[0][:, :, t], d[1][:, t], d[2][:, :, t])), *cache)
        # the forward rounds its softmax weights to bf16: 2^-8 of the largest value, and each output half a step
        assert (o.double() - whole[:, :, t].double()).abs().max().item() <= 2.0 ** -7 * 4


def test_hybrid_layer_serves_a_prompt_and_tokens(cuda_ok):
    """The two mixers as a hybrid stack runs them: a ragged batch's prompt
    through the scan and the window attention's cache, then tokens through both,
    the scan's output as the attention's query and value, captured as one graph."""
    B, H, D, N, T, w, steps = 3, 4, 64, 16, 50, 40, 12
    lengths = [50, 17, 33]
    i = ssm_reference.inputs(B, H, T + steps, D, N, dtype=BF16, seed=41)
    i["conv_state_in"], i["S0"] = None, None
    g = torch.Generator().manual_seed(42)
    keys = torch.randn(B, T + steps, D, generator=g).to(BF16)
    # each sequence's tokens: its prompt, then `steps` more
    def piece(t, b, lo, hi):
        return t[b, :, lo:hi]
    d = {n: (t.cuda() if t is not None else None) for n, t in i.items()}
    head = {n: (t[:, :, :T].contiguous() if n in ("x", "dt", "z", "Bm", "Cm") else t) for n, t in d.items()}
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, S, cs = rdm.rdm_ssm_fwd(*(head[n] for n in ("x", "dt", "A", "Bm", "Cm")), z=head["z"], dt_bias=head["dt_bias"],
                               feedthrough=head["feedthrough"], conv_weight=head["conv_weight"], conv_bias=head["conv_bias"],
                               lengths=ln, return_state=True)
    cache = rdm.rdm_ska_q8_cache(B, H, D, D, w, block=16)
    rdm.rdm_ska_q8_fill(keys[:, :T].contiguous().cuda(), y, *cache, lengths=ln)
    yr, _, _ = ssm_reference.scan(i, [n + steps for n in lengths])
    caches = [ref.Cache(H, D, D, w, 16, torch.float8_e4m3fn) for _ in range(B)]
    for b, n in enumerate(lengths):
        ssm_reference.assert_near(y[b, :, :n], yr[b, :, :n], T + N, f"prompt {b}")
        for t in range(n):
            caches[b].add(keys[b, t], y[b, :, t].cpu())
    ref.assert_state(cache, caches, "prompt")
    rows = {n: torch.empty_like(d[n][:, :, 0]) for n in ("x", "dt", "z", "Bm", "Cm")}
    key = torch.empty(B, D, dtype=BF16, device="cuda")

    def token():
        out = rdm.rdm_ssm_step(rows["x"], rows["dt"], d["A"], rows["Bm"], rows["Cm"], S, z=rows["z"], dt_bias=d["dt_bias"],
                               feedthrough=d["feedthrough"], conv_weight=d["conv_weight"], conv_bias=d["conv_bias"], conv_state=cs)
        return out, rdm.rdm_ska_q8_decode(out, key, out, *cache)

    state = [t.clone() for t in (S, cs, *cache)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, o = token()
    for t, was in zip((S, cs, *cache), state):
        t.copy_(was)
    at = torch.arange(B)
    for s in range(steps):
        idx = torch.tensor([n + s for n in lengths])
        for n, dst in rows.items():
            dst.copy_(i[n][at, :, idx])
        key.copy_(keys[at, idx])
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            ssm_reference.assert_near(out[b], yr[b, :, lengths[b] + s], T + N, f"token {s} of sequence {b}")
        qv = out.cpu()
        want = torch.stack([c.attend(qv[b], c.add(keys[b, idx[b]], qv[b]), 1 / 8) for b, c in enumerate(caches)])
        ref.assert_out(o, want, yr.abs().max().item() * 1.1, f"attention at token {s}")
    ref.assert_state(cache, caches, "after the tokens")
    assert rdm.rdm_ddts_sync_status() == 0
