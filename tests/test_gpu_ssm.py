"""GPU tests of the selective scan through the public entry points against the
float64 reference (tests/ssm_reference.py): prompts, gradients and single
tokens over types, state sizes, widths, groups, odd lengths, ragged batches,
segments, carried states, streams and graphs."""
import pytest
import torch

import gated_linear_attention_ddts_b200 as rdm
from tests import ssm_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
PLAIN = ("x", "dt", "A", "Bm", "Cm")


def cuda(i):
    return {n: (t.cuda() if t is not None else None) for n, t in i.items()}


def call(fn, d, *args, **kw):
    return fn(*(d[n] for n in PLAIN), *args, **{n: t for n, t in d.items() if n not in PLAIN}, **kw)


def check_all(i, lengths=None, silu=True, gates="preact", saved=True, seed=1):
    """Forward with its states, and every gradient."""
    B, H, T, D = i["x"].shape
    N, dtype = i["A"].shape[-1], i["x"].dtype
    W = i["conv_weight"].shape[-1] if i["conv_weight"] is not None else 0
    g = torch.Generator().manual_seed(seed)
    gy = torch.randn(B, H, T, D, generator=g).to(dtype)
    gST = torch.randn(B, H, D, N, generator=g)
    gcs = torch.randn(B, H, W - 1, D, generator=g).to(dtype) if W > 1 else None
    d = cuda(i)
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda") if lengths is not None else None
    keep = rdm.rdm_ssm_saved_states(d["x"], d["A"]) if saved else None
    y, ST, cs = call(rdm.rdm_ssm_fwd, d, conv_silu=silu, gates=gates, lengths=ln, return_state=True, saved_states=keep)
    yr, STr, csr = ref.scan(i, lengths, silu, gates)
    got = call(rdm.rdm_ssm_bwd, d, gy.cuda(), gST.cuda(), gcs.cuda() if W > 1 else None, conv_silu=silu, gates=gates,
               lengths=ln, saved_states=keep)
    assert rdm.rdm_ddts_sync_status() == 0
    terms = T + N
    ref.assert_near(y, yr, terms, "y")
    ref.assert_near(ST, STr, terms, "ST")
    if W > 1:
        assert torch.equal(cs.cpu().double(), csr)
    want = ref.gradients(i, gy, gST, gcs, lengths, silu, gates)
    for n, t in want.items():
        ref.assert_near(got[n], t, T + N + H * D, n, grad=True)
    assert all(got[n] is None for n in set(got) - set(want))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,N", [(16, 16), (32, 16), (64, 16), (128, 16), (32, 32), (16, 64), (64, 64), (32, 128)])
def test_sizes(cuda_ok, dtype, D, N):
    check_all(ref.inputs(2, 2, 37, D, N, dtype=dtype, seed=D + N))


@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 31, 32, 33, 64, 131])
def test_lengths_around_the_tiles(cuda_ok, T):
    check_all(ref.inputs(1, 2, T, 32, 16, seed=T))


@pytest.mark.parametrize("W", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("carried", [False, True])
@pytest.mark.parametrize("silu", [False, True])
def test_convolution_widths(cuda_ok, W, carried, silu):
    check_all(ref.inputs(2, 1, 19, 16, 16, W=W, carried=carried, seed=W), silu=silu)


@pytest.mark.parametrize("z,bias,feed", [(False, True, True), (True, False, True), (True, True, False), (False, False, False)])
def test_optional_inputs(cuda_ok, z, bias, feed):
    check_all(ref.inputs(1, 2, 21, 32, 16, z=z, bias=bias, feed=feed, seed=3))


def test_activated_steps(cuda_ok):
    check_all(ref.inputs(2, 2, 40, 32, 16, gates="activated", seed=4), gates="activated")


@pytest.mark.parametrize("H,G", [(4, 1), (4, 2), (4, 4), (6, 3)])
def test_groups(cuda_ok, H, G):
    check_all(ref.inputs(2, H, 35, 16, 32, G=G, seed=H + G))


@pytest.mark.parametrize("saved", [False, True])
def test_ragged_batch(cuda_ok, saved):
    """Lengths of zero, one, less than the filter, on and beside tile borders."""
    check_all(ref.inputs(7, 2, 70, 16, 16, seed=9), lengths=[70, 0, 1, 2, 32, 33, 48], saved=saved)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [640, 1027])
def test_segments(cuda_ok, dtype, T):
    """Few channels and many tokens: the sequences are cut; a length ends a
    token behind a cut, so the filter reaches from one segment into the next."""
    i = ref.inputs(2, 1, T, 32, 16, dtype=dtype, seed=T)
    d = cuda(i)
    assert rdm.rdm_ssm_fwd_workspace_size(*(d[n] for n in PLAIN), conv_weight=d["conv_weight"]) > 0
    check_all(i)
    check_all(i, lengths=[T, 513], saved=False)
    # without a workspace the sequences stay whole (each y is rounded once, so each
    # is held to the reference: two rounded values may differ by a whole step)
    y, ST, _ = call(rdm.rdm_ssm_fwd, d, return_state=True, workspace=False)
    yr, STr, _ = ref.scan(i)
    ref.assert_near(ST, STr, T + 16, "ST without segments")
    ref.assert_near(y, yr, T + 16, "y without segments")


@pytest.mark.parametrize("N", [16, 64])
@pytest.mark.parametrize("T", [65, 130, 397, 1040])
def test_segment_counts(cuda_ok, T, N):
    """More segments than the chunks divide into (the last ones are empty), and
    sequences that end a few tokens behind any 16th: the filter's gradient then
    reaches over a cut to carried-out inputs of both sides."""
    ends = [T, 1, 33, 34, 49, 50, 51, T // 32 * 16 + 1, T // 32 * 16 + 2]
    check_all(ref.inputs(len(ends), 1, T, 16, N, seed=T + N), lengths=[min(n, T) for n in ends])


def test_rows_behind_the_end_are_left(cuda_ok):
    i = ref.inputs(2, 2, 50, 32, 16, dtype=BF16, seed=11)
    d = cuda(i)
    y = torch.full_like(d["x"], 7.0)
    for n in ("x", "dt", "z", "Bm", "Cm"):  # what stands behind an end is not used
        d[n][1, :, 20:] = float("nan")
    ln = torch.tensor([50, 20], dtype=torch.int32, device="cuda")
    y, ST, cs = call(rdm.rdm_ssm_fwd, d, lengths=ln, y=y, return_state=True)
    yr, STr, csr = ref.scan(i, [50, 20])
    assert (y[1, :, 20:] == 7).all()
    ref.assert_near(y[1, :, :20], yr[1, :, :20], 66, "y")
    ref.assert_near(ST, STr, 66, "ST")
    assert torch.equal(cs.cpu().double(), csr)
    gy = torch.randn(2, 2, 50, 32, generator=torch.Generator().manual_seed(2)).to(BF16)
    bad = gy.clone()
    bad[1, :, 20:] = float("nan")
    got = call(rdm.rdm_ssm_bwd, d, bad.cuda(), lengths=ln)
    want = ref.gradients(i, gy, lengths=[50, 20])
    for n, t in want.items():
        ref.assert_near(got[n], t, 50 + 16 + 64, n, grad=True)


def test_steps_of_zero_keep_the_state(cuda_ok):
    """Decays of exactly 1: a sequence that ends inside a tile has the state of its
    last token, and steps of zero leave a state bit by bit."""
    i = cuda(ref.inputs(1, 2, 50, 32, 16, seed=13, gates="activated"))
    ln = torch.tensor([20], dtype=torch.int32, device="cuda")
    _, ST, _ = call(rdm.rdm_ssm_fwd, i, gates="activated", lengths=ln, return_state=True)
    head = {n: (t[:, :, :20].contiguous() if n in ("x", "dt", "z", "Bm", "Cm") else t) for n, t in i.items()}
    _, ST1, _ = call(rdm.rdm_ssm_fwd, head, gates="activated", return_state=True)
    assert torch.equal(ST, ST1)
    _, ST2, _ = call(rdm.rdm_ssm_fwd, {**i, "dt": torch.zeros_like(i["dt"])}, gates="activated", return_state=True)
    assert torch.equal(ST2, i["S0"])


@pytest.mark.parametrize("lengths,clamped", [([-3, 9], [0, 9]), ([40, 100], [40, 40])])
def test_length_out_of_range_is_reported(cuda_ok, lengths, clamped):
    i = ref.inputs(2, 1, 40, 16, 16, seed=1)
    d = cuda(i)
    y, ST, _ = call(rdm.rdm_ssm_fwd, d, lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"), return_state=True)
    assert rdm.rdm_ddts_sync_status() == rdm.RDM_ERR_INVALID_ARG
    assert rdm.rdm_ddts_sync_status() == 0
    yr, STr, _ = ref.scan(i, clamped)
    ref.assert_near(y, yr, 56, "y")
    ref.assert_near(ST, STr, 56, "ST")


def test_no_tokens(cuda_ok):
    i = ref.inputs(2, 2, 0, 32, 16, seed=2)
    d = cuda(i)
    y, ST, cs = call(rdm.rdm_ssm_fwd, d, return_state=True)
    assert y.shape == (2, 2, 0, 32) and torch.equal(ST, d["S0"]) and torch.equal(cs, d["conv_state_in"])
    gST, gcs = torch.randn_like(ST), torch.randn_like(cs)
    g = call(rdm.rdm_ssm_bwd, d, torch.empty_like(y), gST, gcs)
    assert torch.equal(g["dS0"], gST) and torch.equal(g["dconv_state_in"], gcs)
    for n in ("dA", "ddt_bias", "dfeed", "dconv_weight", "dconv_bias"):
        assert not g[n].any(), n


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,W,G", [(16, 4, 1), (32, 3, 2), (64, 2, 1), (128, 1, 4), (16, 0, 2)])
def test_steps_follow_the_prompt(cuda_ok, dtype, N, W, G):
    """A prompt of 21 tokens, then 6 single tokens: each equals the whole
    sequence's scan at that token, and so do the state and the inputs kept."""
    B, H, D, T0, T = 3, 4, 16, 21, 27
    i = ref.inputs(B, H, T, D, N, G=G, W=W, dtype=dtype, seed=N + W)
    yr, STr, csr = ref.scan(i)
    d = cuda(i)
    head = {n: (t[:, :, :T0].contiguous() if n in ("x", "dt", "z", "Bm", "Cm") else t) for n, t in d.items()}
    _, S, cs = call(rdm.rdm_ssm_fwd, head, return_state=True)
    keep = {n: d[n] for n in ("A", "dt_bias", "feedthrough", "conv_weight", "conv_bias")}
    for t in range(T0, T):
        row = {n: d[n][:, :, t].contiguous() for n in ("x", "dt", "Bm", "Cm", "z")}
        y = rdm.rdm_ssm_step(row["x"], row["dt"], keep["A"], row["Bm"], row["Cm"], S, z=row["z"], dt_bias=keep["dt_bias"],
                             feedthrough=keep["feedthrough"], conv_weight=keep["conv_weight"], conv_bias=keep["conv_bias"],
                             conv_state=cs if W > 1 else None)
        ref.assert_near(y, yr[:, :, t], T + N, f"token {t}")
    ref.assert_near(S, STr, T + N, "state")
    if W > 1:
        assert torch.equal(cs.cpu().double(), csr)


def test_prompt_in_pieces(cuda_ok):
    i = ref.inputs(2, 2, 100, 32, 16, G=2, dtype=BF16, seed=8)
    d = cuda(i)
    yr, STr, csr = ref.scan(i)
    S, cs, at = d["S0"], d["conv_state_in"], 0
    for n in (1, 2, 30, 67):
        piece = {k: (t[:, :, at:at + n].contiguous() if k in ("x", "dt", "z", "Bm", "Cm") else t) for k, t in d.items()}
        piece.update(S0=S, conv_state_in=cs)
        y, S, cs = call(rdm.rdm_ssm_fwd, piece, return_state=True)
        ref.assert_near(y, yr[:, :, at:at + n], 116, f"piece at {at}")
        at += n
    ref.assert_near(S, STr, 116, "state")
    assert torch.equal(cs.cpu().double(), csr)


def test_long_memory_and_large_steps(cuda_ok):
    """Decays next to 1 over 2000 tokens, and steps so large that the state is
    forgotten at once; a zero, a huge and a tiny pre-activation."""
    i = ref.inputs(1, 1, 2000, 16, 16, W=0, seed=3)
    i["A"] = i["A"] * 1e-3
    check_all(i)
    i = ref.inputs(1, 1, 40, 16, 16, W=4, seed=4)
    i["dt"][:, :, 5], i["dt"][:, :, 6], i["dt"][:, :, 7] = 60.0, -60.0, 0.0
    check_all(i)


def test_gradients_against_differences(cuda_ok):
    """<grad, v> against (L(+h v) - L(-h v)) / 2h of the GPU forward in float32.
    L adds about 2000 products of size 1: rounding leaves 2000 2^-21 / h = 0.1 at
    h = 1e-2 at the very most, about sqrt(2000) 2^-21 / h = 2e-3 with random
    signs; the third derivatives leave h^2 of the value.  Bound: 1e-2 of
    |grad| |v| plus 1e-2."""
    i = ref.inputs(2, 2, 33, 16, 16, G=2, seed=21)
    g = torch.Generator().manual_seed(22)
    w = [torch.randn(s, generator=g) for s in ((2, 2, 33, 16), (2, 2, 16, 16), (2, 2, 3, 16))]

    def loss(j):
        out = call(rdm.rdm_ssm_fwd, cuda(j), return_state=True)
        return sum((a.cpu().double() * b.double()).sum() for a, b in zip(out, w)).item()

    got = call(rdm.rdm_ssm_bwd, cuda(i), *(t.cuda() for t in w))
    h = 1e-2
    for n, t in i.items():
        v = torch.randn(t.shape, generator=g)
        v = v / v.norm()
        diff = (loss({**i, n: t + h * v}) - loss({**i, n: t - h * v})) / (2 * h)
        gr = got[ref.NAMES[n]].cpu().double()
        assert abs(diff - (gr * v.double()).sum().item()) <= 1e-2 * gr.norm().item() + 1e-2, n


def test_same_bits_every_time(cuda_ok):
    i = cuda(ref.inputs(2, 4, 300, 32, 16, seed=5, dtype=BF16))
    gy = torch.randn_like(i["x"])
    first = call(rdm.rdm_ssm_bwd, i, gy)
    for _ in range(3):
        again = call(rdm.rdm_ssm_bwd, i, gy)
        assert all(torch.equal(first[n], again[n]) for n in first)


def test_two_streams_at_once(cuda_ok):
    """Two training steps of cut sequences on two streams equal the same calls one
    after the other."""
    ds = [cuda(ref.inputs(1, 2, 700, 32, 16, seed=50 + k, dtype=BF16)) for k in range(2)]
    gys = [torch.randn_like(d["x"]) for d in ds]
    want = [call(rdm.rdm_ssm_bwd, d, gy) for d, gy in zip(ds, gys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for k in range(2):
            got[k].append(call(rdm.rdm_ssm_bwd, ds[k], gys[k], stream=streams[k]))
    torch.cuda.synchronize()
    assert all(torch.equal(g[n], want[k][n]) for k in range(2) for g in got[k] for n in g)


def test_other_stream_and_graph(cuda_ok):
    """A call on a side stream, and a captured prompt and token replayed with
    new inputs in the same buffers."""
    i, j = ref.inputs(1, 2, 700, 32, 16, seed=31), ref.inputs(1, 2, 700, 32, 16, seed=32)
    d = cuda(i)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, ST, _ = call(rdm.rdm_ssm_fwd, d, return_state=True, stream=side)
    side.synchronize()
    ref.assert_near(y, ref.scan(i)[0], 716, "side stream")
    gy = torch.randn_like(d["x"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, ST, _ = call(rdm.rdm_ssm_fwd, d, return_state=True)
        grads = call(rdm.rdm_ssm_bwd, d, gy)
    for k in (j, i):
        for n, t in k.items():
            d[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        yr, STr, _ = ref.scan(k)
        ref.assert_near(y, yr, 716, "replayed y")
        ref.assert_near(ST, STr, 716, "replayed ST")
        plain = call(rdm.rdm_ssm_bwd, d, gy)
        assert all(torch.equal(plain[n], grads[n]) for n in plain)


def test_binding_refusals(cuda_ok):
    d = cuda(ref.inputs(1, 2, 8, 32, 16, seed=1))
    with pytest.raises(ValueError):
        call(rdm.rdm_ssm_fwd, {**d, "x": d["x"].transpose(2, 3).contiguous().transpose(2, 3)})
    with pytest.raises(ValueError):
        call(rdm.rdm_ssm_fwd, {**d, "dt_bias": d["dt_bias"][:1]})
    with pytest.raises(TypeError):
        call(rdm.rdm_ssm_fwd, {**d, "z": d["z"].to(BF16)})
    with pytest.raises(TypeError):
        call(rdm.rdm_ssm_fwd, {n: (t.half() if n in ("x", "dt", "z", "Bm", "Cm", "conv_state_in") else t) for n, t in d.items()})
    with pytest.raises(ValueError):
        call(rdm.rdm_ssm_fwd, {**d, "conv_weight": None, "conv_bias": None})
    with pytest.raises(rdm.RdmError):
        call(rdm.rdm_ssm_bwd, d, torch.empty_like(d["x"]), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
