"""GPU tests of the gated linear recurrence, the 8-bit activation checkpoints and
the RMS norm against plain 64-bit implementations (tests/ops_ref.py)."""
import pytest
import torch

import gated_delta_rule_chunkwise_amd as kda
import ops_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(shape, seed, dtype=F32, scale=1.0):
    return (scale * torch.randn(shape, generator=gen(seed))).to(dtype)


def gate(shape, seed, dtype=F32, kind="softplus"):
    if kind == "softplus":
        return -torch.nn.functional.softplus(randn(shape, seed)).to(dtype)
    u = torch.rand(shape, generator=gen(seed))
    return torch.log(0.5 + u * (0.9999 - 0.5)).to(dtype)


def cu_of(lengths):
    cu = torch.zeros(len(lengths) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lengths, dtype=torch.int32), 0)
    return cu.to(DEV)


def off_by_one(t):
    """The same values, contiguous, one element behind an aligned address."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
    v = buf[1:].reshape(t.shape)
    v.copy_(t)
    return v


# ------------------------------------------------- gated linear recurrence
GLR_CASES = [
    # lengths, D
    ([1], 1), ([1], 64), ([3], 7), ([17], 65), ([64], 128), ([255], 256), ([256], 260), ([257], 129),
    ([1000], 96), ([2500], 512), ([40, 0, 1, 700, 0], 130), ([1] * 300, 64), ([0, 5, 0], 33), ([513, 511, 1025], 384),
    ([1500], 1), ([5000], 20), ([16, 16, 16], 1024), ([31, 33, 2, 1, 600], 1028),
]


def glr_inputs(lengths, D, io, gt, seed, kind):
    T, N = sum(lengths), len(lengths)
    x, la = randn((T, D), seed, io), gate((T, D), seed + 1, gt, kind)
    h0, gh = randn((N, D), seed + 2), randn((T, D), seed + 3, io)
    return x, la, h0, gh, 0.3 * randn((N, D), seed + 4)


@pytest.mark.parametrize("io,gt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("lengths,D", GLR_CASES)
def test_glr_forward_and_backward(lengths, D, io, gt):
    kind = "uniform" if D % 2 else "softplus"
    x, la, h0, gh, ghT = glr_inputs(lengths, D, io, gt, 7 * D + len(lengths), kind)
    cu = cu_of(lengths) if len(lengths) > 1 else None
    g = lambda t: t.to(DEV)  # noqa: E731
    for state in (h0, None):
        want = ref.glr_fwd(x, la, state, lengths)
        h, hT = kda.kda_glr_fwd(g(x), g(la), h0=None if state is None else g(state), cu_seqlens=cu)
        ref.assert_within(h, want[0], want[2], "h")
        ref.assert_within(hT, want[1], want[3], "h_T")
        gs = ghT if state is not None else None
        wb = ref.glr_bwd(la, h.cpu(), gh, state, gs, lengths)
        dx, dla, dh0 = kda.kda_glr_bwd(g(la), h, g(gh), h0=None if state is None else g(state),
                                       grad_hT=None if gs is None else g(gs), cu_seqlens=cu)
        for got, w, e, name in zip((dx, dla, dh0), wb[:3], wb[3:], ("dx", "dla", "dh0")):
            ref.assert_within(got, w, e, name)
        codes, scales = kda.kda_act8_pack(h)
        h8 = ref.unpack(codes.cpu().reshape(-1, D), scales.cpu().reshape(-1, ref.blocks(D)))
        wb = ref.glr_bwd(la, h8, gh, state, gs, lengths)
        got = kda.kda_glr_bwd_act8(g(la), codes, scales, g(gh), h0=None if state is None else g(state),
                                   grad_hT=None if gs is None else g(gs), cu_seqlens=cu)
        for a, w, e, name in zip(got, wb[:3], wb[3:], ("dx", "dla", "dh0")):
            ref.assert_within(a, w, e, name + " (8-bit h)")
        assert torch.equal(got[0], dx) and torch.equal(got[2], dh0)   # these do not read h


@pytest.mark.parametrize("B,T,D", [(3, 1, 40), (2, 300, 64), (5, 257, 256), (64, 33, 48), (2, 2048, 8)])
@pytest.mark.parametrize("io", [BF, F32])
def test_glr_equal_length_batch(B, T, D, io):
    lengths = [T] * B
    x, la, h0, gh, ghT = glr_inputs(lengths, D, io, io, 11 * T + B, "uniform")
    sh = lambda t: t.reshape(B, T, D).to(DEV)  # noqa: E731
    want = ref.glr_fwd(x, la, h0, lengths)
    h, hT = kda.kda_glr_fwd(sh(x), sh(la), h0=h0.to(DEV))
    ref.assert_within(h.reshape(-1, D), want[0], want[2], "h")
    ref.assert_within(hT, want[1], want[3], "h_T")
    wb = ref.glr_bwd(la, h.reshape(-1, D).cpu(), gh, h0, ghT, lengths)
    got = kda.kda_glr_bwd(sh(la), h, sh(gh), h0=h0.to(DEV), grad_hT=ghT.to(DEV))
    for a, w, e, name in zip(got, wb[:3], wb[3:], ("dx", "dla", "dh0")):
        ref.assert_within(a.reshape(w.shape), w, e, name)


@pytest.mark.parametrize("T,D", [(700, 256), (2100, 40)])
@pytest.mark.parametrize("io", [BF, F32])
def test_glr_misaligned_inputs(T, D, io):
    x, la, h0, gh, ghT = glr_inputs([T], D, io, io, 91, "softplus")
    want = ref.glr_fwd(x, la, h0, [T])
    h = off_by_one(torch.zeros(T, D, dtype=io))
    h, hT = kda.kda_glr_fwd(off_by_one(x), off_by_one(la), h0=off_by_one(h0), h=h)
    ref.assert_within(h, want[0], want[2], "h")
    ref.assert_within(hT, want[1], want[3], "h_T")
    wb = ref.glr_bwd(la, h.cpu(), gh, h0, ghT, [T])
    codes, scales = kda.kda_act8_pack(h)
    for got in (kda.kda_glr_bwd(off_by_one(la), h, off_by_one(gh), h0=off_by_one(h0), grad_hT=off_by_one(ghT)),):
        for a, w, e, name in zip(got, wb[:3], wb[3:], ("dx", "dla", "dh0")):
            ref.assert_within(a, w, e, name)
    a = kda.kda_glr_bwd_act8(la.to(DEV), codes, scales, gh.to(DEV), h0=h0.to(DEV), grad_hT=ghT.to(DEV))
    b = kda.kda_glr_bwd_act8(off_by_one(la), off_by_one(codes), off_by_one(scales), off_by_one(gh),
                             h0=off_by_one(h0), grad_hT=off_by_one(ghT))
    for u, v, name in zip(a, b, ("dx", "dla", "dh0")):
        ref.assert_within(v, u.double().cpu(), 1e-5 * u.double().abs().max().cpu() + 0 * u.double().cpu(), name)


def test_glr_resets_cut_the_history():
    """log_alpha = -inf (or below fp32's exponential) drops what came before, also
    infinities and NaN, and the gradients behind it."""
    T, D = 3000, 72
    x, la, h0, gh, _ = glr_inputs([T], D, F32, F32, 5, "uniform")
    cuts = [1, 2, 40, 900, 1024, 2047, 2999]
    la[cuts] = float("-inf")
    la[1800] = -200.0
    dirty = x.clone()
    dirty[3:40] = float("nan")
    dirty[850] = float("inf")
    want = ref.glr_fwd(x, la, h0, [T])
    h, hT = kda.kda_glr_fwd(dirty.to(DEV), la.to(DEV), h0=h0.to(DEV))
    hc = h.cpu()
    assert torch.isnan(hc[3:40]).all() and not torch.isfinite(hc[850:900]).any()
    keep = torch.ones(T, dtype=torch.bool)
    keep[3:40] = keep[850:900] = False
    ref.assert_within(h[keep.to(DEV)], want[0][keep], want[2][keep], "h")
    ref.assert_within(hT, want[1], want[3], "h_T")
    # the same backwards: a NaN gradient stays behind its reset
    bad = gh.clone()
    bad[1200] = float("nan")
    clean_h = want[0].float()
    wb = ref.glr_bwd(la, clean_h, gh, h0, None, [T])
    dx, dla, dh0 = kda.kda_glr_bwd(la.to(DEV), clean_h.to(DEV), bad.to(DEV), h0=h0.to(DEV))
    keep = torch.ones(T, dtype=torch.bool)
    keep[1024:1201] = False
    assert torch.isnan(dx.cpu()[1024:1201]).all()
    ref.assert_within(dx[keep.to(DEV)], wb[0][keep], wb[3][keep], "dx")
    ref.assert_within(dla[keep.to(DEV)], wb[1][keep], wb[4][keep], "dla")
    assert (dla.cpu()[cuts] == 0).all()
    ref.assert_within(dh0, wb[2], wb[5], "dh0")


def test_glr_slow_decay_keeps_its_rate():
    """Constant gates near 1 over a long sequence: the decay's distance from 1 is
    what counts.  bf16 rounds the gate itself, so the gate is taken as given."""
    T, D = 20000, 8
    la = torch.tensor([-1e-5, -3e-5, -1e-4, -1e-3, -1e-2, -0.02, -0.1, 0.0])[None, :].expand(T, D).contiguous()
    x = torch.rand(T, D, generator=gen(3))
    want = ref.glr_fwd(x, la, None, [T])
    h, hT = kda.kda_glr_fwd(x.to(DEV), la.to(DEV))
    ref.assert_within(h, want[0], want[2], "h")
    ref.assert_within(hT, want[1], want[3], "h_T")


def test_glr_rows_behind_the_last_sequence_are_left():
    lengths, T, D = [300, 450], 900, 132
    x, la, h0, gh, ghT = glr_inputs(lengths + [150], D, BF, BF, 21, "softplus")
    cu = cu_of(lengths)
    x[750:] = float("nan")
    la[750:] = float("nan")
    h = torch.full((T + 3, D), 7.0, dtype=BF, device=DEV)
    out, hT = kda.kda_glr_fwd(x.to(DEV), la.to(DEV), h0=h0[:2].to(DEV), cu_seqlens=cu, h=h[:T])
    want = ref.glr_fwd(x[:750], la[:750], h0[:2], lengths)
    ref.assert_within(out[:750], want[0], want[2], "h")
    ref.assert_within(hT, want[1], want[3], "h_T")
    assert (h[750:] == 7.0).all()


def test_glr_empty_sequences():
    D = 50
    h0, ghT = randn((3, D), 1).to(DEV), randn((3, D), 2).to(DEV)
    e = torch.empty((0, D), dtype=BF, device=DEV)
    cu = cu_of([0, 0, 0])
    h, hT = kda.kda_glr_fwd(e, e, h0=h0, cu_seqlens=cu)
    assert h.shape == (0, D) and torch.equal(hT, h0)
    assert torch.equal(kda.kda_glr_fwd(e, e, cu_seqlens=cu)[1], torch.zeros_like(h0))
    dx, dla, dh0 = kda.kda_glr_bwd(e, e, e, h0=h0, grad_hT=ghT, cu_seqlens=cu)
    assert torch.equal(dh0, ghT)
    e3 = torch.empty((3, 0, D), dtype=BF, device=DEV)
    assert torch.equal(kda.kda_glr_fwd(e3, e3, h0=h0)[1], h0)
    # in place: h_T over h0
    x = randn((3, 5, D), 4, BF).to(DEV)
    la = gate((3, 5, D), 5, BF).to(DEV)
    s = h0.clone()
    want = kda.kda_glr_fwd(x, la, h0=h0)
    got = kda.kda_glr_fwd(x, la, h0=s, h_T=s)
    assert torch.equal(got[0], want[0]) and torch.equal(s, want[1])


def test_glr_in_place_state_over_long_sequences():
    """h_T may be h0 itself, also where a sequence is worked on in many tiles."""
    lengths, D = [3000, 1, 0, 2000], 260
    x, la, h0, _, _ = glr_inputs(lengths, D, BF, BF, 31, "uniform")
    cu = cu_of(lengths)
    a = h0.to(DEV)
    want = kda.kda_glr_fwd(x.to(DEV), la.to(DEV), h0=a, cu_seqlens=cu)
    s = h0.to(DEV)
    got = kda.kda_glr_fwd(x.to(DEV), la.to(DEV), h0=s, cu_seqlens=cu, h_T=s)
    assert torch.equal(got[0], want[0]) and torch.equal(s, want[1])


@pytest.mark.parametrize("D", [131, 50, 261, 5])
@pytest.mark.parametrize("io", [BF, F32])
def test_glr_in_place_state_of_an_odd_number_of_channels(D, io):
    """The last lanes' channels overlap there; sequences of one and two tokens, and
    some that end in another tile, have their h0 overwritten by their h_T."""
    lengths = [3000, 1, 0, 2, 700, 2, 1, 1, 0, 300]
    x, la, h0, _, _ = glr_inputs(lengths, D, io, io, 37, "uniform")
    cu = cu_of(lengths)
    want = kda.kda_glr_fwd(x.to(DEV), la.to(DEV), h0=h0.to(DEV), cu_seqlens=cu)
    for _ in range(3):
        s = h0.to(DEV)
        got = kda.kda_glr_fwd(x.to(DEV), la.to(DEV), h0=s, cu_seqlens=cu, h_T=s)
        assert torch.equal(got[0], want[0]) and torch.equal(s, want[1])


@pytest.mark.parametrize("N,D,most", [(3000, 40, 5), (1500, 132, 9)])
def test_glr_more_sequences_than_are_staged(N, D, most):
    lengths = torch.randint(0, most + 1, (N,), generator=gen(N)).tolist()
    x, la, h0, gh, ghT = glr_inputs(lengths, D, BF, BF, 61, "softplus")
    cu, g = cu_of(lengths), lambda t: t.to(DEV)  # noqa: E731
    want = ref.glr_fwd(x, la, h0, lengths)
    h, hT = kda.kda_glr_fwd(g(x), g(la), h0=g(h0), cu_seqlens=cu)
    ref.assert_within(h, want[0], want[2], "h")
    ref.assert_within(hT, want[1], want[3], "h_T")
    wb = ref.glr_bwd(la, h.cpu(), gh, h0, ghT, lengths)
    got = kda.kda_glr_bwd(g(la), h, g(gh), h0=g(h0), grad_hT=g(ghT), cu_seqlens=cu)
    for a, w, e, name in zip(got, wb[:3], wb[3:], ("dx", "dla", "dh0")):
        ref.assert_within(a, w, e, name)


@pytest.mark.parametrize("io", [BF, F32])
def test_glr_gates_of_the_types_lowest_value(io):
    """finfo.min is what masks are filled with: a reset, like -inf, however many follow."""
    T, D = 700, 36
    x, la, h0, gh, _ = glr_inputs([T], D, io, io, 15, "softplus")
    low, inf = la.clone(), la.clone()
    rows = [0, 5, 6, 7, 300, 301, 699]
    low[rows], inf[rows] = torch.finfo(io).min, float("-inf")
    a = kda.kda_glr_fwd(x.to(DEV), low.to(DEV), h0=h0.to(DEV))
    b = kda.kda_glr_fwd(x.to(DEV), inf.to(DEV), h0=h0.to(DEV))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = kda.kda_glr_bwd(low.to(DEV), a[0], gh.to(DEV), h0=h0.to(DEV))
    gb = kda.kda_glr_bwd(inf.to(DEV), a[0], gh.to(DEV), h0=h0.to(DEV))
    assert all(torch.equal(u, v) for u, v in zip(ga, gb)) and not torch.isnan(ga[1]).any()
    want = ref.glr_fwd(x, inf, h0, [T])
    ref.assert_within(a[0], want[0], want[2], "h")


def test_glr_split_and_step_continue_a_sequence():
    T, D = 2400, 192
    x, la, h0, _, _ = glr_inputs([T], D, F32, F32, 13, "uniform")
    x, la, h0 = x.to(DEV), la.to(DEV), h0.to(DEV)
    want, ET = ref.glr_fwd(x.cpu(), la.cpu(), h0.cpu(), [T])[0], ref.glr_fwd(x.cpu(), la.cpu(), h0.cpu(), [T])[2]
    h1, s = kda.kda_glr_fwd(x[:1300], la[:1300], h0=h0)
    h2, s = kda.kda_glr_fwd(x[1300:2390], la[1300:2390], h0=s)
    steps = [kda.kda_glr_step(x[t:t + 1], la[t:t + 1], s) for t in range(2390, T)]
    ref.assert_within(torch.cat([h1, h2] + steps), want, ET, "h")


@pytest.mark.parametrize("B,D", [(1, 1), (1, 2048), (7, 33), (256, 4096), (3, 130)])
@pytest.mark.parametrize("io,gt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_glr_step(B, D, io, gt):
    x, la, S = randn((B, D), 1, io), gate((B, D), 2, gt), randn((B, D), 3)
    la[0, 0] = float("-inf")
    S[0, 0] = float("nan")
    want = ref.glr_fwd(x.reshape(1, -1), la.reshape(1, -1), S.reshape(1, -1), [1])
    want = [t.reshape(B, D) for t in (want[0], want[2])]
    for put in (lambda t: t.to(DEV), off_by_one):
        s = put(S)
        h = kda.kda_glr_step(put(x), put(la), s)
        ref.assert_within(h, want[0], want[1], "h")
        ref.assert_within(s, want[0], want[1], "S")


@pytest.mark.parametrize("act8", [False, True])
def test_glr_autograd_against_differences(act8):
    """The directional derivative of a weighted sum of h and h_T, by central
    differences of the 64-bit recurrence, against the gradients.  The loss is
    linear in x and h0 (differences exact up to 64-bit rounding); in log_alpha the
    third-order term of the difference, eps^2 T^2-ish, is far below the tolerance.
    fp32 gradients: 1e-5 relative of the sum of magnitudes; with h in 8 bits each
    factor h is off by at most half a scale, which adds sum |v c| scale / 2."""
    lengths, D = [300, 180], 24
    x, la, h0, wh, wT = glr_inputs(lengths, D, F32, F32, 77, "uniform")
    leaves = [t.to(DEV).requires_grad_() for t in (x, la, h0)]
    h, hT = kda.gated_linear_recurrence(*leaves, cu_of(lengths), act8=act8)
    ((h * wh.to(DEV)).sum() + (hT * wT.to(DEV)).sum()).backward()

    def loss(x, la, h0):
        h, hT, _, _ = ref.glr_fwd(x, la, h0, lengths)
        return float((h * wh).sum() + (hT * wT).sum())

    eps = 1e-5
    base = [x.double(), la.double(), h0.double()]
    for i in range(3):
        v = randn(base[i].shape, 100 + i).double()
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + eps * v, base[i] - eps * v
        want = (loss(*hi) - loss(*lo)) / (2 * eps)
        prod = leaves[i].grad.double().cpu() * v
        tol = 1e-5 * float(prod.abs().sum())
        if act8 and i == 1:
            # c_t = dla_t / h_{t-1} in magnitude, from the exact backward
            hd = ref.glr_fwd(x, la, h0, lengths)[0]
            _, dla, _, _, _, _ = ref.glr_bwd(la, torch.ones_like(hd), wh, torch.ones_like(h0), wT, lengths)
            scale = hd.abs().amax(-1, keepdim=True) / 127
            prev = torch.cat([torch.zeros(1, 1).double(), scale[:-1]])
            tol += float((v * dla).abs().mul(prev / 2 * 1.01).sum())
        assert abs(float(prod.sum()) - want) <= tol, (i, float(prod.sum()), want, tol)


def test_glr_results_repeat_and_streams():
    """Bitwise the same on every call, on another stream and with a given workspace."""
    lengths, D = [4000, 3, 2777], 516
    x, la, h0, gh, ghT = [t.to(DEV) for t in glr_inputs(lengths, D, BF, BF, 8, "uniform")]
    cu = cu_of(lengths)

    def both(ws=None):
        h, hT = kda.kda_glr_fwd(x, la, h0=h0, cu_seqlens=cu, workspace=ws)
        return (h, hT) + kda.kda_glr_bwd(la, h, gh, h0=h0, grad_hT=ghT, cu_seqlens=cu, workspace=ws)

    first = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = [both() for _ in range(3)]
    side.synchronize()
    need = kda.kda_glr_workspace_size(1, sum(lengths), D, len(lengths), kda.KDA_BF16)
    ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device=DEV)
    again.append(both(ws))
    again.append(both(ws))
    for out in again:
        assert all(torch.equal(a, b) for a, b in zip(first, out))


# ---------------------------------------------- 8-bit activation checkpoints
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 127), (3, 128), (4, 129), (64, 64), (7, 1000), (2, 4096), (33, 257),
                                       (1000, 128), (17, 8), (300, 2)])
@pytest.mark.parametrize("io", [BF, F32])
def test_act8_pack_and_unpack(rows, cols, io):
    x = randn((rows, cols), rows + cols, io, scale=3.0)
    x[0, 0] = 0.0
    wc, ws = ref.pack(x)
    for put in (lambda t: t.to(DEV), off_by_one):
        codes, scales = kda.kda_act8_pack(put(x))
        assert torch.equal(codes.cpu(), wc) and torch.equal(scales.cpu(), ws)
        for dt in (BF, F32):
            back = kda.kda_act8_unpack(put(codes), put(scales), dt)
            assert torch.equal(back.cpu(), (codes.cpu().float() * ws.repeat_interleave(128, 1)[:, :cols]).to(dt))


def test_act8_ties_zeros_and_values_that_are_not_finite():
    """max 127 gives scale 1: halves are ties, to even; a value one fp32 step off a
    tie keeps its side."""
    rows = torch.zeros(8, 256)
    rows[0, :12] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, 125.5, -126.5, 3.0, -127.0])
    near = torch.tensor([0.5, 1.5, 2.5, 63.5, 126.5])
    rows[1, 0] = 127.0
    rows[1, 1:6] = torch.nextafter(near, torch.tensor(1000.0))
    rows[1, 6:11] = torch.nextafter(near, torch.tensor(-1000.0))
    rows[2, 130] = float("nan")          # only the second block
    rows[2, 3] = 2.0
    rows[3, 5] = float("inf")
    rows[4, 7] = float("-inf")
    rows[5, :4] = torch.tensor([1e-45, -1e-44, 3e-40, 1e-38])
    rows[6, :2] = torch.tensor([3.4028234663852886e38, -1e38])
    rows[7, 200] = -254.0
    rows[7, 201:204] = torch.tensor([1.0, 3.0, -5.0])
    wc, ws = ref.pack(rows)
    codes, scales = kda.kda_act8_pack(rows.to(DEV))
    assert torch.equal(codes.cpu(), wc)
    assert torch.equal(scales.cpu().nan_to_num(-1), ws.nan_to_num(-1))
    assert codes.cpu()[0, :12].tolist() == [127, 0, 2, 2, 0, -2, -2, 126, 126, -126, 3, -127]
    back = kda.kda_act8_unpack(codes, scales, F32).cpu()
    assert torch.isnan(back[2, 128:]).all() and torch.isfinite(back[2, :128]).all()
    assert torch.isnan(back[3, :128]).all() and torch.isnan(back[4, :128]).all()
    assert torch.isfinite(back[6]).all() and (back[0, 128:] == 0).all()


def test_act8_random_quotients_near_ties():
    """fp32 rows whose values sit within a few steps of the middles between codes."""
    g = gen(17)
    amax = torch.rand(2000, 1, generator=g) * 10 + 0.1
    s = amax * torch.tensor(127.0).reciprocal()
    k = torch.randint(-126, 126, (2000, 127), generator=g).float() + 0.5
    x = (k.double() * s.double()).float()
    bits = x.view(torch.int32) + torch.randint(-2, 3, x.shape, generator=g).int()
    x = torch.cat([amax, bits.view(torch.float32)], 1)
    wc, ws = ref.pack(x)
    codes, scales = kda.kda_act8_pack(x.to(DEV))
    assert torch.equal(scales.cpu(), ws) and torch.equal(codes.cpu(), wc)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("dk,dv,lengths", [(128, 128, [70, 0, 129]), (64, 128, [200]), (128, 64, [65])])
def test_chunk_backwards_from_8_bit_checkpoints(io, dk, dv, lengths):
    """Bitwise the backward at the values that the codes stand for, through the
    calls and through autograd."""
    H, T, N = 3, sum(lengths), len(lengths)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = unit(randn((T, H, dk), 1)).to(io).to(DEV), unit(randn((T, H, dk), 2)).to(io).to(DEV)
    v, go = randn((T, H, dv), 3, io).to(DEV), randn((T, H, dv), 4, io).to(DEV)
    beta = torch.sigmoid(randn((T, H), 5)).to(io).to(DEV)
    la, sla = gate((T, H, dk), 6, io).to(DEV), gate((T, H), 7, io).to(DEV)
    h0, ghT = randn((N, H, dk, dv), 8, scale=0.1).to(DEV), randn((N, H, dk, dv), 9, scale=0.1).to(DEV)
    cu = cu_of(lengths) if N > 1 else None
    p8 = [kda.kda_act8_pack(t) for t in (q, k, v)]
    back = [kda.kda_act8_unpack(c, s, io) for c, s in p8]
    for gates, plain, packed, auto in ((la, kda.kda_chunk_bwd, kda.kda_chunk_bwd_act8, kda.chunk_kda),
                                       (sla, kda.kda_gdn_chunk_bwd, kda.kda_gdn_chunk_bwd_act8,
                                        kda.chunk_gated_delta_rule),
                                       (None, kda.kda_gdn_chunk_bwd, kda.kda_gdn_chunk_bwd_act8, None)):
        want = plain(*back, gates, beta, go, h0=h0, grad_hT=ghT, cu_seqlens=cu)
        got = packed(*p8, gates, beta, go, h0=h0, grad_hT=ghT, cu_seqlens=cu)
        for a, b in zip(got, want):
            assert (a is None and b is None) or torch.equal(a, b)
        if auto is not None:
            leaves = [t.clone().requires_grad_() for t in (q, k, v, gates, beta, h0)]
            o, hT = auto(*leaves, cu, act8=True)
            plain_o, plain_hT = auto(q, k, v, gates, beta, h0, cu)
            assert torch.equal(o, plain_o) and torch.equal(hT, plain_hT)
            torch.autograd.backward([o, hT], [go, ghT])
            for leaf, b in zip(leaves, want):
                assert torch.equal(leaf.grad, b)


# ------------------------------------------------------------------- RMS norm
NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (1000, 128), (4, 129), (9, 1000), (2, 1024), (33, 2048), (3, 4096), (2, 5000),
               (2, 8192), (2, 16384), (3, 20001), (700, 256), (1, 512), (130, 96)]


@pytest.mark.parametrize("io,wt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_rmsnorm(rows, cols, io, wt):
    eps = 1e-5
    x, res = randn((rows, cols), 1, io), randn((rows, cols), 2, io, scale=2.0)
    w = (1 + 0.2 * randn((cols,), 3)).to(wt)
    gy, gr = randn((rows, cols), 4, io), randn((rows, cols), 5, io)
    if rows > 1:
        x[1], res[1] = 0, 0               # a row of zeros
    for put in (lambda t: t.to(DEV), off_by_one):
        for residual, weight in ((res, w), (None, w), (res, None)):
            if put is off_by_one and weight is None:
                continue
            r, y, rstd, rel = ref.norm_fwd(x, weight, residual, eps)
            gp = lambda t: None if t is None else put(t)  # noqa: E731
            yg, rg, rsg = kda.kda_rmsnorm_fwd(put(x), gp(weight), gp(residual), eps)
            assert torch.equal(rg.cpu(), r)
            ref.assert_within(yg, y, rel * y.abs(), "y")
            ref.assert_within(rsg, rstd, rel * rstd, "rstd")
            codes, scales, rg, rs8 = kda.kda_rmsnorm_fwd_act8(put(x), gp(weight), gp(residual), eps)
            assert torch.equal(rg.cpu(), r) and torch.equal(rs8, rsg)
            _, ws = ref.pack(y)
            ref.assert_within(scales, ws.double(), rel * ws.double() + U(ws), "scales")
            half = scales.cpu().double().repeat_interleave(128, 1)[:, :cols] / 2
            got = ref.unpack(codes.cpu(), scales.cpu())
            assert ((got - y).abs() <= half * (1 + 1e-6) + (rel + 2.0 ** -22) * y.abs()).all()
            # backward, from r and from its 8-bit form
            pc, ps = kda.kda_act8_pack(rg)
            for g_r in (gr, None):
                dx, dw, E, Ew = ref.norm_bwd(r, weight, rsg.cpu(), gy, g_r)
                dxg, dwg = kda.kda_rmsnorm_bwd(put(r), gp(weight), rsg, put(gy), gp(g_r))
                ref.assert_within(dxg, dx, E, "dx")
                ref.assert_within(dwg, dw, Ew, "dw")
                back = ref.unpack(pc.cpu(), ps.cpu())
                dx, dw, E, Ew = ref.norm_bwd(back, weight, rsg.cpu(), gy, g_r)
                dxg, dwg = kda.kda_rmsnorm_bwd_act8(put(pc), put(ps), gp(weight), rsg, put(gy), gp(g_r))
                ref.assert_within(dxg, dx, E + 3 * ref.U32 * dx.abs(), "dx (8-bit r)")
                ref.assert_within(dwg, dw, Ew * 1.5, "dw (8-bit r)")


def U(t):
    return 2 * ref.U32 * t.double()


def test_rmsnorm_in_place_and_guard_rows():
    rows, cols = 37, 516
    x, res = randn((rows, cols), 1, BF).to(DEV), randn((rows, cols), 2, BF).to(DEV)
    w = (1 + 0.2 * randn((cols,), 3)).to(BF).to(DEV)
    gy, gr = randn((rows, cols), 4, BF).to(DEV), randn((rows, cols), 5, BF).to(DEV)
    y, r, rstd = kda.kda_rmsnorm_fwd(x, w, res)
    for alias in (0, 1):
        a, b = x.clone(), res.clone()
        y2, r2, rs2 = kda.kda_rmsnorm_fwd(a, w, b, r=(a, b)[alias])
        assert torch.equal(y2, y) and torch.equal((a, b)[alias], r) and torch.equal(rs2, rstd)
    dx, dw = kda.kda_rmsnorm_bwd(r, w, rstd, gy, gr)
    for alias in (0, 1):
        a, b = gy.clone(), gr.clone()
        d2, w2 = kda.kda_rmsnorm_bwd(r, w, rstd, a, b, grad_x=(a, b)[alias])
        assert torch.equal(d2, dx) and torch.equal(w2, dw)
    buf = torch.full((rows + 2, cols), 9.0, dtype=BF, device=DEV)
    kda.kda_rmsnorm_fwd(x, w, res, y=buf[1:-1])
    assert (buf[0] == 9).all() and (buf[-1] == 9).all() and torch.equal(buf[1:-1], y)
    buf.fill_(9.0)
    kda.kda_rmsnorm_bwd(r, w, rstd, gy, gr, grad_x=buf[1:-1])
    assert (buf[0] == 9).all() and (buf[-1] == 9).all() and torch.equal(buf[1:-1], dx)


def test_rmsnorm_rows_of_none_and_rows_that_are_not_finite():
    w = torch.ones(40, device=DEV)
    e = torch.empty((0, 40), device=DEV)
    y, r, rstd = kda.kda_rmsnorm_fwd(e, w)
    assert y.shape == (0, 40) and rstd.shape == (0,)
    dx, dw = kda.kda_rmsnorm_bwd(e, w, rstd, e)
    assert dx.shape == (0, 40) and (dw == 0).all()
    x = randn((4, 300), 1)
    x[1, 299] = float("nan")
    x[2, 0] = float("inf")
    y, _, rstd = kda.kda_rmsnorm_fwd(x.to(DEV))
    codes, scales, _, _ = kda.kda_rmsnorm_fwd_act8(x.to(DEV))
    y = y.cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 0]) and (y[2, 1:] == 0).all()
    assert torch.isfinite(y[[0, 3]]).all() and torch.isfinite(scales.cpu()[[0, 3]]).all()
    assert torch.isnan(scales.cpu()[1]).all() and torch.isnan(scales.cpu()[2, 0])


@pytest.mark.parametrize("rows,cols", [(20000, 64), (3000, 1028)])
def test_rmsnorm_weight_gradient_over_many_rows(rows, cols):
    r, gy = randn((rows, cols), 1, BF), randn((rows, cols), 2, BF)
    w = torch.ones(cols)
    _, _, rstd = kda.kda_rmsnorm_fwd(r.to(DEV))
    dx, dw, E, _ = ref.norm_bwd(r, w, rstd.cpu(), gy, None)
    dxg, dwg = kda.kda_rmsnorm_bwd(r.to(DEV), w.to(DEV), rstd, gy.to(DEV))
    # terms of random sign: partial sums are about sqrt(n) terms large, and n roundings of them in one
    # chain add up to about n / sqrt(2) U32 of a term, i.e. under one U32 of the sum of magnitudes;
    # 64 of them leave room for six orders of luck and for any tree
    terms = (gy.double() * r.double() * rstd.cpu().double()[:, None]).abs()
    assert ((dwg.cpu().double() - dw).abs() <= terms.sum(0) * 64 * ref.U32).all()
    ref.assert_within(dxg, dx, E, "dx")
    again = kda.kda_rmsnorm_bwd(r.to(DEV), w.to(DEV), rstd, gy.to(DEV))
    assert torch.equal(again[0], dxg) and torch.equal(again[1], dwg)


@pytest.mark.parametrize("act8", [False, True])
def test_rms_norm_autograd_against_differences(act8):
    """Central differences of the 64-bit norm.  The difference's own error is of
    order eps^2; with the sum saved in 8 bits, dx and dw are off by what an error of
    half a scale in r does to them, bounded by evaluating the gradient's magnitudes:
    |d dx| <= rstd^2 (|wg| + 2 |m'|...) half, taken as 4 half rstd^2 max|wg|."""
    rows, cols, eps_n = 12, 160, 1e-5
    x, res, w = randn((rows, cols), 1), randn((rows, cols), 2), 1 + 0.2 * randn((cols,), 3)
    wy, wr = randn((rows, cols), 4), randn((rows, cols), 5)
    leaves = [t.to(DEV).requires_grad_() for t in (x, w, res)]
    y, r = kda.rms_norm(leaves[0], leaves[1], leaves[2], eps_n, act8=act8)
    ((y * wy.to(DEV)).sum() + (r * wr.to(DEV)).sum()).backward()
    assert torch.equal(leaves[0].grad, leaves[2].grad)

    def loss(x, w, res):
        r = x + res
        y = r / torch.sqrt(r.square().mean(-1, keepdim=True) + eps_n) * w
        return float((y * wy).sum() + (r * wr).sum())

    base = [x.double(), w.double(), res.double()]
    rd = (x + res).double()
    rstd = 1 / torch.sqrt(rd.square().mean(-1, keepdim=True) + eps_n)
    half = rd.abs().amax(-1, keepdim=True) / 127 / 2
    for i, step in ((0, 1e-5), (1, 1e-5)):
        v = randn(base[i].shape, 30 + i).double()
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + step * v, base[i] - step * v
        want = (loss(*hi) - loss(*lo)) / (2 * step)
        prod = leaves[i].grad.double().cpu() * v
        tol = 2e-6 * float(prod.abs().sum())
        if act8:
            if i == 0:
                tol += float((4 * half * rstd.square() * (w * wy).abs().amax(-1, keepdim=True) * v.abs()).sum())
            else:
                tol += float(((wy.abs() * rstd * half).sum(0) * v.abs()).sum())
        assert abs(float(prod.sum()) - want) <= tol, (i, float(prod.sum()), want, tol)


# ------------------------------------------------------------- used together
def test_a_recurrent_layer_trains_from_8_bit_checkpoints():
    """norm with residual -> recurrence and KDA on its output -> per-head norm, the
    backward of all of it from 8-bit checkpoints: the gradients against the same
    layer's without them.  Every saved value is off by at most half a scale (its
    block's largest magnitude / 254, at most 2% of the block's root mean square
    here), and each gradient is a sum of products of at most four of them: a
    relative distance below 0.08."""
    T, H, d = 300, 2, 64
    D = H * d
    x, res = randn((T, D), 1, BF).to(DEV), randn((T, D), 2, BF).to(DEV)
    w1, w2 = torch.ones(D, dtype=BF, device=DEV), torch.ones(d, dtype=BF, device=DEV)
    la = gate((T, D), 3, BF).to(DEV)
    beta = torch.sigmoid(randn((T, H), 4)).to(BF).to(DEV)
    go = randn((T, D), 5, BF).to(DEV)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    qk = [unit(randn((T, H, d), s)).to(BF).to(DEV) for s in (6, 7)]

    def layer(act8):
        leaves = [t.clone().requires_grad_() for t in (x, res, w1, la, w2, *qk)]
        xs, rs, a, g, b, q, k = leaves
        y, stream = kda.rms_norm(xs, a, rs, act8=act8)
        h, _ = kda.gated_linear_recurrence(y, g, act8=act8)
        o, _ = kda.chunk_kda(q, k, h.reshape(T, H, d), g.reshape(T, H, d), beta, act8=act8)
        z = kda.rms_norm(o.contiguous(), b, act8=act8).reshape(T, D) + stream
        z.backward(go)
        return z, [t.grad for t in leaves]

    z, exact = layer(False)
    z8, packed = layer(True)
    assert torch.equal(z, z8)
    for a, b in zip(exact, packed):
        a, b = a.double(), b.double()
        assert float((a - b).norm() / a.norm()) < 0.08


def test_prefill_then_decode_with_8_bit_norm_output():
    T, D = 130, 256
    x, res = randn((T, D), 1, BF).to(DEV), randn((T, D), 2, BF).to(DEV)
    la = gate((T, D), 3, BF).to(DEV)
    codes, scales, r, _ = kda.kda_rmsnorm_fwd_act8(x, None, res)
    inp = kda.kda_act8_unpack(codes, scales)
    h, S = kda.kda_glr_fwd(inp[:100], la[:100])
    outs = [h] + [kda.kda_glr_step(inp[t:t + 1], la[t:t + 1], S) for t in range(100, T)]
    want = ref.glr_fwd(inp.cpu(), la.cpu(), None, [T])
    ref.assert_within(torch.cat(outs), want[0], want[2], "h")


def test_calls_captured_into_graphs():
    """Two graphs of the same calls on their own workspaces, replayed in turn with
    new inputs and eager work between, against the eager calls."""
    T, D = 3000, 260
    x, la, h0, gh, ghT = [t.to(DEV) for t in glr_inputs([T], D, BF, BF, 3, "uniform")]
    w = torch.ones(D, dtype=BF, device=DEV)

    def calls():
        h, hT = kda.kda_glr_fwd(x, la, h0=h0)
        p = kda.kda_act8_pack(h)
        grads = kda.kda_glr_bwd_act8(la, *p, gh, h0=h0, grad_hT=ghT)
        y, r, rstd = kda.kda_rmsnorm_fwd(h, w, x)
        n = kda.kda_rmsnorm_bwd(r, w, rstd, gh)
        return (h, hT, *p, *grads, y, r, rstd, *n)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = calls()
        graphs.append((g, out))
    for k in range(4):
        x.copy_(randn((T, D), 50 + k, BF))
        gh.copy_(randn((T, D), 60 + k, BF))
        want = calls()
        torch.cuda.synchronize()
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own."""
    T, D = 6000, 384
    sets = [[t.to(DEV) for t in glr_inputs([T], D, BF, BF, 40 + k, "uniform")] for k in range(2)]
    want = [kda.kda_glr_fwd(s[0], s[1], h0=s[2]) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(kda.kda_glr_fwd(sets[k][0], sets[k][1], h0=sets[k][2]))
    torch.cuda.synchronize()
    for k in range(2):
        for h, hT in got[k]:
            assert torch.equal(h, want[k][0]) and torch.equal(hT, want[k][1])


def test_long_offsets():
    """More than 2^31 elements in one tensor: offsets pass 32 bits."""
    T, D = 70000, 32768
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    x = torch.zeros((T, D), dtype=BF, device=DEV)
    la = torch.full((T, D), float("-inf"), dtype=BF, device=DEV)
    tail = 300
    x[-tail:] = randn((tail, D), 1, BF).to(DEV)
    la[-tail + 1:] = gate((tail - 1, D), 2, BF).to(DEV)
    h, hT = kda.kda_glr_fwd(x, la)
    small, sT = kda.kda_glr_fwd(x[-tail:].contiguous(), la[-tail:].contiguous())
    assert float((h[-tail:].float() - small.float()).abs().max()) <= 2.0 ** -6
    assert float((hT - sT).abs().max()) <= 1e-4 and not h[:-tail].any()
    codes, scales = kda.kda_act8_pack(h)
    wc, ws = kda.kda_act8_pack(h[-tail:].contiguous())
    assert torch.equal(codes[-tail:], wc) and torch.equal(scales[-tail:], ws)
    back = kda.kda_act8_unpack(codes, scales)
    assert torch.equal(back[-tail:], kda.kda_act8_unpack(wc, ws))
    del back
    y, _, rstd = kda.kda_rmsnorm_fwd(h)
    y2, _, _ = kda.kda_rmsnorm_fwd(h[-tail:].contiguous())
    assert torch.equal(y[-tail:], y2)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_on_another_device():
    x, la, h0, _, _ = glr_inputs([700], 128, BF, BF, 3, "uniform")
    want = kda.kda_glr_fwd(x.to(DEV), la.to(DEV), h0=h0.to(DEV))
    got = kda.kda_glr_fwd(x.to("cuda:1"), la.to("cuda:1"), h0=h0.to("cuda:1"))
    assert all(torch.equal(a.cpu(), b.cpu()) for a, b in zip(got, want))



def test_binding_refusals():
    """Shapes, types, devices and strides that do not fit are refused before any launch."""
    x = torch.zeros((6, 256), dtype=BF, device=DEV)
    la, f = torch.zeros_like(x), torch.zeros((1, 256), device=DEV)
    codes, scales = kda.kda_act8_pack(x)
    rstd, w = torch.zeros(6, device=DEV), torch.zeros(256, device=DEV)
    bad = [
        lambda: kda.kda_glr_fwd(x, la[:5]), lambda: kda.kda_glr_fwd(x.t(), la.t()),
        lambda: kda.kda_glr_fwd(x, la, h0=f.to(BF)), lambda: kda.kda_glr_fwd(x, la, h0=torch.cat([f, f])),
        lambda: kda.kda_glr_fwd(x, la, cu_seqlens=cu_of([6]).long()), lambda: kda.kda_glr_fwd(x, la.cpu()),
        lambda: kda.kda_glr_fwd(x.half(), la), lambda: kda.kda_glr_fwd(x, la, h=torch.zeros_like(x[:5])),
        lambda: kda.kda_glr_fwd(x[0], la[0]), lambda: kda.kda_glr_fwd(x[:, ::2], la[:, ::2]),
        lambda: kda.kda_glr_bwd(la, x.float(), x), lambda: kda.kda_glr_bwd(la, x, x, grad_hT=f[:, :5]),
        lambda: kda.kda_glr_bwd_act8(la, codes, scales[:, :1], x), lambda: kda.kda_glr_bwd_act8(la, x, scales, x),
        lambda: kda.kda_glr_step(x, la, torch.zeros_like(x)), lambda: kda.kda_glr_step(x[0], la[0], f[0]),
        lambda: kda.kda_act8_pack(x.t()), lambda: kda.kda_act8_pack(x.half()), lambda: kda.kda_act8_pack(x[:, :0]),
        lambda: kda.kda_act8_unpack(codes, scales[:5]), lambda: kda.kda_act8_unpack(x, scales),
        lambda: kda.kda_act8_unpack(codes, scales, torch.float16),
        lambda: kda.kda_rmsnorm_fwd(x, w[:5]), lambda: kda.kda_rmsnorm_fwd(x, w, x.float()),
        lambda: kda.kda_rmsnorm_fwd(x, w, r=x), lambda: kda.kda_rmsnorm_fwd(x, w.half()),
        lambda: kda.kda_rmsnorm_bwd(x, w, rstd[:5], x), lambda: kda.kda_rmsnorm_bwd(x, w, rstd, x, x.float()),
        lambda: kda.kda_rmsnorm_bwd_act8(codes, scales[:, :1], w, rstd, x),
    ]
    for k, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail("call %d was taken" % k)
    for call in (lambda: kda.kda_rmsnorm_fwd(x, w, eps=0.0), lambda: kda.kda_rmsnorm_fwd(x, w, eps=float("nan")),
                 lambda: kda.kda_glr_fwd(x[None].repeat(2, 1, 1), la[None].repeat(2, 1, 1), cu_seqlens=cu_of([6, 6]))):
        with pytest.raises(kda.KDAError) as e:
            call()
        assert e.value.code == kda.KDA_ERR_INVALID_ARGUMENT
    big = torch.zeros((9000, 256), dtype=BF, device=DEV)
    if kda.kda_glr_workspace_size(1, 9000, 256, 0, kda.KDA_BF16):
        with pytest.raises(kda.KDAError) as e:
            kda.kda_glr_fwd(big, big, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
        assert e.value.code == kda.KDA_ERR_WORKSPACE


@pytest.mark.parametrize("act8", [False, True])
def test_second_derivatives_are_refused(act8):
    """The gradients are the library's own and have no formula of a second order:
    asking for one is an error, not a gradient that leaves a part out."""
    x = randn((1, 5, 3), 1).to(DEV).requires_grad_()
    g = gate((1, 5, 3), 2).to(DEV)
    for y in (kda.gated_linear_recurrence(x, g, act8=act8)[0], kda.rms_norm(x, act8=act8)):
        (dx,) = torch.autograd.grad((y * y).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            dx.sum().backward()


@pytest.mark.parametrize("act8", [False, True])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("D", [3, 64, 130])
def test_glr_infinities_last_until_a_reset(D, io, act8):
    """An infinity or a NaN stays in the state however far its factor has decayed,
    as in the formula (alpha > 0 times infinity), and ends at a reset; the other
    channels do not see it."""
    T, reset = 5000, 4000
    inf = float("inf")
    x, g = randn((T, D), 1, io).to(DEV), gate((T, D), 2, io, "uniform").to(DEV)
    g[:, 2] = -6.0                      # decays within a span
    g[reset] = -inf
    clean, _ = kda.kda_glr_fwd(x, g)
    y = x.clone()
    y[7, 0], y[9, 1], y[11, 2] = inf, float("nan"), -inf
    h, hT = kda.kda_glr_fwd(y, g)
    assert (h[7:reset, 0] == inf).all() and h[9:reset, 1].isnan().all() and (h[11:reset, 2] == -inf).all()
    for c, t in ((0, 7), (1, 9), (2, 11)):
        assert torch.equal(h[:t, c], clean[:t, c])
    assert torch.equal(h[reset:], clean[reset:]) and torch.equal(h[:, 3:], clean[:, 3:])
    assert hT.isfinite().all()

    saved = kda.kda_act8_pack(clean) if act8 else (clean,)
    bwd = kda.kda_glr_bwd_act8 if act8 else kda.kda_glr_bwd
    want, _, _ = bwd(g, *saved, x)
    y = x.clone()
    y[T - 7, 0], y[reset - 9, 1], y[reset - 11, 2] = inf, float("nan"), -inf
    dx, _, dh0 = bwd(g, *saved, y)
    assert (dx[reset:T - 6, 0] == inf).all() and torch.equal(dx[:reset, 0], want[:reset, 0])
    assert dx[:reset - 8, 1].isnan().all() and (dx[:reset - 10, 2] == -inf).all()
    assert torch.equal(dx[reset:, 1:], want[reset:, 1:]) and torch.equal(dx[:, 3:], want[:, 3:])
    assert dh0[0, 1].isnan() and dh0[0, 2] == -inf and dh0[0, 0].isfinite()
