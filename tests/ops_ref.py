"""Plain 64-bit implementations of the gated linear recurrence, the 8-bit
activation format and the RMS norm, and first-order bounds on what fp32
arithmetic may differ from them by (CPU, torch float64)."""
import torch

BLOCK = 128
U32 = 2.0 ** -24          # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def glr_fwd(x, la, h0, lengths):
    """x, la: [T, D]; h0: [N, D] or None.  Returns h, h_T and a bound of the fp32
    error of each, all float64.

    With e_t the relative error of one decay factor and its product (the
    exponential of la: its argument la * log2(e) is rounded, an absolute error of
    |la| U32 in the exponent, then the exponential, the product and, where spans
    of tokens are composed, the span's products: 8 roundings in all), and H the
    recurrence of the magnitudes, the error obeys E_t = a_t (E_{t-1} + e_t
    H_{t-1}) + U32 H_t."""
    x, la = x.double(), la.double()
    T, D = x.shape
    a = la.exp()
    e = (8 + 2 * la.abs().clamp_max(200)) * U32
    h, E = torch.zeros(T, D).double(), torch.zeros(T, D).double()
    hT, ET = torch.zeros(len(lengths), D).double(), torch.zeros(len(lengths), D).double()
    t = 0
    for n, length in enumerate(lengths):
        s = torch.zeros(D).double() if h0 is None else h0[n].double()
        m, err = s.abs(), torch.zeros(D).double()
        for _ in range(length):
            reset = a[t] == 0
            err = torch.where(reset, 0.0, a[t] * (err + e[t] * m))
            s = torch.where(reset, 0.0, a[t] * s) + x[t]
            m = torch.where(reset, 0.0, a[t] * m) + x[t].abs()
            err = err + U32 * m
            h[t], E[t] = s, err
            t += 1
        hT[n], ET[n] = s, err
    return h, hT, E, ET


def glr_bwd(la, h, gh, h0, ghT, lengths):
    """Gradients (dx, dla, dh0) and their fp32 error bounds, as glr_fwd.  The last
    rounding of dla's product is a U32 of its own."""
    la, h, gh = la.double(), h.double(), gh.double()
    T, D = la.shape
    a = la.exp()
    e = (8 + 2 * la.abs().clamp_max(200)) * U32
    z = lambda *s: torch.zeros(*s).double()  # noqa: E731
    dx, dla, dh0 = z(T, D), z(T, D), z(len(lengths), D)
    Ex, El, E0 = z(T, D), z(T, D), z(len(lengths), D)
    end = sum(lengths)
    for n in reversed(range(len(lengths))):
        c = z(D) if ghT is None else ghT[n].double()
        m, err = c.abs(), z(D)
        for t in reversed(range(end - lengths[n], end)):
            reset = a[t] == 0
            g = gh[t] + c
            gm = gh[t].abs() + m
            err = err + U32 * gm
            dx[t], Ex[t] = g, err
            c = torch.where(reset, 0.0, a[t] * g)
            m = torch.where(reset, 0.0, a[t] * gm)
            err = torch.where(reset, 0.0, a[t] * (err + e[t] * gm))
            if t == end - lengths[n]:
                prev = z(D) if h0 is None else h0[n].double()
            else:
                prev = h[t - 1]
            dla[t] = torch.where(reset, 0.0, prev * c)
            El[t] = torch.where(reset, 0.0, prev.abs() * (err + 2 * U32 * c.abs()))
        dh0[n], E0[n] = c, err
        end -= lengths[n]
    return dx, dla, dh0, Ex, El, E0


def blocks(cols):
    return -(-cols // BLOCK)


def pack(v):
    """codes (int8) and scales (float32) of v [rows, cols], any float type."""
    rows, cols = v.shape
    wide = torch.zeros(rows, blocks(cols) * BLOCK, dtype=torch.float64)
    wide[:, :cols] = v.double()
    wide = wide.reshape(rows, -1, BLOCK)
    amax = wide.abs().amax(-1)          # NaN stays NaN
    scale = (amax.float() * torch.tensor(127.0).reciprocal()).double().clamp_min(2.0 ** -126)
    bad = ~torch.isfinite(amax)
    q = torch.round(wide / scale[..., None])
    q = torch.where(bad[..., None], 0.0, q)
    scale = torch.where(bad, float("nan"), scale)
    return q.reshape(rows, -1)[:, :cols].to(torch.int8), scale.float()


def unpack(codes, scales):
    rows, cols = codes.shape
    s = scales.double().repeat_interleave(BLOCK, 1)[:, :cols]
    return codes.double() * s


def norm_fwd(x, w, res, eps):
    """r (in x's type), y and rstd in float64, the bound of y's and rstd's fp32
    relative error.  The sum of squares adds cols non-negative terms, at most
    cols / 64 of them one after another and 16 levels above: a relative error of
    at most that many U32, halved by the square root; the mean, the root, the
    reciprocal and eps's addition take 6 more, and y's two products 2."""
    r = x if res is None else (x.float() + res.float()).to(x.dtype)
    rd = r.double()
    rstd = 1.0 / torch.sqrt(rd.square().mean(-1) + eps)
    wd = torch.ones(x.shape[-1]).double() if w is None else w.double()
    y = rd * rstd[:, None] * wd
    rel = (x.shape[-1] / 64 + 16 + 12) / 2 * U32
    return r, y, rstd, rel


def norm_bwd(r, w, rstd, gy, gr):
    """dx, dw in float64 and bounds of their fp32 errors: m is a sum of cols
    products of three factors (depth cols / 64 + 16), dx four more roundings, dw a
    sum over rows of products (any order: at most rows of them) in fp32."""
    r, rs, gy = r.double(), rstd.double()[:, None], gy.double()
    rows, cols = r.shape
    wd = torch.ones(cols).double() if w is None else w.double()
    m = (r * wd * gy).mean(-1, keepdim=True)
    mabs = (r * wd * gy).abs().mean(-1, keepdim=True)
    dx = rs * (wd * gy - r * rs.square() * m)
    E = rs * (4 * U32 * (wd * gy).abs() + r.abs() * rs.square() * (cols / 64 + 16 + 10) * U32 * mabs)
    if gr is not None:
        dx = dx + gr.double()
        E = E + U32 * dx.abs()
    dw = (gy * r * rs).sum(0)
    Ew = (gy * r * rs).abs().sum(0) * (rows + 4) * U32
    return dx, dw, E, Ew


def assert_within(got, want, err, name):
    """|got - want| within the fp32 bound plus half a step of got's type (of the
    value the type rounds, which may be off by the bound itself)."""
    got, hs = got.detach().cpu(), half_step(got.dtype)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    tol = err + hs * (want.abs() + err) * (got.dtype != torch.float32)
    tol = tol + U32 * want.abs() + torch.finfo(torch.float32).tiny
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), "%s: %d values off, worst %g of %g allowed" % (
        name, int(bad.sum()), float((got.double() - want).abs()[bad].max()), float(tol[bad].min()))
