"""CPU tests of the C ABI of the gated linear recurrence, the 8-bit activation
checkpoints and the RMS norm: invalid arguments are refused on the host, before
any HIP call, and the autograd functions and bindings refuse CPU tensors."""
import math
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_chunkwise_amd", "csrc")
P = 1 << 20   # a fake, aligned "device" address; never dereferenced
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def kda():
    import gated_delta_rule_chunkwise_amd as kda
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_chunkwise_amd import build
        build.build()
    kda.load_library()
    return kda


def glr_fwd(lib, **kw):
    a = dict(x=P, la=P, h0=None, cu=None, N=0, h=P, hT=P, B=1, T=100, D=64, io=1, gt=1, ws=None, wsb=0)
    a.update(kw)
    return lib.kda_glr_fwd(*[a[k] for k in ("x", "la", "h0", "cu", "N", "h", "hT", "B", "T", "D", "io", "gt", "ws",
                                            "wsb")], None)


def glr_bwd(lib, **kw):
    a = dict(la=P, h=P, h0=None, cu=None, N=0, gh=P, ghT=None, dx=P, dla=P, dh0=P, B=1, T=100, D=64, io=1, gt=1,
             ws=None, wsb=0)
    a.update(kw)
    return lib.kda_glr_bwd(*[a[k] for k in ("la", "h", "h0", "cu", "N", "gh", "ghT", "dx", "dla", "dh0", "B", "T",
                                            "D", "io", "gt", "ws", "wsb")], None)


def glr_bwd8(lib, **kw):
    a = dict(la=P, c=P, s=P, h0=None, cu=None, N=0, gh=P, ghT=None, dx=P, dla=P, dh0=P, B=1, T=100, D=64, io=1, gt=1,
             ws=None, wsb=0)
    a.update(kw)
    return lib.kda_glr_bwd_act8(*[a[k] for k in ("la", "c", "s", "h0", "cu", "N", "gh", "ghT", "dx", "dla", "dh0",
                                                 "B", "T", "D", "io", "gt", "ws", "wsb")], None)


SIZES = [(dict(io=2), UNSUPPORTED), (dict(gt=-1), UNSUPPORTED), (dict(B=0), INVALID), (dict(T=-1), INVALID),
         (dict(D=0), INVALID), (dict(cu=P, N=2, B=2), INVALID), (dict(cu=P, N=0), INVALID),
         (dict(cu=P + 2, N=2), INVALID), (dict(N=3), INVALID), (dict(h0=P + 2), INVALID),
         (dict(B=1 << 30, T=1 << 30, D=1 << 20), INVALID), (dict(ws=P + 8, wsb=1 << 60), INVALID)]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(x=None), INVALID), (dict(la=None), INVALID), (dict(h=None), INVALID), (dict(x=P + 1), INVALID),
    (dict(x=P + 2, io=0), INVALID), (dict(la=P + 2, gt=0), INVALID), (dict(hT=P + 2), INVALID),
    (dict(T=0, x=None, la=None, h=None, hT=None), OK)])
def test_glr_fwd_refusals(kda, kw, code):
    assert glr_fwd(kda.load_library(), **kw) == code


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(la=None), INVALID), (dict(gh=None), INVALID), (dict(dx=None), INVALID), (dict(dla=None), INVALID),
    (dict(ghT=P + 2), INVALID), (dict(dh0=P + 1), INVALID), (dict(dla=P + 2, gt=0), INVALID),
    (dict(T=0, la=None, gh=None, dx=None, dla=None, dh0=None), OK)])
def test_glr_bwd_refusals(kda, kw, code):
    lib = kda.load_library()
    assert glr_bwd(lib, **kw) == code
    assert glr_bwd8(lib, **kw) == code


def test_rows_beyond_32_bit_positions_are_refused(kda):
    lib = kda.load_library()
    big = (1 << 30) + 1
    assert glr_fwd(lib, T=1, D=big) == glr_bwd(lib, T=1, D=big) == glr_bwd8(lib, T=1, D=big) == UNSUPPORTED
    assert kda.kda_glr_workspace_size(1, 5000, big) == 0
    assert lib.kda_act8_pack(P, P, P, 1, big, 1, None) == UNSUPPORTED
    assert lib.kda_act8_unpack(P, P, P, 1, big, 1, None) == UNSUPPORTED
    assert lib.kda_rmsnorm_fwd(P, None, None, P, None, None, 1, big, 1e-6, 1, 1, None) == UNSUPPORTED
    assert lib.kda_rmsnorm_bwd(P, None, P, P, None, P, None, 1, big, 1, 1, None, 0, None) == UNSUPPORTED
    assert kda.kda_rmsnorm_bwd_workspace_size(1, big) == 0


def test_glr_bwd_saved_h(kda):
    lib = kda.load_library()
    assert glr_bwd(lib, h=None) == INVALID
    assert glr_bwd(lib, h=P + 1) == INVALID
    assert glr_bwd8(lib, c=None) == INVALID
    assert glr_bwd8(lib, s=None) == INVALID
    assert glr_bwd8(lib, s=P + 2) == INVALID


def test_glr_workspace(kda):
    lib = kda.load_library()
    size = kda.kda_glr_workspace_size
    need = size(1, 65536, 4096, 0, kda.KDA_BF16)
    assert need <= 0.15 * 65536 * 4096 + (1 << 20)
    assert size(1, 1, 4096) == size(1, 64, 64) == 0
    assert size(0, 10, 10) == size(1, -1, 10) == size(1, 10, 0) == size(2, 10, 10, 3) == size(1, 10, 10, 0, 7) == 0
    if need:
        assert glr_fwd(lib, T=65536, D=4096) == WORKSPACE
        assert glr_fwd(lib, T=65536, D=4096, ws=P, wsb=need - 1) == WORKSPACE
        assert glr_bwd(lib, T=65536, D=4096, ws=P, wsb=need - 1) == WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(io=9), UNSUPPORTED), (dict(gt=9), UNSUPPORTED), (dict(B=0), INVALID), (dict(D=-1), INVALID),
    (dict(x=None), INVALID), (dict(la=None), INVALID), (dict(S=None), INVALID), (dict(h=None), INVALID),
    (dict(S=P + 2), INVALID), (dict(la=P + 2, gt=0), INVALID), (dict(B=1 << 30, D=1 << 12), UNSUPPORTED)])
def test_glr_step_refusals(kda, kw, code):
    a = dict(x=P, la=P, S=P, h=P, B=4, D=64, io=1, gt=1)
    a.update(kw)
    assert kda.load_library().kda_glr_step(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(io=3), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(x=None), INVALID),
    (dict(x=P + 1), INVALID), (dict(x=P + 2, io=0), INVALID), (dict(c=None), INVALID), (dict(s=None), INVALID),
    (dict(s=P + 2), INVALID), (dict(rows=0, x=None, c=None, s=None), OK), (dict(rows=1 << 49, cols=1 << 10), INVALID),
    (dict(rows=1 << 40), UNSUPPORTED)])
def test_act8_refusals(kda, kw, code):
    a = dict(x=P, c=P, s=P, rows=10, cols=128, io=1)
    a.update(kw)
    lib = kda.load_library()
    assert lib.kda_act8_pack(a["x"], a["c"], a["s"], a["rows"], a["cols"], a["io"], None) == code
    assert lib.kda_act8_unpack(a["c"], a["s"], a["x"], a["rows"], a["cols"], a["io"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(io=3), UNSUPPORTED), (dict(wt=3), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(x=None), INVALID), (dict(x=P + 1), INVALID), (dict(res=P, r=None), INVALID), (dict(res=P + 1), INVALID),
    (dict(r=P + 1, res=P), INVALID), (dict(w=P + 1), INVALID), (dict(w=P + 2, wt=0), INVALID),
    (dict(rstd=P + 2), INVALID), (dict(rows=0, x=None, y=None, s=None), OK), (dict(rows=1 << 40), UNSUPPORTED),
    (dict(y=None), INVALID)])
def test_rmsnorm_fwd_refusals(kda, kw, code):
    a = dict(x=P, res=None, w=P, y=P, s=P, r=None, rstd=P, rows=10, cols=128, eps=1e-6, io=1, wt=1)
    a.update(kw)
    lib = kda.load_library()
    tail = [a[k] for k in ("r", "rstd", "rows", "cols", "eps", "io", "wt")]
    assert lib.kda_rmsnorm_fwd(a["x"], a["res"], a["w"], a["y"], *tail, None) == code
    assert lib.kda_rmsnorm_fwd_act8(a["x"], a["res"], a["w"], a["y"], a["s"], *tail, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(io=3), UNSUPPORTED), (dict(wt=3), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(r=None), INVALID), (dict(rstd=None), INVALID), (dict(rstd=P + 2), INVALID), (dict(gy=None), INVALID),
    (dict(gy=P + 1), INVALID), (dict(gr=P + 1), INVALID), (dict(gx=None), INVALID), (dict(gw=P + 1), INVALID),
    (dict(gw=P + 2, wt=0), INVALID), (dict(w=P + 1), INVALID), (dict(rows=1 << 40), UNSUPPORTED),
    (dict(rows=0, gw=None, r=None, gy=None, gx=None, rstd=None), OK), (dict(ws=P + 8), INVALID)])
def test_rmsnorm_bwd_refusals(kda, kw, code):
    a = dict(r=P, s=P, w=P, rstd=P, gy=P, gr=None, gx=P, gw=P, rows=10, cols=128, io=1, wt=1, ws=P, wsb=1 << 60)
    a.update(kw)
    lib = kda.load_library()
    tail = [a[k] for k in ("w", "rstd", "gy", "gr", "gx", "gw", "rows", "cols", "io", "wt", "ws", "wsb")]
    assert lib.kda_rmsnorm_bwd(a["r"], *tail, None) == code
    assert lib.kda_rmsnorm_bwd_act8(a["r"], a["s"], *tail, None) == code


def test_rmsnorm_bwd_workspace(kda):
    lib = kda.load_library()
    assert kda.kda_rmsnorm_bwd_workspace_size(-1, 5) == kda.kda_rmsnorm_bwd_workspace_size(5, 0) == 0
    need = kda.kda_rmsnorm_bwd_workspace_size(65536, 4096)
    assert need <= 64 << 20
    if need:
        assert lib.kda_rmsnorm_bwd(P, P, P, P, None, P, P, 65536, 4096, 1, 1, P, need - 1, None) == WORKSPACE
        assert lib.kda_rmsnorm_bwd(P, P, P, P, None, P, P, 65536, 4096, 1, 1, None, need, None) == WORKSPACE


def chunk8(lib, fn="kda_chunk_bwd_act8", **kw):
    a = dict(qc=P, qs=P, kc=P, ks=P, vc=P, vs=P, la=P, beta=P, h0=None, cu=None, N=0, go=P, ghT=None, dq=P, dk=P,
             dv=P, dla=P, db=P, dh0=P, B=1, T=128, H=2, d_k=128, d_v=128, io=1, gt=1, ws=P, wsb=0)
    a.update(kw)
    return getattr(lib, fn)(*a.values(), None)


@pytest.mark.parametrize("fn", ["kda_chunk_bwd_act8", "kda_gdn_chunk_bwd_act8"])
@pytest.mark.parametrize("kw,code", [
    (dict(d_k=96), UNSUPPORTED), (dict(io=4), UNSUPPORTED), (dict(gt=9), UNSUPPORTED), (dict(B=0), INVALID),
    (dict(T=-1), INVALID), (dict(beta=None), INVALID), (dict(go=None), INVALID), (dict(dq=P + 4), INVALID),
    (dict(h0=P + 4), INVALID), (dict(cu=P, N=2, B=2), INVALID), (dict(N=3), INVALID), (dict(ws=P + 8), INVALID),
    (dict(H=65536, T=1), UNSUPPORTED), (dict(), WORKSPACE), (dict(ws=None), WORKSPACE),
    (dict(qc=None), INVALID), (dict(ks=None), INVALID), (dict(vs=P + 2), INVALID)])
def test_chunk_bwd_act8_refusals(kda, fn, kw, code):
    lib = kda.load_library()
    assert chunk8(lib, fn, **kw) == code
    need = kda.kda_chunk_bwd_act8_workspace_size(1, 128, 2, 128, 128, 0, kda.KDA_BF16)
    base = kda.kda_chunk_bwd_workspace_size(1, 128, 2, 128, 128, 0, kda.KDA_BF16)
    assert need >= base + 3 * 128 * 2 * 128 * 2
    if code == WORKSPACE:
        assert chunk8(lib, fn, wsb=need - 1) == WORKSPACE


def test_chunk_bwd_act8_workspace_of_refused_sizes(kda):
    size = kda.kda_chunk_bwd_act8_workspace_size
    assert size(1, 100, 2, 96, 128) == size(2, 100, 2, 64, 64, 3) == size(0, 100, 2, 64, 64) == 0
    assert size(1, 100, 2, 64, 64, 0, 5) == 0


def test_bindings_refuse_cpu_tensors(kda):
    x = torch.zeros(4, 8)
    s = torch.zeros(4, 1)
    c = torch.zeros(4, 8, dtype=torch.int8)
    for call in (lambda: kda.kda_glr_fwd(x, x), lambda: kda.kda_glr_bwd(x, x, x), lambda: kda.kda_glr_step(x, x, x),
                 lambda: kda.kda_glr_bwd_act8(x, c, s, x), lambda: kda.kda_act8_pack(x),
                 lambda: kda.kda_act8_unpack(c, s), lambda: kda.kda_rmsnorm_fwd(x), lambda: kda.rms_norm(x),
                 lambda: kda.kda_rmsnorm_fwd_act8(x), lambda: kda.kda_rmsnorm_bwd(x, None, s[:, 0], x),
                 lambda: kda.gated_linear_recurrence(x, x),
                 lambda: kda.kda_chunk_bwd_act8((c, s), (c, s), (c, s), x, x, x[:, None])):
        with pytest.raises(ValueError):
            call()


def test_largest_scale(kda):
    """The largest scale of the 8-bit form times 127 is finite in fp32, the next one's is not."""
    s = torch.tensor(2.67938851e36)
    assert math.isfinite(float(s * 127)) and not math.isfinite(float(torch.nextafter(s, torch.tensor(math.inf)) * 127))


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_validation_under_asan_and_ubsan(tmp_path):
    """kda_ops_api.cpp beside kda_api.cpp, with host-only launchers, under the
    address and undefined-behaviour sanitizers."""
    exe = str(tmp_path / "ops_driver")
    here = os.path.join(ROOT, "tests", "host_sanitize")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "kda_api.cpp"), os.path.join(CSRC, "kda_ops_api.cpp"),
           os.path.join(here, "stub_launchers.cpp"), os.path.join(here, "ops_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "ops driver: ok" in r.stdout
