"""CPU tests of the block operators' C ABI (include/block/): the library
exports what the headers declare and rejects bad arguments before any HIP call
(pointers here are fake and never read), and the ABI layer runs clean under
AddressSanitizer / UndefinedBehaviorSanitizer with its launches replaced."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from selective_state_space_56_amd import block as bk
from selective_state_space_56_amd import binding as bd
from test_sanitizers import ENV, SAN

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = os.path.join(ROOT, "include", "block")
INVALID, UNSUPPORTED = 1, 2
FAKE = 0x7F0000000000
NAMES = {"mamba_gated_scan_workspace_size", "mamba_gated_scan_bwd_workspace_size", "mamba_gated_scan_fwd",
         "mamba_gated_scan_bwd", "mamba_gated_update", "mamba_rmsnorm_fwd", "mamba_rmsnorm_quant_fwd",
         "mamba_rmsnorm_bwd_workspace_size", "mamba_rmsnorm_bwd", "mamba_conv1d_bwd_workspace_size",
         "mamba_conv1d_bwd"}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from selective_state_space_56_amd.build import build
        build()
    return bk._library()


def err(lib):
    return lib.mamba_last_error().decode()


def P(k):
    """A fake device address; an int is the k-th region of 1 MiB."""
    return None if k is None else FAKE + 0x100000 * k if isinstance(k, int) and k < 1000 else k


def test_exports_every_declared_symbol(lib):
    names = set()
    for h in os.listdir(HEADERS):
        src = re.sub(r"/\*.*?\*/", "", open(os.path.join(HEADERS, h)).read(), flags=re.S)
        names |= set(re.findall(r"\b(mamba_[a-z0-9_]+)\s*\(", src))
    assert names == NAMES
    for n in names:
        assert hasattr(lib, n)


def gd(batch=2, seqlen=8, dim=16, io=1, flags=0):
    return bk.GatedDesc(batch, seqlen, dim, io, flags)


def ptrs(order, given, base):
    v = dict(zip(order, range(1, 1 + len(order))))
    v.update(given)
    return [P(v[n]) for n in order]


FWD = ["x", "r", "g", "A", "h0", "reset", "out", "last", "ck"]
BWD = ["x", "r", "g", "A", "reset", "ck", "dout", "dlast", "dx", "dr", "dg", "dA", "dh0"]
UPD = ["state", "x", "r", "g", "A", "out"]


def fwd(lib, d, s=None, ws=50, ws_bytes=1 << 40, **kw):
    return lib.mamba_gated_scan_fwd(None if d is None else ctypes.byref(d), None if s is None else ctypes.byref(s),
                                    *ptrs(FWD, kw, 1), P(ws), ws_bytes if ws_bytes is not None else 0, None)


def bwd(lib, d, s=None, ws=50, ws_bytes=1 << 40, **kw):
    return lib.mamba_gated_scan_bwd(ctypes.byref(d), None if s is None else ctypes.byref(s), *ptrs(BWD, kw, 1), P(ws),
                                    ws_bytes, None)


def upd(lib, d, s=None, **kw):
    return lib.mamba_gated_update(ctypes.byref(d), None if s is None else ctypes.byref(s), *ptrs(UPD, kw, 1), None)


def test_gated_descriptors(lib):
    assert fwd(lib, None) == INVALID and "desc is NULL" in err(lib)
    for kw in (dict(batch=-1), dict(seqlen=-1), dict(dim=-1), dict(io=2), dict(flags=1)):
        assert fwd(lib, gd(**kw)) == INVALID and bwd(lib, gd(**kw)) == INVALID, kw
        assert lib.mamba_gated_scan_workspace_size(ctypes.byref(gd(**kw))) == 0
        assert lib.mamba_gated_scan_bwd_workspace_size(ctypes.byref(gd(**kw))) == 0
    for kw in (dict(dim=(1 << 26) + 1), dict(batch=1 << 16, dim=1 << 16), dict(batch=1 << 20, seqlen=1 << 20, dim=1),
               dict(seqlen=1 << 31, dim=1), dict(batch=1 << 23, seqlen=1, dim=1), dict(batch=1, seqlen=1 << 20, dim=1 << 21), dict(batch=1 << 62)):
        assert fwd(lib, gd(**kw)) == UNSUPPORTED, kw
        assert lib.mamba_gated_scan_workspace_size(ctypes.byref(gd(**kw))) == 0
    assert upd(lib, gd(seqlen=2)) == INVALID and "seqlen" in err(lib)


@pytest.mark.parametrize("call,names", [(fwd, ["x", "r", "g", "A", "out"]),
                                        (bwd, ["x", "r", "g", "A", "ck", "dout", "dx", "dr", "dg", "dA"])])
def test_gated_required(lib, call, names):
    for n in names:
        assert call(lib, gd(), **{n: None}) == INVALID, n
        assert "NULL" in err(lib)
    for n in ("state", "x", "r", "g", "A", "out"):
        assert upd(lib, gd(seqlen=1), **{n: None}) == INVALID


def test_gated_overlaps_alignment_strides(lib):
    for o in ("out", "last", "ck"):
        for i in ("x", "r", "g", "A", "h0", "reset"):
            assert fwd(lib, gd(), **{o: FWD.index(i) + 1}) == INVALID
            assert "overlaps" in err(lib)
    assert fwd(lib, gd(), last=FWD.index("out") + 1) == INVALID
    for o in ("dx", "dr", "dg", "dA", "dh0"):
        for i in ("x", "r", "g", "A", "reset", "ck", "dout", "dlast"):
            assert bwd(lib, gd(), **{o: BWD.index(i) + 1}) == INVALID
    assert bwd(lib, gd(), dr=BWD.index("dg") + 1) == INVALID
    for i in ("x", "r", "g", "A", "state"):
        assert upd(lib, gd(seqlen=1), out=UPD.index(i) + 1) == INVALID
    for n in ("x", "r", "g", "out"):
        assert fwd(lib, gd(), **{n: P(FWD.index(n) + 1) + 1}) == INVALID and "aligned" in err(lib)
    for n in ("A", "h0", "last", "ck"):
        assert fwd(lib, gd(), **{n: P(FWD.index(n) + 1) + 2}) == INVALID and "aligned" in err(lib)
    assert fwd(lib, gd(), bk.GatedStrides(15)) == INVALID and "stride" in err(lib)
    assert fwd(lib, gd(), bk.GatedStrides(-1)) == INVALID
    assert fwd(lib, gd(), bk.GatedStrides(0, 0, 0, (1 << 26) + 1)) == UNSUPPORTED
    # halves of one buffer may interleave, but not share a column
    half = P(20)
    assert bwd(lib, gd(), bk.GatedStrides(dr=32, dg=31), dr=half, dg=half + 32) == INVALID
    assert bwd(lib, gd(), bk.GatedStrides(dr=32, dg=32), dr=half, dg=half + 30) == INVALID
    assert bwd(lib, gd(), bk.GatedStrides(dr=31, dg=31), dr=half, dg=half + 32) == INVALID


def test_gated_workspace(lib):
    d = gd(batch=1, seqlen=5000, dim=256)
    for size, call in ((lib.mamba_gated_scan_workspace_size, fwd), (lib.mamba_gated_scan_bwd_workspace_size, bwd)):
        need = size(ctypes.byref(d))
        assert need % 256 == 0
        if need:
            far = dict(x=100, r=110, g=120, A=130, reset=131, ck=140)
            far.update(dict(h0=132, out=150, last=133) if call is fwd else
                       dict(dout=150, dlast=132, dx=160, dr=170, dg=180, dA=133, dh0=134))
            assert call(lib, d, ws=None, ws_bytes=0, **far) == INVALID and "workspace" in err(lib)
            assert call(lib, d, ws=200, ws_bytes=need - 1, **far) == INVALID and "workspace" in err(lib)
            assert call(lib, d, ws=P(200) + 8, ws_bytes=need, **far) == INVALID and "aligned" in err(lib)
            assert call(lib, d, ws=100, ws_bytes=need, **far) == INVALID and "overlaps" in err(lib)


def test_gated_nothing_to_do(lib):
    assert fwd(lib, gd(batch=0), x=None, out=None) == 0
    assert fwd(lib, gd(dim=0), x=None, out=None) == 0
    assert fwd(lib, gd(seqlen=0), x=None, out=None, last=None) == 0
    assert bwd(lib, gd(dim=0), x=None, dA=None) == 0
    assert upd(lib, gd(batch=0, seqlen=1), state=None) == 0


def nd(rows=4, dim=32, group=0, io=1, res=1, eps=1e-6, flags=0):
    return bk.NormDesc(rows, dim, group, io, res, eps, flags)


def norm(lib, d, s=None, quant=False, **kw):
    order = ["x", "residual", "weight", "out"] + (["scale"] if quant else []) + ["sum"]
    f = lib.mamba_rmsnorm_quant_fwd if quant else lib.mamba_rmsnorm_fwd
    return f(None if d is None else ctypes.byref(d), None if s is None else ctypes.byref(s), *ptrs(order, kw, 1), None)


NB = ["sum", "weight", "dout", "dsum", "dresidual", "dx", "dweight"]


def norm_bwd(lib, d, s=None, ws=50, ws_bytes=1 << 40, **kw):
    kw.setdefault("dx", None)
    return lib.mamba_rmsnorm_bwd(ctypes.byref(d), None if s is None else ctypes.byref(s), *ptrs(NB, kw, 1), P(ws),
                                 ws_bytes, None)


def test_norm_refusals(lib):
    assert norm(lib, None) == INVALID
    for kw in (dict(rows=-1), dict(dim=-1), dict(io=5), dict(res=5), dict(flags=2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(group=-1)):
        assert norm(lib, nd(**kw)) == INVALID, kw
        assert norm(lib, nd(**kw), quant=True) == INVALID, kw
        assert norm_bwd(lib, nd(**kw)) == INVALID, kw
    assert norm(lib, nd(group=128)) == INVALID
    assert norm(lib, nd(group=64), quant=True) == UNSUPPORTED
    assert norm(lib, nd(io=0, res=1)) == UNSUPPORTED
    assert norm(lib, nd(dim=65537)) == UNSUPPORTED
    assert norm(lib, nd(rows=1 << 31)) == UNSUPPORTED
    assert norm(lib, nd(dim=0), quant=True) == UNSUPPORTED
    for n in ("x", "weight", "out", "sum"):
        assert norm(lib, nd(), **{n: None}) == INVALID
        assert norm(lib, nd(), quant=True, **{n: None}) == INVALID
    assert norm(lib, nd(), quant=True, scale=None) == INVALID
    assert norm(lib, nd(), residual=None) == INVALID               # sum without a residual
    assert norm(lib, nd(res=0), residual=None, sum=None) == INVALID
    for o in ("out", "sum"):
        assert norm(lib, nd(), **{o: 1}) == INVALID and "overlaps" in err(lib)
    assert norm(lib, nd(), bk.NormStrides(sum=40), sum=2) == INVALID   # in place needs one stride
    assert norm(lib, nd(res=0), sum=P(2) + 4) == INVALID
    assert norm(lib, nd(), bk.NormStrides(x=31)) == INVALID
    assert norm(lib, nd(), bk.NormStrides(out=(1 << 26) + 1)) == UNSUPPORTED
    assert norm(lib, nd(), x=P(1) + 1) == INVALID and "aligned" in err(lib)
    for n in ("sum", "weight", "dout", "dresidual", "dweight"):
        assert norm_bwd(lib, nd(), **{n: None}) == INVALID
    assert norm_bwd(lib, nd(), dx=6) == INVALID                        # dx is dresidual
    assert norm_bwd(lib, nd(), dresidual=3) == INVALID
    assert norm_bwd(lib, nd(), dweight=2) == INVALID
    assert norm_bwd(lib, nd(), ws=None, ws_bytes=0) == INVALID
    assert norm_bwd(lib, nd(), ws=1) == INVALID
    assert norm(lib, nd(rows=0), x=None) == 0 and norm_bwd(lib, nd(dim=0), dweight=None) == 0


CB = ["xin", "weight", "bias", "state_in", "dout", "dstate_out", "dxin", "dweight", "dbias", "dstate_in"]


def conv(lib, d, ws=50, ws_bytes=1 << 40, **kw):
    return lib.mamba_conv1d_bwd(None if d is None else ctypes.byref(d), *ptrs(CB, kw, 1), P(ws), ws_bytes, None)


def test_conv_bwd_refusals(lib):
    def cd(batch=2, seqlen=8, dim=16, width=4, io=1, flags=0):
        return bd.ConvDesc(batch, seqlen, dim, width, io, flags)

    assert conv(lib, None) == INVALID
    for kw in (dict(batch=-1), dict(seqlen=-1), dict(dim=-1), dict(io=7), dict(width=0), dict(flags=1)):
        assert conv(lib, cd(**kw)) == INVALID, kw
        assert lib.mamba_conv1d_bwd_workspace_size(ctypes.byref(cd(**kw))) == 0
    for kw in (dict(width=5), dict(batch=65536), dict(seqlen=1 << 41)):
        assert conv(lib, cd(**kw)) == UNSUPPORTED, kw
    for n in ("xin", "weight", "dout", "dxin", "dweight"):
        assert conv(lib, cd(), **{n: None}) == INVALID and "NULL" in err(lib)
    for o in ("dxin", "dweight", "dbias", "dstate_in"):
        for i in ("xin", "weight", "bias", "state_in", "dout", "dstate_out"):
            assert conv(lib, cd(), **{o: CB.index(i) + 1}) == INVALID, (o, i)
    assert conv(lib, cd(), dxin=P(7) + 1) == INVALID and conv(lib, cd(), dbias=P(9) + 2) == INVALID
    assert conv(lib, cd(), ws=None, ws_bytes=0) == INVALID
    assert conv(lib, cd(), ws=P(50) + 16) == INVALID
    assert conv(lib, cd(dim=0), dweight=None) == 0


def test_python_refusals_without_a_gpu():
    """Tensors that are not on a GPU, of other types or shapes, are refused by name."""
    t = torch.zeros((2, 4, 8))
    with pytest.raises(ValueError, match="runs on a GPU tensor"):
        bk.gated_scan_fwd(t, t, t, torch.zeros(8))
    with pytest.raises(ValueError, match="x must be"):
        bk.gated_scan_fwd(t[0], t, t, torch.zeros(8))
    with pytest.raises(ValueError, match="runs on a GPU tensor"):
        bk.gated_update(t[0], t[0], t[0], t[0], torch.zeros(8))
    with pytest.raises(ValueError, match="runs on a GPU tensor"):
        bk.rmsnorm_fwd(t[0], torch.ones(8))
    with pytest.raises(ValueError, match="dout must be"):
        bk.rmsnorm_bwd(t[0], torch.ones(8), t)
    with pytest.raises(ValueError, match="runs on a GPU tensor"):
        bk.conv1d_bwd(t, torch.zeros((8, 4)), t)
    assert bk._rows(t, "x", t.shape, torch.float32, t.device, 1) == 0
    assert bk._rows(torch.zeros((2, 4, 20))[..., 3:11], "x", t.shape, torch.float32, t.device, 1) == 20
    with pytest.raises(TypeError, match="x has dtype"):
        bk._rows(t, "x", t.shape, torch.bfloat16, t.device, 1)
    with pytest.raises(ValueError, match="x has shape"):
        bk._rows(t, "x", torch.Size((2, 4, 9)), torch.float32, t.device, 1)
    with pytest.raises(ValueError, match="contiguous"):
        bk._rows(torch.zeros((2, 4, 16))[..., ::2], "x", t.shape, torch.float32, t.device, 1)
    with pytest.raises(ValueError, match="rows overlap"):
        bk._rows(torch.zeros(64).as_strided((2, 4, 8), (16, 4, 1)), "x", t.shape, torch.float32, t.device, 1)
    with pytest.raises(ValueError, match="zero-stride"):
        bk._rows(torch.zeros((2, 1, 8)).expand(2, 4, 8), "x", t.shape, torch.float32, t.device, 1)
    with pytest.raises(TypeError, match="reset has dtype"):
        bk._reset(torch.zeros((2, 4)), (2, 4), t.device)


def test_abi_layer_under_sanitizers(tmp_path):
    if shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include/hip"):
        pytest.skip("g++ or the HIP headers not found")
    csrc, san = os.path.join(ROOT, "selective_state_space_56_amd", "csrc"), os.path.join(ROOT, "tests", "sanitize")
    exe = str(tmp_path / "block_driver")
    cmd = ["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I",
           os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "api.cpp"), os.path.join(csrc, "api_block.cpp"),
           os.path.join(san, "api_stubs.cpp"), os.path.join(san, "block_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=ENV)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "every case ran clean" in out and "runtime error" not in out, out
