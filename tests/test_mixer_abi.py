"""CPU tests of the mixer operators' C ABI (include/mixer/): the library exports
what the headers declare and rejects bad arguments before any HIP call (pointers
here are fake and never read), the binding refuses by name, and the ABI layer runs
clean under AddressSanitizer / UndefinedBehaviorSanitizer with its launches
replaced."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from selective_state_space_56_amd import binding as bd
from selective_state_space_56_amd import mixer as mx
from test_sanitizers import ENV, SAN

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = os.path.join(ROOT, "include", "mixer")
INVALID, UNSUPPORTED = 1, 2
FAKE = 0x7F0000000000
NAMES = {"mamba_linattn_workspace_size", "mamba_linattn_bwd_workspace_size", "mamba_linattn_fwd", "mamba_linattn_bwd",
         "mamba_linattn_update", "mamba_qknorm_fwd", "mamba_qknorm_bwd_workspace_size", "mamba_qknorm_bwd"}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from selective_state_space_56_amd.build import build
        build()
    return mx._library()


def err(lib):
    return lib.mamba_last_error().decode()


def P(k):
    """A fake device address; an int is the k-th region of 16 MiB."""
    return None if k is None else FAKE + 0x1000000 * k if isinstance(k, int) and k < 1000 else k


def ptrs(order, given):
    v = dict(zip(order, range(1, 1 + len(order))))
    v.update(given)
    return [P(v[n]) for n in order]


def ref(s):
    return None if s is None else ctypes.byref(s)


def test_exports_every_declared_symbol(lib):
    names = set()
    for h in os.listdir(HEADERS):
        src = re.sub(r"/\*.*?\*/", "", open(os.path.join(HEADERS, h)).read(), flags=re.S)
        names |= set(re.findall(r"\b(mamba_[a-z0-9_]+)\s*\(", src))
    assert names == NAMES
    for n in names:
        assert hasattr(lib, n)


@pytest.mark.parametrize("header", ["mamba_linattn.h", "mamba_qknorm.h"])
def test_headers_are_c(header, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not found")
    src = tmp_path / "h.c"
    src.write_text(f'#include "mixer/{header}"\nint main(void) {{ return 0; }}\n')
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                        "-fsyntax-only", str(src)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr


def ld(batch=2, seqlen=8, heads=4, groups=2, K=16, V=24, io=1, flags=0, scale=1.0):
    return mx.LinattnDesc(batch, seqlen, heads, groups, K, V, io, flags, scale)


FWD = ["q", "k", "v", "g", "h0", "offsets", "out", "last"]
BWD = ["q", "k", "v", "g", "h0", "offsets", "dout", "dlast", "dq", "dk", "dv", "dg", "dh0"]
UPD = ["state", "q", "k", "v", "g", "out"]
TURN = ["q", "k", "positions", "freqs", "wq", "wk", "qo", "ko"]
BACK = ["q", "k", "positions", "freqs", "wq", "wk", "dqo", "dko", "dq", "dk", "dwq", "dwk"]


def fwd(lib, d, s=None, ws=50, ws_bytes=1 << 40, **kw):
    if d is not None and not d.flags & mx.PACKED:
        kw.setdefault("offsets", None)
    return lib.mamba_linattn_fwd(ref(d), ref(s), *ptrs(FWD, kw), P(ws), ws_bytes, None)


def bwd(lib, d, s=None, ws=50, ws_bytes=1 << 40, **kw):
    if d is not None and not d.flags & mx.PACKED:
        kw.setdefault("offsets", None)
    return lib.mamba_linattn_bwd(ref(d), ref(s), *ptrs(BWD, kw), P(ws), ws_bytes, None)


def upd(lib, d, s=None, **kw):
    return lib.mamba_linattn_update(ref(d), ref(s), *ptrs(UPD, kw), None)


def turn(lib, d, s=None, **kw):
    return lib.mamba_qknorm_fwd(ref(d), ref(s), *ptrs(TURN, kw), None)


def back(lib, d, s=None, ws=50, ws_bytes=1 << 40, **kw):
    return lib.mamba_qknorm_bwd(ref(d), ref(s), *ptrs(BACK, kw), P(ws), ws_bytes, None)


def test_descriptors(lib):
    for call in (fwd, bwd, upd):
        assert call(lib, None) == INVALID and "desc is NULL" in err(lib)
    for kw in (dict(batch=-1), dict(seqlen=-1), dict(heads=-2), dict(groups=0), dict(groups=-1), dict(groups=3), dict(groups=8),
               dict(K=0), dict(V=0), dict(K=-8), dict(io=2), dict(flags=8), dict(flags=mx.ZERO_REST),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        assert fwd(lib, ld(**kw)) == INVALID and bwd(lib, ld(**kw)) == INVALID, kw
        assert lib.mamba_linattn_workspace_size(ref(ld(**kw))) == 0
        assert lib.mamba_linattn_bwd_workspace_size(ref(ld(**kw))) == 0
        assert upd(lib, ld(**{"seqlen": 1, **kw})) == INVALID
    for kw in (dict(K=12), dict(V=20), dict(K=264), dict(V=512), dict(batch=1 << 20, seqlen=1, heads=4),
               dict(batch=1 << 16, seqlen=1 << 16), dict(seqlen=1 << 31, heads=2), dict(batch=1 << 62), dict(seqlen=1 << 62)):
        assert fwd(lib, ld(**kw)) == UNSUPPORTED and bwd(lib, ld(**kw)) == UNSUPPORTED, kw
        assert lib.mamba_linattn_workspace_size(ref(ld(**kw))) == 0
    assert upd(lib, ld(seqlen=2)) == INVALID and "seqlen" in err(lib)
    assert upd(lib, ld(seqlen=0)) == INVALID
    assert upd(lib, ld(seqlen=1, flags=mx.PACKED)) == INVALID and "PACKED" in err(lib)


def test_required(lib):
    for call, names in ((fwd, ["q", "k", "v", "g", "out"]), (bwd, ["q", "k", "v", "g", "dout", "dq", "dk", "dv"])):
        for n in names:
            assert call(lib, ld(), **{n: None}) == INVALID and "NULL" in err(lib), n
        assert call(lib, ld(), offsets=7) == INVALID and "offsets" in err(lib)
        assert call(lib, ld(flags=mx.PACKED), offsets=None) == INVALID and "offsets" in err(lib)
    for n in UPD:
        assert upd(lib, ld(seqlen=1), **{n: None}) == INVALID and "NULL" in err(lib), n


def test_overlaps_alignment_strides(lib):
    d = ld(flags=mx.PACKED, seqlen=16)
    for o in ("out", "last"):
        for i in FWD[:6]:
            assert fwd(lib, d, **{o: FWD.index(i) + 1}) == INVALID and "overlaps" in err(lib), (o, i)
    assert fwd(lib, d, last=FWD.index("out") + 1) == INVALID
    for o in BWD[8:]:
        for i in BWD[:8]:
            assert bwd(lib, d, **{o: BWD.index(i) + 1}) == INVALID and "overlaps" in err(lib), (o, i)
        for i in BWD[8:]:
            if i != o:
                assert bwd(lib, d, **{o: BWD.index(i) + 1}) == INVALID, (o, i)
    for i in UPD[:5]:
        assert upd(lib, ld(seqlen=1), out=UPD.index(i) + 1) == INVALID
    for i in UPD[1:5]:
        assert upd(lib, ld(seqlen=1), state=UPD.index(i) + 1) == INVALID
    for n in ("q", "k", "v", "out"):
        assert fwd(lib, d, **{n: P(FWD.index(n) + 1) + 1}) == INVALID and "aligned" in err(lib)
    for n in ("g", "h0", "last"):
        assert fwd(lib, d, **{n: P(FWD.index(n) + 1) + 2}) == INVALID and "aligned" in err(lib)
    assert fwd(lib, d, offsets=P(6) + 4) == INVALID and "aligned" in err(lib)
    for n in ("dout", "dq", "dk", "dv"):
        assert bwd(lib, d, **{n: P(BWD.index(n) + 1) + 1}) == INVALID and "aligned" in err(lib)
    for n in ("dlast", "dg", "dh0"):
        assert bwd(lib, d, **{n: P(BWD.index(n) + 1) + 2}) == INVALID and "aligned" in err(lib)
    assert fwd(lib, d, mx.LinattnStrides(q=31)) == INVALID and "stride" in err(lib)
    assert fwd(lib, d, mx.LinattnStrides(v=95)) == INVALID
    assert fwd(lib, d, mx.LinattnStrides(out=-1)) == INVALID
    assert fwd(lib, d, mx.LinattnStrides(k=(1 << 23) + 1)) == UNSUPPORTED
    assert bwd(lib, d, mx.LinattnStrides(dv=(1 << 23) + 1)) == UNSUPPORTED
    assert fwd(lib, ld(batch=1, seqlen=1, heads=1 << 16, groups=1, V=256)) == UNSUPPORTED   # rows of 2^24
    # columns of one buffer may interleave, but not share one
    at = P(60)
    wide = mx.LinattnStrides(dq=160, dk=160, dv=160)
    assert bwd(lib, d, wide, ws=None, ws_bytes=0, dq=at, dk=at + 64, dv=at + 128) == INVALID and "workspace" in err(lib)
    assert bwd(lib, d, wide, dq=at, dk=at + 62, dv=at + 128) == INVALID and "overlaps" in err(lib)
    assert bwd(lib, d, mx.LinattnStrides(dq=160, dk=159, dv=160), dq=at, dk=at + 64, dv=at + 128) == INVALID


def test_workspace(lib):
    d = ld(batch=1, seqlen=8192, heads=2, groups=1, K=128, V=128)
    for size, call, order in ((lib.mamba_linattn_workspace_size, fwd, FWD), (lib.mamba_linattn_bwd_workspace_size, bwd, BWD)):
        need = size(ref(d))
        assert need > 0 and need % 256 == 0
        far = {n: 10 * (i + 1) for i, n in enumerate(order) if n != "offsets"}
        assert call(lib, d, ws=None, ws_bytes=0, **far) == INVALID and "workspace" in err(lib)
        assert call(lib, d, ws=200, ws_bytes=need - 1, **far) == INVALID and "workspace" in err(lib)
        assert call(lib, d, ws=P(200) + 8, ws_bytes=need, **far) == INVALID and "aligned" in err(lib)
        assert call(lib, d, ws=10, ws_bytes=need, **far) == INVALID and "overlaps" in err(lib)


def test_workspace_of_many_short_sequences(lib):
    # one state for each, and little beside it: no states between stretches of sequences this short
    d = ld(batch=4096, seqlen=64, heads=4, groups=4, K=128, V=128)
    states = 4096 * 4 * 128 * 128 * 4
    assert states <= lib.mamba_linattn_bwd_workspace_size(ref(d)) < 1.2 * states
    assert lib.mamba_linattn_workspace_size(ref(d)) == 0


def test_nothing_to_do(lib):
    for call in (fwd, bwd):
        assert call(lib, ld(batch=0), q=None) == 0
        assert call(lib, ld(heads=0), q=None) == 0
    assert fwd(lib, ld(seqlen=0), q=None, out=None, last=None) == 0
    assert bwd(lib, ld(seqlen=0), q=None, dq=None, dh0=None) == 0
    assert upd(lib, ld(batch=0, seqlen=1), state=None) == 0
    assert turn(lib, qd(tokens=0), q=None, qo=None) == 0
    assert turn(lib, qd(hq=0, hk=0), q=None, qo=None) == 0
    assert back(lib, qd(tokens=0), q=None, dq=None, dwq=None, dwk=None) == 0


def qd(tokens=8, hq=4, hk=2, dim=32, rotary=16, sections=(8, 0, 0, 0), axes=1, io=1, eps=1e-6, flags=0):
    return mx.QkNormDesc(tokens, hq, hk, dim, rotary, mx._Sections(*sections), axes, io, eps, flags)


def test_norm_and_rotation(lib):
    assert turn(lib, None) == INVALID and back(lib, None) == INVALID
    for kw in (dict(tokens=-1), dict(hq=-1), dict(hk=-1), dict(dim=0), dict(dim=-8), dict(rotary=-8), dict(rotary=40),
               dict(sections=(7, 0, 0, 0)), dict(sections=(4, 4, 0, 0)), dict(sections=(9, -1, 0, 0), axes=2),
               dict(sections=(4, 2, 0, 0), axes=2), dict(axes=0), dict(axes=5), dict(io=2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(flags=2)):
        assert turn(lib, qd(**kw)) == INVALID and back(lib, qd(**kw)) == INVALID, kw
        assert lib.mamba_qknorm_bwd_workspace_size(ref(qd(**kw))) == 0
    for kw in (dict(dim=20), dict(dim=264), dict(rotary=12, sections=(6, 0, 0, 0)), dict(tokens=1 << 31),
               dict(hq=(1 << 20) + 1), dict(tokens=1 << 30, hq=2, hk=1)):
        assert turn(lib, qd(**kw)) == UNSUPPORTED and back(lib, qd(**kw)) == UNSUPPORTED, kw
    for n in ("q", "k", "positions", "freqs", "qo", "ko"):
        assert turn(lib, qd(), **{n: None}) == INVALID and "NULL" in err(lib), n
    for n in ("q", "k", "positions", "freqs", "dqo", "dko", "dq", "dk"):
        assert back(lib, qd(), **{n: None}) == INVALID and "NULL" in err(lib), n
    for o in ("qo", "ko"):
        for i in TURN:
            if i not in (o, o[0]):
                assert turn(lib, qd(), **{o: TURN.index(i) + 1}) == INVALID and "overlaps" in err(lib), (o, i)
        assert turn(lib, qd(), mx.QkNormStrides(**{o: 200}), **{o: TURN.index(o[0]) + 1}) == INVALID  # in place: one stride
        assert turn(lib, qd(), **{o: P(TURN.index(o[0]) + 1) + 2}) == INVALID
    for o in ("dq", "dk", "dwq", "dwk"):
        for i in BACK:
            if i not in (o, o + "o"):
                assert back(lib, qd(), **{o: BACK.index(i) + 1}) == INVALID and "overlaps" in err(lib), (o, i)
    for n in ("q", "k", "qo", "ko"):
        assert turn(lib, qd(), **{n: P(TURN.index(n) + 1) + 1}) == INVALID and "aligned" in err(lib)
    for n in ("wq", "wk", "freqs"):
        assert turn(lib, qd(), **{n: P(TURN.index(n) + 1) + 2}) == INVALID and "aligned" in err(lib)
    assert turn(lib, qd(), positions=P(3) + 4) == INVALID and "aligned" in err(lib)
    assert turn(lib, qd(), mx.QkNormStrides(q=127)) == INVALID and "stride" in err(lib)
    assert turn(lib, qd(), mx.QkNormStrides(ko=-1)) == INVALID
    assert turn(lib, qd(), mx.QkNormStrides(qo=(1 << 26) + 1)) == UNSUPPORTED
    assert back(lib, qd(), ws=None, ws_bytes=0) == INVALID and "workspace" in err(lib)
    assert back(lib, qd(), ws=P(50) + 16) == INVALID and "aligned" in err(lib)
    assert back(lib, qd(), ws=1) == INVALID and "overlaps" in err(lib)


def test_python_refusals_without_a_gpu():
    """Tensors that are not on a GPU, of other types or shapes, are refused by name."""
    t, g = torch.zeros((2, 4, 2, 8)), torch.zeros((2, 4, 2))
    with pytest.raises(ValueError, match="runs on a GPU tensor"):
        mx.linear_attn_fwd(t, t, t, g)
    with pytest.raises(ValueError, match="v must be"):
        mx.linear_attn_fwd(t, t, t[0], g)
    with pytest.raises(ValueError, match="runs on a GPU tensor"):
        mx.linear_attn_bwd(t, t, t, g, t)
    with pytest.raises(ValueError, match="runs on a GPU tensor"):
        mx.linear_attn_update(t[0], t[0], t[0], t[0], g[0])
    with pytest.raises(ValueError, match="q must be"):
        mx.qk_norm_rope_fwd(t, None, torch.zeros(2), torch.zeros(4))
    with pytest.raises(ValueError, match="runs on a GPU tensor"):
        mx.qk_norm_rope_fwd(t[0], None, torch.zeros(4), torch.zeros(4))
    F, shape = torch.float32, t.shape
    assert mx._heads(None, "q", shape, F, t.device) == 0
    assert mx._heads(t, "q", shape, F, t.device) == 0
    assert mx._heads(torch.zeros((2, 4, 5, 8))[:, :, 1:3], "q", shape, F, t.device) == 40
    assert mx._heads(torch.zeros((2, 4, 16, 1))[..., 2:10, 0].unsqueeze(2), "q", (2, 4, 1, 8), F, t.device) == 16
    with pytest.raises(TypeError, match="q must be"):
        mx._heads(3, "q", shape, F, t.device)
    with pytest.raises(TypeError, match="q has dtype"):
        mx._heads(t, "q", shape, torch.bfloat16, t.device)
    with pytest.raises(ValueError, match="q has shape"):
        mx._heads(t, "q", torch.Size((2, 4, 2, 9)), F, t.device)
    with pytest.raises(ValueError, match="contiguous"):
        mx._heads(torch.zeros((2, 4, 2, 16))[..., ::2], "q", shape, F, t.device)
    with pytest.raises(ValueError, match="contiguous"):
        mx._heads(torch.zeros((2, 4, 2, 16))[..., :8], "q", shape, F, t.device)   # gaps between heads
    with pytest.raises(ValueError):
        mx._heads(torch.zeros((2, 2, 4, 8)).transpose(1, 2), "q", shape, F, t.device)   # heads before tokens
    with pytest.raises(ValueError, match="rows overlap"):
        mx._heads(torch.zeros(256).as_strided(shape, (32, 8, 8, 1)), "q", shape, F, t.device)
    with pytest.raises(ValueError, match="zero-stride"):
        mx._heads(torch.zeros((2, 1, 2, 8)).expand(2, 4, 2, 8), "q", shape, F, t.device)


def test_abi_layer_under_sanitizers(tmp_path):
    if shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include/hip"):
        pytest.skip("g++ or the HIP headers not found")
    csrc, san = os.path.join(ROOT, "selective_state_space_56_amd", "csrc"), os.path.join(ROOT, "tests", "sanitize")
    exe = str(tmp_path / "mixer_driver")
    cmd = ["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I",
           os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "api.cpp"), os.path.join(csrc, "api_mixer.cpp"),
           os.path.join(san, "api_stubs.cpp"), os.path.join(san, "mixer_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=ENV)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "every case ran clean" in out and "runtime error" not in out, out
