"""The operators of include/pkv_ops.h without a GPU: rotation frequencies against exact
arithmetic, and every argument that the host refuses (nothing is enqueued)."""
import ctypes
from decimal import Decimal, getcontext

import pytest

import paged_kv_cache_101_gb300 as pkv
from paged_kv_cache_101_gb300 import _build

torch = pytest.importorskip("torch")

OK, NULL, SHAPE, DTYPE, ALIGN, RANGE, WORKSPACE, CUDA, UNSUP = range(9)
A = 1 << 20          # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.lib()


# ---------------------------------------------------------------- frequencies
def exact_turns(r, base):
    getcontext().prec = 60
    two_pi = Decimal("6.283185307179586476925286766559005768394338798750211641949889")
    return [(Decimal(base).ln() * Decimal(-2 * i) / Decimal(r)).exp() / two_pi
            for i in range(r // 2)]


@pytest.mark.parametrize("r,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (20, 1e6)])
def test_turns(lib, r, base):
    got = pkv.rotary_turns(r, base)
    assert got.dtype == torch.int64 and got.shape == (r // 2,)
    for g, f in zip(got.tolist(), exact_turns(r, base)):
        # doubles: the exponent's rounding (2^-53 of at most 1) moves base^x by
        # ln(base) 2^-53 <= 14 * 2^-53 of itself, pow, the division and 2 pi by 4 * 2^-53
        # more; the fixed point by one step
        assert (abs(Decimal(g % 2 ** 64) / Decimal(2 ** 64) - f)
                <= f * Decimal(2) ** -48 + Decimal(2) ** -64)


def test_scaled_turns(lib):
    plain = [float(t) for t in pkv.rotary_turns(128).tolist()]
    linear = pkv.rotary_turns(128, kind="linear", factor=4.0).tolist()
    assert all(abs(a / 4 - b) <= a * 2.0 ** -48 + 2 for a, b in zip(plain, linear))
    base = pkv.rotary_turns(128, kind="base", factor=4.0).tolist()
    assert base[0] == int(plain[0]) and abs(base[-1] / plain[-1] - 0.25) < 1e-9
    ramp = pkv.rotary_turns(128, kind="ramp", factor=8.0, original_length=4096, low=1.0,
                            high=32.0).tolist()
    for a, b in zip(plain, ramp):
        n = 4096 * a / 2.0 ** 64                          # turns within the original length
        keep = min(1.0, max(0.0, (n - 1) / 31))
        want = a * (keep + (1 - keep) / 8)
        assert abs(b - want) <= want * 2.0 ** -45 + 2     # keep is a difference


def test_turns_refusals(lib):
    buf = (ctypes.c_uint64 * 64)()
    p = ctypes.addressof(buf)
    call = lib.pkv_rotary_turns
    nan, inf = float("nan"), float("inf")
    assert call(128, 1e4, 0, 1, 1, 1, 2, None) == NULL
    for r in (0, -2, 7):
        assert call(r, 1e4, 0, 1, 1, 1, 2, p) == SHAPE
    assert call(2, 1e4, 2, 2, 1, 1, 2, p) == SHAPE
    assert call(8, 1e4, 4, 1, 1, 1, 2, p) == UNSUP and call(8, 1e4, -1, 1, 1, 1, 2, p) == UNSUP
    for base in (0.0, -1.0, nan, inf):
        assert call(8, base, 0, 1, 1, 1, 2, p) == RANGE
    for kind in (1, 2, 3):
        for f in (0.0, -2.0, nan, inf):
            assert call(8, 1e4, kind, f, 100, 1, 2, p) == RANGE
    for L, lo, hi in ((0, 1, 2), (nan, 1, 2), (100, 2, 2), (100, nan, 2), (100, 1, inf)):
        assert call(8, 1e4, 3, 2, L, lo, hi, p) == RANGE
    with pytest.raises(ValueError):
        pkv.rotary_turns(8, kind="other")
    with pytest.raises(pkv.PkvError):
        pkv.rotary_turns(7)


# ---------------------------------------------------------------- rotation + append
ROPE = dict(q=A, qs=512, k=A, ks=128, v=A, vs=128, pos=A, turns=A, slots=A, n=4, qo=2 * A, kc=A,
            vc=A, nb=8, Hq=8, Hkv=2, D=64, r=64, inter=0, scale=1.0)


def rope(lib, fp8=False, **over):
    a = dict(ROPE, kscale=A, vscale=A)
    a.update(over)
    head = [a[x] for x in ("q", "qs", "k", "ks", "v", "vs", "pos", "turns", "slots", "n", "qo",
                           "kc", "vc")]
    tail = [a[x] for x in ("nb", "Hq", "Hkv", "D", "r", "inter", "scale")] + [None]
    if fp8:
        return lib.pkv_rope_kv_append_fp8_block(*head, a["kscale"], a["vscale"], *tail)
    return lib.pkv_rope_kv_append(*head, *tail)


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_refusals(lib, fp8):
    go = lambda **o: rope(lib, fp8, **o)  # noqa: E731
    assert go(n=0) == OK and go(n=0, k=None, pos=None) == OK
    for o in (dict(n=-1), dict(nb=0), dict(Hq=-1), dict(Hkv=0), dict(D=0), dict(r=0), dict(r=66),
              dict(r=31), dict(ks=120), dict(vs=127), dict(qs=511),
              dict(qo=A, qs=520)):
        assert go(**o) == SHAPE, o
    for o in ("k", "v", "pos", "turns", "slots", "kc", "vc", "q", "qo"):
        assert go(**{o: None}) == NULL, o
    assert go(Hq=0) == NULL                       # q given, but no heads
    if fp8:
        assert go(kscale=None) == NULL and go(vscale=None) == NULL
        assert go(D=264, r=64, qs=8 * 264, ks=528, vs=528) == RANGE
    assert go(D=68, r=64) == UNSUP
    assert go(qo=A, r=20) == UNSUP and go(qo=A, r=20, inter=1) == UNSUP
    for o in (dict(D=1032, qs=8 * 1032, ks=2064, vs=2064), dict(Hkv=1025, ks=1 << 20, vs=1 << 20),
              dict(n=(1 << 30) + 1), dict(nb=(1 << 40) + 1), dict(scale=float("nan")),
              dict(scale=float("inf"))):
        assert go(**o) == RANGE, o
    for o in (dict(q=A + 8), dict(k=A + 2), dict(v=A + 8), dict(qo=2 * A + 8), dict(kc=A + 4),
              dict(vc=A + 4), dict(pos=A + 4), dict(turns=A + 4), dict(slots=A + 4), dict(qs=516),
              dict(ks=132), dict(vs=132)):
        assert go(**o) == ALIGN, o


# ---------------------------------------------------------------- attention
ATT = dict(q=A, kc=A, vc=A, nb=8, ks=None, vs=None, bt=A, mb=4, cl=A, S=2, nq=1, Hq=8, Hkv=2,
           D=128, scale=0.1, cap=0.0, sl=None, win=0, out=A, odt=0, ws=A, wsb=1 << 30)


def att(lib, **over):
    a = dict(ATT)
    a.update(over)
    return lib.pkv_paged_decode_attention_scored(*[a[x] for x in (
        "q", "kc", "vc", "nb", "ks", "vs", "bt", "mb", "cl", "S", "nq", "Hq", "Hkv", "D", "scale",
        "cap", "sl", "win", "out", "odt", "ws", "wsb")], None)


def test_attention_refusals(lib):
    assert att(lib, S=0) == OK
    for o in (dict(S=-1), dict(nq=0), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(nb=0), dict(mb=0)):
        assert att(lib, **o) == SHAPE, o
    for o in (dict(D=96), dict(nq=5), dict(Hq=132, Hkv=2), dict(D=64, ks=A, vs=A)):
        assert att(lib, **o) == UNSUP, o
    assert att(lib, odt=2) == DTYPE
    for o in (dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(win=-1),
              dict(mb=(1 << 26) + 1), dict(nb=1 << 31), dict(S=(1 << 24) + 1)):
        assert att(lib, **o) == RANGE, o
    for o in (dict(q=None), dict(kc=None), dict(vc=None), dict(bt=None), dict(cl=None),
              dict(out=None), dict(ks=A), dict(vs=A)):
        assert att(lib, **o) == NULL, o
    assert att(lib, ws=None) == WORKSPACE
    for o in (dict(q=A + 8), dict(kc=A + 8), dict(vc=A + 8), dict(out=A + 8), dict(bt=A + 2),
              dict(cl=A + 2), dict(sl=A + 2), dict(ws=A + 128)):
        assert att(lib, **o) == ALIGN, o


def test_caps_that_leave_float_are_refused(lib):
    assert att(lib, cap=1e-40) == RANGE and att(lib, cap=1e-10, scale=1e35) == RANGE
    assert att(lib, cap=1e-40, scale=1e-5, S=0) == OK


def test_fp8_block_refusals(lib):
    def go(**over):
        a = dict(ATT, ks=A, vs=A)
        a.update(over)
        return lib.pkv_paged_decode_attention_fp8_block(*[a[x] for x in (
            "q", "kc", "vc", "nb", "ks", "vs", "bt", "mb", "cl", "S", "nq", "Hq", "Hkv", "D",
            "scale", "out", "odt", "ws", "wsb")], None)
    assert go(S=0) == OK
    assert go(ks=None) == NULL and go(vs=None) == NULL and go(ks=None, vs=None) == NULL
    assert go(D=64) == UNSUP and go(nq=5) == UNSUP and go(S=-1) == SHAPE
    assert go(ws=None) == WORKSPACE and go(q=A + 4) == ALIGN


def test_workspace_size_of_unsupported_geometries(lib):
    for g in ((-1, 1, 8, 2, 128), (2, 0, 8, 2, 128), (2, 5, 8, 2, 128), (2, 1, 7, 2, 128),
              (2, 1, 8, 2, 96), (2, 1, 130, 2, 128)):
        assert pkv.workspace_size_scored(*g) == 0
    assert pkv.workspace_size_scored(0, 1, 8, 2, 128) == 256


# ---------------------------------------------------------------- the Python face
def test_python_refuses_cpu_tensors_and_wrong_types():
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        pkv.rope_kv_append(b(3, 4, 64), b(3, 2, 64), b(3, 2, 64), i, i, i, b(2, 16, 2, 64),
                           b(2, 16, 2, 64), b(3, 4, 64))
    with pytest.raises(TypeError):
        pkv.rope_kv_append(None, [1], b(3, 2, 64), i, i, i, b(2, 16, 2, 64), b(2, 16, 2, 64), None)
    t = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.paged_decode_attention_scored(b(1, 4, 64), b(2, 16, 2, 64), b(2, 16, 2, 64), t, t[0], 1,
                                          1.0, b(1, 4, 64))
    with pytest.raises(ValueError):
        pkv.paged_decode_attention_fp8_block(b(1, 4, 64), b(2, 16, 2, 64), b(2, 16, 2, 64), None,
                                             None, t, t[0], 1, 1.0, b(1, 4, 64))
