"""The 8-bit operators on the host: the oracle's E4M3 against torch's, the C
entry points' refusals and the binding's (no GPU: every call returns or raises
before anything is launched)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from routed_expert_ffn_fp32_b200 import build, moe

A = 0x100000  # aligned, never dereferenced
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.load_library()


def _p(addr=A):
    return ctypes.c_void_p(addr)


def test_e4m3_table_and_rounding_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(F.decode(codes), want)
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-12, 9, 4000),
                        F.decode(codes[:127]), (F.decode(codes[:126]) + F.decode(codes[1:127])) / 2])
    v = np.clip(v, -448, 448)
    got = F.encode(v)
    # every value here is a float32, so torch's rounding sees it exactly
    v32 = v.astype(np.float32)
    want = torch.from_numpy(v32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(F.encode(v32), want)
    assert (np.abs(F.decode(got) - v) <= np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10)).all()
    assert F.encode([1e9, -1e9]).tolist() == [0x7E, 0xFE] and F.encode([np.nan])[0] == 0x7F


def test_workspace_bytes(lib):
    s = moe.shape_of(5, 4096, 2048, 256, 8)
    n = lib.moe_expert_ffn_fp8_workspace_bytes(s, 0)
    assert n >= 40 * (2048 + 16 * 4) + moe.MOE_FP8_STATUS_BYTES
    assert lib.moe_expert_ffn_fp8_workspace_bytes(s, 1) >= n + 5 * 2048
    for bad in [(0, 256, 128, 8, 2), (1, 250, 128, 8, 2), (1, 256, 120, 8, 2), (1, 256, 128, 1025, 2),
                (1, 256, 128, 8, 17)]:
        assert lib.moe_expert_ffn_fp8_workspace_bytes(moe.shape_of(*bad), 0) == 0, bad


def test_norm_refusals(lib):
    def call(x=A, res=A, w=A, rows=4, H=256, dt=0, eps=1e-6, ro=A, y=A, q=A, s=A):
        return lib.moe_rmsnorm_quant_fp8(x, res, w, rows, H, dt, eps, ro, y, q, s, None)

    for kw in [dict(x=None), dict(w=None), dict(q=None), dict(s=None), dict(x=A + 2), dict(res=A + 4),
               dict(ro=A + 8), dict(y=A + 2), dict(dt=3), dict(dt=-1), dict(eps=-1.0), dict(eps=float("nan"))]:
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    for kw in [dict(H=0), dict(H=8), dict(H=24), dict(H=16400), dict(rows=-1), dict(rows=(1 << 21) + 1)]:
        assert call(**kw) == moe.MOE_ERR_UNSUPPORTED_SHAPE, kw
    assert call(rows=0) == moe.MOE_OK


def test_gemm_refusals(lib):
    def call(aq=A, as_=A, wq=A, ws_=A, rows=4, N=100, K=256, dt=0, out=A, ws=A, n=BIG):
        return lib.moe_gemm_fp8(aq, as_, wq, ws_, rows, N, K, dt, out, ws, n, None)

    for kw in [dict(aq=None), dict(as_=None), dict(wq=None), dict(ws_=None), dict(out=None), dict(ws=None),
               dict(aq=A + 8), dict(wq=A + 1), dict(ws_=A + 4), dict(out=A + 2), dict(dt=3)]:
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    for kw in [dict(rows=-1), dict(rows=(1 << 21) + 1), dict(N=0), dict(N=65537), dict(K=0), dict(K=24),
               dict(K=65552)]:
        assert call(**kw) == moe.MOE_ERR_UNSUPPORTED_SHAPE, kw
    assert call(n=64) == moe.MOE_ERR_WORKSPACE
    assert call(rows=0) == moe.MOE_OK


def test_grouped_refusals(lib):
    def gemm(aq=A, a_rows=8, off=A, ent=A, P=8, E=4, N=100, K=256, div=0, sc=1, dt=0, out=A, ws=A, n=BIG):
        return lib.moe_grouped_gemm_fp8(aq, A, a_rows, A, A, off, ent, P, E, N, K, div, sc, dt, out, ws, n, None)

    def swiglu(aq=A, a_rows=8, off=A, ent=A, P=8, E=4, I=128, H=256, div=2, q=A, ws=A, n=BIG):
        return lib.moe_grouped_swiglu_fp8(aq, A, a_rows, A, A, A, A, off, ent, P, E, I, H, div, q, A, ws, n, None)

    inv, shp = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE
    for kw in [dict(aq=None), dict(off=None), dict(ent=None), dict(out=None), dict(ws=A + 8), dict(div=-1),
               dict(dt=9), dict(a_rows=7), dict(ent=A + 4), dict(sc=0, div=2, ent=None)]:
        assert gemm(**kw) == inv, kw
    for kw in [dict(P=-1), dict(E=0), dict(E=1025), dict(N=0), dict(K=20), dict(a_rows=0)]:
        assert gemm(**kw) == shp, kw
    for kw in [dict(aq=A + 2), dict(off=None), dict(ent=None), dict(q=None), dict(div=-2), dict(div=0, a_rows=7)]:
        assert swiglu(**kw) == inv, kw
    for kw in [dict(I=120), dict(I=0), dict(H=100), dict(E=2000), dict(P=-1)]:
        assert swiglu(**kw) == shp, kw
    assert gemm(n=127) == moe.MOE_ERR_WORKSPACE and swiglu(n=127) == moe.MOE_ERR_WORKSPACE
    assert gemm(P=0) == moe.MOE_OK and swiglu(P=0, a_rows=0) == moe.MOE_OK


def test_expert_ffn_refusals(lib):
    s = moe.shape_of(4, 256, 128, 8, 2)
    ex = moe.moe_fp8_experts_t(A, A, A, A, A, A, 8)

    def call(e=ex, sh=None, xq=A, off=A, shape=s, out=A, n=BIG):
        return lib.moe_expert_ffn_fp8(ctypes.byref(e), None if sh is None else ctypes.byref(sh), xq, A, off, A,
                                      shape, out, A, n, None)

    assert call(e=moe.moe_fp8_experts_t(A, A, A, A, A, A, 7)) == moe.MOE_ERR_INVALID_ARG
    assert call(e=moe.moe_fp8_experts_t(A, A, A, None, A, A, 8)) == moe.MOE_ERR_INVALID_ARG
    assert call(sh=moe.moe_fp8_experts_t(A, A, A, A, A, A, 2)) == moe.MOE_ERR_INVALID_ARG
    assert call(xq=None) == moe.MOE_ERR_INVALID_ARG and call(off=A + 4) == moe.MOE_ERR_INVALID_ARG
    assert call(shape=moe.shape_of(4, 256, 120, 8, 2)) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(n=200) == moe.MOE_ERR_WORKSPACE


def _t(*shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_shapes_and_types():
    f32, ws = torch.float32, _t(256)
    aq, as_ = _t(4, 272), _t(4, 3, dtype=f32)
    wq, ws_ = _t(100, 272), _t(1, 3, dtype=f32)
    out = _t(4, 100, dtype=torch.bfloat16)
    bad = [dict(a_s=_t(4, 2, dtype=f32)), dict(a_q=_t(4, 272, dtype=torch.int8)), dict(w_q=_t(100, 256)),
           dict(w_s=_t(3, 1, dtype=f32)), dict(out=_t(4, 99, dtype=torch.bfloat16)), dict(out=_t(4, 100)),
           dict(a_s=_t(4, 3, dtype=torch.float64))]
    for kw in bad:
        args = dict(a_q=aq, a_s=as_, w_q=wq, w_s=ws_, out=out, ws=ws) | kw
        with pytest.raises(ValueError):
            moe.moe_gemm_fp8(**args)
    with pytest.raises(ValueError, match="CUDA"):  # right shapes, but host tensors
        moe.moe_gemm_fp8(aq, as_, wq, ws_, out, ws)
    off, ent = _t(3, dtype=torch.int32), _t(4, dtype=torch.int32)
    mq, ms = _t(2, 100, 272), _t(2, 1, 3, dtype=f32)
    for kw in [dict(offsets=_t(2, dtype=torch.int32)), dict(offsets=_t(3, dtype=torch.int64)),
               dict(entries=_t(3, dtype=torch.int32)), dict(w_q=_t(2, 100, 256)), dict(out=_t(4, 98, dtype=f32))]:
        args = dict(a_q=aq, a_s=as_, w_q=mq, w_s=ms, offsets=off, entries=ent, out=out, ws=ws) | kw
        with pytest.raises(ValueError):
            moe.moe_grouped_gemm_fp8(**args)
    gq, gs = _t(2, 128, 272), _t(2, 1, 3, dtype=f32)
    for kw in [dict(up_q=_t(2, 144, 272), up_s=_t(2, 2, 3, dtype=f32)), dict(q_out=_t(4, 144)),
               dict(s_out=_t(4, 2, dtype=f32))]:
        args = dict(a_q=aq, a_s=as_, gate_q=gq, gate_s=gs, up_q=gq, up_s=gs, offsets=off, entries=ent,
                    q_out=_t(4, 128), s_out=_t(4, 1, dtype=f32), ws=ws) | kw
        with pytest.raises(ValueError):
            moe.moe_grouped_swiglu_fp8(**args)
    x = _t(4, 256, dtype=torch.float16)
    for kw in [dict(weight=_t(256, dtype=torch.float16)), dict(weight=_t(255, dtype=f32)),
               dict(x=_t(4, 256, dtype=torch.float64)), dict(residual=_t(4, 256, dtype=f32)),
               dict(s_out=_t(4, 1, dtype=f32)), dict(y_out=_t(3, 256, dtype=torch.float16))]:
        args = dict(x=x, weight=_t(256, dtype=f32), eps=1e-6, q_out=_t(4, 256), s_out=_t(4, 2, dtype=f32)) | kw
        with pytest.raises(ValueError):
            moe.moe_rmsnorm_quant_fp8(**args)
    if torch.cuda.is_available():
        with pytest.raises(ValueError, match="one device"):
            moe.moe_rmsnorm_quant_fp8(x.cuda(), _t(256, dtype=f32), 1e-6, _t(4, 256), _t(4, 2, dtype=f32))


def test_binding_calls_on_the_tensors_device(monkeypatch):
    """A call for tensors of another device than the current one runs with that
    device current and on its stream."""
    current, seen = [0], []

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.old, current[0] = current[0], self.d

        def __exit__(self, *a):
            current[0] = self.old

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)

    def fn(*args):
        seen.append((current[0], args))
        return moe.MOE_OK

    moe._call(fn, "x", 1, None, (7,))
    moe._call(fn, "x", 0, None, (8,))
    assert seen == [(1, (7, 101)), (0, (8, 100))] and current == [0]


def _rounded(x):
    """The nearest number of 24 significant bits, ties to even (no range limits)."""
    if x == 0:
        return x
    e = abs(x.numerator).bit_length() - x.denominator.bit_length()
    e -= Fraction(2) ** e > abs(x)
    unit = Fraction(2) ** (e - 23)
    return round(x / unit) * unit


def test_quotients_round_as_the_division():
    """The kernels' quotient: with h = 1 / s and d = 1 - h s, both rounded to float32
    (d is exact), e = d + d^2 and v h + (v h) e, each step rounded once.  As 1 / s =
    h / (1 - d), before its last rounding it is off by the roundings of e, of v h
    and of their product, each 2^-24 of a term of 2^-24, and by d^3: 3 * 2^-24
    units at most.  A code changes only where the rounded quotient crosses a border
    of five significant bits, that is, where v / s lies that near to the middle
    between the border and the next float32: for v, s as 24-bit whole numbers A, S
    and the middle m, where |A 2^k - m S| is a few units.  As m is next to a multiple
    of 2^20, S has to be as well; all such S, m and A are gone through (and quotients
    at random)."""
    def check(A, S):
        h = _rounded(Fraction(1, S))
        d = 1 - h * S
        assert d == _rounded(d)
        e = _rounded(d + d * d)
        assert _rounded(A * h + _rounded(_rounded(A * h) * e)) == _rounded(Fraction(A, S)), (A, S)

    found = 0
    for S in (c * 2 ** 20 + d for c in range(8, 17) for d in range(-24, 25)):
        if not 2 ** 23 <= S < 2 ** 24:
            continue
        for border in range(16, 32):
            for finer in (20, 21, 22):        # below a power of two the next float32 is nearer
                for side in (-1, 1):
                    m = border * 2 ** finer + side
                    for j in range(-24, 25):
                        k = (m * S + j).bit_length() - 24
                        if (m * S + j) % 2 ** k == 0:
                            check((m * S + j) >> k, S)
                            found += 1
    assert found > 500
    rng = np.random.default_rng(0)
    for A, S in rng.integers(2 ** 23, 2 ** 24, (4000, 2)):
        check(int(A), int(S))


class _Faked(torch.Tensor):
    """A host tensor that says it lies on a CUDA device."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.on

    @property
    def device(self):
        return torch.device("cuda", self.on)


def _on(d, *shape, dtype=torch.uint8):
    t = torch.zeros(shape, dtype=dtype).as_subclass(_Faked)
    t.on = d
    return t


def test_expert_ffn_refuses_tensors_of_several_devices(monkeypatch, lib):
    f32, i32 = torch.float32, torch.int32
    T, H, I, E, k = 4, 256, 128, 8, 2
    calls = []
    monkeypatch.setattr(moe, "_call", lambda fn, where, dev, stream, args: calls.append(dev))

    def experts(n, d=1):
        return moe.Fp8Experts(_on(d, n, I, H), _on(d, n, 1, 2, dtype=f32), _on(d, n, I, H), _on(d, n, 1, 2, dtype=f32),
                              _on(d, n, H, I), _on(d, n, 2, 1, dtype=f32))

    def call(ex, sh, **kw):
        a = dict(x_q=_on(1, T, H), x_s=_on(1, T, 2, dtype=f32), offsets=_on(1, E + 1, dtype=i32),
                 entries=_on(1, T * k, dtype=i32), partial_out=_on(1, T * (k + 1), H, dtype=f32), ws=_on(1, 1 << 16)) | kw
        moe.moe_expert_ffn_fp8(ex, sh, shape=moe.shape_of(T, H, I, E, k), **a)

    call(experts(E), experts(1))
    assert calls == [1]
    for which in (0, 1):
        for field in ("gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s"):
            pair = [experts(E), experts(1)]
            setattr(pair[which], field, getattr(experts((E, 1)[which], 0), field))
            with pytest.raises(ValueError, match="one device"):
                call(*pair)
    for name, t in [("x_s", _on(0, T, 2, dtype=f32)), ("ws", _on(2, 1 << 16))]:
        with pytest.raises(ValueError, match="one device"):
            call(experts(E), experts(1), **{name: t})
    assert calls == [1]


def test_binding_refuses_integers_past_32_bits():
    """A group width that wraps into range is not taken for one that is."""
    f32, i32 = torch.float32, torch.int32
    aq, as_ = _t(4, 272), _t(4, 3, dtype=f32)
    off, ent, ws = _t(3, dtype=i32), _t(4, dtype=i32), _t(256)
    mq, ms = _t(2, 128, 272), _t(2, 1, 3, dtype=f32)
    for div in (1 << 31, 1 << 40, -(1 << 31) - 1, -(1 << 32) + 1, -(1 << 40)):
        with pytest.raises(ValueError, match="2\\^31"):
            moe.moe_grouped_gemm_fp8(aq, as_, mq, ms, off, ent, _t(4, 128, dtype=f32), ws, a_div=div)
        with pytest.raises(ValueError, match="2\\^31"):
            moe.moe_grouped_swiglu_fp8(aq, as_, mq, ms, mq, ms, off, ent, _t(4, 128), _t(4, 1, dtype=f32), ws, a_div=div)
    for div in (1 << 70, -(1 << 70), 1.5, "2"):
        with pytest.raises(TypeError, match="integer"):
            moe.moe_grouped_gemm_fp8(aq, as_, mq, ms, off, ent, _t(4, 128, dtype=f32), ws, a_div=div)


def test_workspace_calls_run_on_the_workspaces_device(monkeypatch):
    """Zeroing a workspace, setting its limits and reading its error are ordered
    with the calls that use it: on its device's current stream, with that device
    current, whatever device the caller is on."""
    current, seen = [0], []

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.old, current[0] = current[0], self.d

        def __exit__(self, *a):
            current[0] = self.old

    class Stream:
        cuda_stream = property(lambda self: 100 + current[0])

    class Lib:
        def __getattr__(self, name):
            def fn(*args):
                seen.append((name, current[0], args[-1]))
                return moe.MOE_OK
            return fn

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(moe, "load_library", Lib)
    for d in (0, 1):
        ws = _on(d, 256)
        for stream, want in ((None, 100 + d), (7, 7)):
            seen.clear()
            moe.moe_workspace_init(ws, stream)
            moe.moe_workspace_set_limits(ws, 1000, 0, stream)
            assert moe.moe_get_error(ws, stream) == 0
            assert seen == [(n, d, want) for n in ("moe_workspace_init", "moe_workspace_set_limits", "moe_get_error")]
            assert current == [0]
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_get_error(_t(256))


class _Compilers:
    """Stands in for subprocess.run: records the commands, fails those that
    `broken` picks."""

    def __init__(self, monkeypatch, tmp_path):
        self.ran, self.broken = [], lambda cmd: False
        monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
        monkeypatch.setattr(build.subprocess, "run", self)

    def __call__(self, cmd, **kw):
        self.ran.append(cmd)
        return build.subprocess.CompletedProcess(cmd, int(self.broken(cmd)), "", "")

    def build(self):
        self.ran.clear()
        build.build()
        return [c for c in self.ran if build.BINDING in c]


def test_binding_is_rebuilt_for_another_torch_or_python(lib, monkeypatch, tmp_path):
    c = _Compilers(monkeypatch, tmp_path)
    c.build()
    assert c.build() == []
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert len(c.build()) == 1
    assert c.build() == []
    monkeypatch.setattr(build.sys, "version", "another Python")
    assert len(c.build()) == 1
    c.broken = lambda cmd: build.BINDING in cmd
    monkeypatch.setattr(torch, "__version__", "a third")
    for _ in range(2):  # a build that failed is not taken for done
        with pytest.raises(RuntimeError):
            c.build()


def test_library_is_built_where_the_binding_cannot_be(lib, monkeypatch, tmp_path):
    """The C ABI needs no torch headers."""
    c = _Compilers(monkeypatch, tmp_path)
    c.broken = lambda cmd: build.BINDING in cmd
    monkeypatch.setattr(torch, "__version__", "other")
    monkeypatch.setattr(build, "_stale", lambda target, deps: True)
    with pytest.raises(RuntimeError, match="binding"):
        c.build()
    assert any(cmd[cmd.index("-o") + 1] == build.LIB for cmd in c.ran)
