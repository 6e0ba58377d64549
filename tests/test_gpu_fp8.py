"""The 8-bit operators on the GPU against the fp64 oracle, element by element.

Bounds, with u = 2^-24 and half(t) = finfo(t).eps / 2 of the output type:

products  The tensor core adds the 128 products of a block in four steps of 32
          to its float32 accumulator; a step loses at most one unit (2 u) of
          the largest partial sum for each of its 32 products and the
          accumulator, so a block at most 4 * 33 * 2 u of its terms' magnitude
          sum.  The two scales' product rounds once, and every block is scaled
          and added with one more: |err| <= (264 + blocks + 2) u M, M = sum
          |a w| scaled.
norm      The sum of squares has only positive terms and meets at most 16 fmas
          per thread and chunk pair, 5 shuffle and 16 warp additions (< 64
          roundings); its root halves that; the reciprocal root is within 2
          units (4 u), and the sum v, the mean, and two products round once
          each: |err| <= 40 u |n|.
codes     A code is off by half a step: 2^-4 of the value, 2^-10 of the scale
          below the normal range; plus the value's own error.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle as O
from oracle import fp8_oracle as F
from routed_expert_ffn_fp32_b200 import build, moe

from helpers import bits_np, rel_l2_rows

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe.load_library()


def half(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    """Half a step of the subnormals."""
    return torch.finfo(dt).tiny * torch.finfo(dt).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def codes_np(t):
    return t.view(torch.uint8).cpu().numpy()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def make_ws(n=256):
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    return ws


def rows8(rng, rows, K, spread=3):
    """Quantised N(0, 1) rows, each at its own magnitude 2^-spread .. 2^spread."""
    v = rng.standard_normal((rows, K)) * 2.0 ** rng.uniform(-spread, spread, (rows, 1))
    q, s = F.quantise(v)
    return q, s.astype(np.float32)


def mats8(rng, n, N, K):
    """Random codes of moderate size with block scales of very different sizes."""
    v = torch.from_numpy(rng.standard_normal((n, N, K), dtype=np.float32) * np.float32(60.0))
    q = v.to(FP8).view(torch.uint8).numpy()  # below 448 all of them
    assert (q & 0x7F != 0x7F).all()
    s = (2.0 ** rng.uniform(-12, -6, (n, F.blocks(N), F.blocks(K)))).astype(np.float32)
    return q, s


def prod_bound(K):
    return (264 + F.blocks(K) + 2) * U


def check_prod(got, want, mag, K, dt):
    err = np.abs(f64(got) - want)
    tol = prod_bound(K) * mag
    tol = tol + half(dt) * (np.abs(want) + tol) + tiny(dt)
    assert (err <= tol).all(), float((err / tol).max())


def check_codes(q, s, h, dh):
    """Codes and scales of rows h known within dh."""
    q, s = codes_np(q), f64(s)
    n = h.shape[1]
    want = F.scales(h)
    pad = np.zeros((h.shape[0], F.blocks(n) * 128))
    pad[:, :n] = dh
    ds = pad.reshape(h.shape[0], -1, 128).max(axis=2) / F.MAX + 2 * U * want
    assert (np.abs(s - want) <= ds).all(), float(np.abs(s / want - 1).max())
    wide = np.repeat(s, 128, axis=1)[:, :n]
    got = F.decode(q) * wide
    # reciprocal of the scale and the product with it: two roundings; a scale
    # below its block's maximum saturates it by its own error
    slack = dh + 4 * U * np.abs(h) + 448 * np.repeat(ds, 128, axis=1)[:, :n]
    tol = np.maximum(2.0 ** -4 * (np.abs(h) + slack), 2.0 ** -10 * wide) + slack
    assert (np.abs(got - h) <= tol).all(), float((np.abs(got - h) / tol).max())


# --------------------------------------------------------------------- norm ---
def run_norm(x, res, w, dt, eps=1e-6, y=True, res_out=None):
    rows, H = x.shape
    q = torch.full((rows, H), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, F.blocks(H)), -1.0, device="cuda")
    if res is not None and res_out is None:
        res_out = torch.empty_like(x)
    yo = torch.empty_like(x) if y else None
    moe.moe_rmsnorm_quant_fp8(x, w, eps, q, s, residual=res, residual_out=res_out, y_out=yo)
    torch.cuda.synchronize()
    return q, s, res_out, yo


NORM_CASES = [(1, 16), (3, 128), (1, 256), (130, 272), (5, 1024), (7, 1040), (33, 1408), (2, 2048), (5, 4096),
              (3, 7088), (2, 8192), (3, 8208), (2, 16384)]


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("rows,H", NORM_CASES)
def test_norm(rows, H, dt):
    rng = np.random.default_rng(H + rows)
    residual = (rows + H) % 3 != 0
    x = dev(rng.standard_normal((rows, H)) * 2.0 ** rng.uniform(-4, 4, (rows, 1)), dt)
    r = dev(rng.standard_normal((rows, H)), dt) if residual else None
    w = dev(1 + 0.2 * rng.standard_normal(H), F32)
    q, s, ro, y = run_norm(x, r, w, dt)
    v, n = F.rmsnorm(f64(x), None if r is None else f64(r), f64(w), 1e-6)
    if residual:
        assert (np.abs(f64(ro) - v) <= (half(dt) + 2 * U) * np.abs(v) + tiny(dt)).all()
    # v's own rounding is relative to v, so one unit of n
    dn = 40 * U * np.abs(n)
    assert (np.abs(f64(y) - n) <= dn + half(dt) * (np.abs(n) + dn) + tiny(dt)).all()
    check_codes(q, s, n, dn)


def test_norm_zero_rows_and_empty_call():
    w = torch.ones(256, device="cuda")
    x = torch.zeros(2, 256, dtype=BF16, device="cuda")
    q, s, _, y = run_norm(x, None, w, BF16)
    assert (codes_np(q) & 0x7F == 0).all() and (f64(s) == F.MIN_SCALE).all() and (f64(y) == 0).all()
    run_norm(x[:0], None, w, BF16)


def test_norm_nonfinite_rows_stay_local():
    rng = np.random.default_rng(4)
    xv = rng.standard_normal((4, 512))
    x = dev(xv, BF16)
    x[1, 5] = float("nan")
    x[2, 300] = float("inf")
    q, s, _, y = run_norm(x, None, torch.ones(512, device="cuda"), BF16)
    assert np.isnan(f64(y)[1]).all() and np.isnan(F.decode(codes_np(q)[1])).all()
    assert np.isnan(f64(y)[2, 300]) and np.isnan(F.decode(codes_np(q)[2, 300]))
    good = [0, 3]
    _, n = F.rmsnorm(f64(x)[good], None, np.ones(512), 1e-6)
    check_codes(q[good], s[good], n, 40 * U * np.abs(n))


def test_norm_in_place_residual():
    rng = np.random.default_rng(5)
    x, r = dev(rng.standard_normal((9, 4096)), BF16), dev(rng.standard_normal((9, 4096)), BF16)
    w = dev(1 + 0.1 * rng.standard_normal(4096), F32)
    q0, s0, ro0, y0 = run_norm(x, r, w, BF16)
    r1, x1 = r.clone(), x.clone()
    q1, s1 = torch.empty_like(q0), torch.empty_like(s0)
    moe.moe_rmsnorm_quant_fp8(x1, w, 1e-6, q1, s1, residual=r1, residual_out=r1, y_out=x1)
    for a, b in [(q0, q1), (s0, s1), (ro0, r1), (y0, x1)]:
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------- dense ---
GEMM_CASES = [
    # rows, N, K
    (1, 1, 16), (1, 2048, 4096), (2, 100, 128), (5, 136, 144), (7, 1000, 1424), (31, 129, 272), (33, 256, 1408),
    (64, 640, 512), (127, 128, 256), (128, 257, 384), (129, 384, 2048), (300, 1000, 1424), (257, 2050, 640),
    (1300, 4100, 272),   # 256-column tiles, ragged on both sides
    (16, 200, 384), (16, 136, 640), (15, 72, 640),   # whole and short last stages of several K blocks
    (700, 1600, 256), (700, 1602, 384),              # 128-column tiles, whole and odd sectors
]


@pytest.mark.parametrize("rows,N,K", GEMM_CASES)
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_gemm(rows, N, K, dt):
    rng = np.random.default_rng(rows + N + K)
    aq, as_ = rows8(rng, rows, K)
    wq, ws_ = mats8(rng, 1, N, K)
    ws = make_ws()
    out = torch.full((rows + 1, N), 7.0, dtype=dt, device="cuda")
    moe.moe_gemm_fp8(dev(aq), dev(as_), dev(wq[0]), dev(ws_[0]), out[:rows], ws)
    assert moe.moe_get_error(ws) == 0
    want, mag = F.gemm(F.dequant_rows(aq, as_), F.dequant_mats(wq[0], ws_[0]))
    check_prod(out[:rows], want, mag, K, dt)
    assert (out[rows:] == 7.0).all()  # the row behind the last is left alone


def test_gemm_many_tiles_per_sm():
    """Several tiles on every SM with a short K: the rings wrap within tiles and
    across them."""
    rng = np.random.default_rng(12)
    rows, N, K = 2100, 9000, 656
    aq, as_ = rows8(rng, rows, K)
    wq, ws_ = mats8(rng, 1, N, K)
    ws = make_ws()
    moe.moe_workspace_set_limits(ws, 100000)
    out = torch.empty(rows, N, device="cuda")
    args = [dev(t) for t in (aq, as_, wq[0], ws_[0])]
    for _ in range(4):
        moe.moe_gemm_fp8(*args, out, ws)
    assert moe.moe_get_error(ws) == 0
    a, w = F.dequant_rows(aq, as_), F.dequant_mats(wq[0], ws_[0])
    pick = rng.permutation(rows)[:200]
    want, mag = F.gemm(a[pick], w)
    check_prod(out[dev(pick)], want, mag, K, F32)


@pytest.mark.slow
@pytest.mark.parametrize("rows,N,K", [(33000, 65536, 16), (1 << 21, 16, 1040)])
def test_gemm_past_32_bit_offsets(rows, N, K):
    """Outputs, and operands, of more than 2^31 values: the last rows are right."""
    g = torch.Generator(device="cuda").manual_seed(3)
    aq = torch.randint(0, 96, (rows, K), generator=g, dtype=torch.uint8, device="cuda")  # values up to 8
    as_ = torch.rand(rows, F.blocks(K), generator=g, device="cuda") + 0.5
    wq = torch.randint(0, 96, (N, K), generator=g, dtype=torch.uint8, device="cuda")
    ws_ = torch.rand(F.blocks(N), F.blocks(K), generator=g, device="cuda") + 0.5
    out = torch.empty(rows, N, dtype=BF16, device="cuda")
    assert max(out.numel(), aq.numel()) > 2 ** 31
    ws = make_ws()
    moe.moe_gemm_fp8(aq, as_, wq, ws_, out, ws)
    assert moe.moe_get_error(ws) == 0
    pick = torch.tensor([0, 1, 127, 128, rows // 2, rows - 130, rows - 2, rows - 1], device="cuda")
    a = F.dequant_rows(codes_np(aq[pick]), f64(as_[pick]))
    want, mag = F.gemm(a, F.dequant_mats(codes_np(wq), f64(ws_)))
    check_prod(out[pick], want, mag, K, BF16)


def test_gemm_block_scales_and_order():
    """One-hot operands: every (row, column, K) position meets its own scales."""
    N, K, rows = 384, 512, 4
    rng = np.random.default_rng(0)
    as_ = rng.uniform(0.5, 2.0, (rows, 4)).astype(np.float32)
    ws_ = rng.uniform(0.5, 2.0, (3, 4)).astype(np.float32)
    ws = make_ws()
    for k in (0, 31, 127, 128, 300, 511):
        aq = np.zeros((rows, K), np.uint8)
        aq[:, k] = F.encode(np.arange(1, rows + 1))
        wq = F.encode(np.tile(np.arange(N)[:, None] % 13 - 6.0, (1, K)))
        out = torch.empty(rows, N, device="cuda")
        moe.moe_gemm_fp8(dev(aq), dev(as_), dev(wq), dev(ws_), out, ws)
        want, _ = F.gemm(F.dequant_rows(aq, as_), F.dequant_mats(wq, ws_))
        assert (np.abs(f64(out) - want) <= 3 * U * np.abs(want)).all(), k


def test_gemm_nan_stays_in_its_row_and_column():
    rng = np.random.default_rng(1)
    rows, N, K = 40, 300, 400
    aq, as_ = rows8(rng, rows, K)
    wq, ws_ = mats8(rng, 1, N, K)
    aq[3, 399] = 0x7F
    wq[0, 270, 0] = 0xFF
    out = torch.empty(rows, N, device="cuda")
    moe.moe_gemm_fp8(dev(aq), dev(as_), dev(wq[0]), dev(ws_[0]), out, make_ws())
    nan = np.isnan(f64(out))
    want = np.zeros((rows, N), bool)
    want[3] = True
    want[:, 270] = True
    np.testing.assert_array_equal(nan, want)


# ----------------------------------------------------------------- grouped ---
def routing(rng, T, k, E, skew=1.0, counts=None):
    """Pairs sorted by expert: (offsets, entries), experts by a skewed draw or
    with the given bucket sizes (k = 1)."""
    if counts is not None:
        idx = np.repeat(np.arange(E), counts)
        idx = idx[rng.permutation(len(idx))]
    else:
        p = np.arange(1, E + 1) ** -skew
        idx = np.stack([rng.choice(E, k, replace=False, p=p / p.sum()) for _ in range(T)]).reshape(-1)
    ent = np.argsort(idx, kind="stable").astype(np.int32)
    off = np.concatenate([[0], np.cumsum(np.bincount(idx, minlength=E))]).astype(np.int32)
    return off, ent


GROUP_CASES = [
    # T, k, E, N, K, skew
    (1, 8, 64, 256, 512, 0.0),
    (1, 1, 1, 1, 16, 0.0),
    (5, 2, 64, 1408, 1024, 1.0),
    (5, 8, 256, 1000, 272, 1.0),
    (77, 2, 8, 1000, 1424, 1.2),
    (200, 4, 16, 640, 384, 1.0),
    (300, 8, 1024, 128, 144, 0.5),
    (700, 2, 3, 2050, 256, 1.0),
    (1100, 8, 1024, 272, 144, 0.1),   # as many experts as there may be, full tiles
]


@pytest.mark.parametrize("T,k,E,N,K,skew", GROUP_CASES)
@pytest.mark.parametrize("a_div,scatter,dt", [(0, True, F32), (-1, False, BF16), (1, True, F16), (-1, True, F32),
                                              (0, False, BF16)])
def test_grouped(T, k, E, N, K, skew, a_div, scatter, dt):
    rng = np.random.default_rng(T + k + E + N)
    a_div = k if a_div < 0 else a_div
    off, ent = routing(rng, T, k, E, skew)
    P = T * k
    aq, as_ = rows8(rng, T if a_div == k else P, K)
    wq, ws_ = mats8(rng, E, N, K)
    ws = make_ws()
    out = torch.empty(P, N, dtype=dt, device="cuda")
    moe.moe_grouped_gemm_fp8(dev(aq), dev(as_), dev(wq), dev(ws_), dev(off), dev(ent), out, ws, a_div=a_div,
                             scatter=scatter)
    assert moe.moe_get_error(ws) == 0
    want, mag = F.grouped(F.dequant_rows(aq, as_), F.dequant_mats(wq, ws_), off, ent, a_div)
    got = out[dev(ent).long()] if scatter else out
    check_prod(got, want, mag, K, dt)


def test_grouped_bucket_sizes_around_tiles():
    counts = [0, 1, 127, 0, 128, 129, 3, 256, 31, 32, 33, 0, 63, 64, 65, 16, 17, 193]
    rng = np.random.default_rng(8)
    off, ent = routing(rng, 0, 1, len(counts), counts=counts)
    P, N, K = sum(counts), 200, 320
    aq, as_ = rows8(rng, P, K)
    wq, ws_ = mats8(rng, len(counts), N, K)
    for a_div in (0, 1):
        out = torch.empty(P, N, device="cuda")
        moe.moe_grouped_gemm_fp8(dev(aq), dev(as_), dev(wq), dev(ws_), dev(off), dev(ent), out, make_ws(),
                                 a_div=a_div, scatter=True)
        want, mag = F.grouped(F.dequant_rows(aq, as_), F.dequant_mats(wq, ws_), off, ent, a_div)
        check_prod(out[dev(ent).long()], want, mag, K, F32)


@pytest.mark.parametrize("T,skew", [(6, 0.5), (400, 0.5)])
def test_grouped_share_of_the_experts(T, skew):
    """A rank's experts: offsets that start and end inside the pairs; every
    other output row is left as it was."""
    rng = np.random.default_rng(9)
    k, E, N, K, e0, e1 = 4, 16, 136, 272, 4, 12
    off, ent = routing(rng, T, k, E, skew)
    aq, as_ = rows8(rng, T, K)
    wq, ws_ = mats8(rng, E, N, K)
    out = torch.full((T * k, N), 3.0, device="cuda")
    ws = make_ws()
    moe.moe_grouped_gemm_fp8(dev(aq), dev(as_), dev(wq[e0:e1]), dev(ws_[e0:e1]), dev(off[e0:e1 + 1]), dev(ent), out,
                             ws, a_div=k, scatter=True)
    assert moe.moe_get_error(ws) == 0
    want, mag = F.grouped(F.dequant_rows(aq, as_), F.dequant_mats(wq, ws_), off, ent, k)
    mine = np.arange(off[e0], off[e1])
    rest = np.setdiff1d(np.arange(T * k), mine)
    check_prod(out[dev(ent[mine]).long()], want[mine], mag[mine], K, F32)
    assert (out[dev(ent[rest]).long()] == 3.0).all()


def swiglu_ref(a, gate, up, off, ent, a_div, K):
    """h and a bound of its error: |silu'| <= 1.1, the exponential, division
    and products a few units."""
    g, gm = F.grouped(a, gate, off, ent, a_div)
    u, um = F.grouped(a, up, off, ent, a_div)
    dg, du = prod_bound(K) * gm, prod_bound(K) * um
    h = F.silu(g) * u
    return h, 1.1 * dg * (np.abs(u) + du) + np.abs(F.silu(g)) * du + 16 * U * np.abs(h) + 2.0 ** -140


SWIGLU_CASES = [
    # T, k, E, I, H, a_div
    (1, 8, 64, 256, 512, -1),
    (1, 2, 4, 16, 16, -1),
    (5, 2, 64, 1408, 1024, -1),
    (5, 4, 16, 144, 272, 0),
    (77, 2, 8, 400, 1424, -1),
    (300, 4, 16, 640, 384, -1),
    (300, 8, 1024, 128, 144, 1),
    (700, 2, 3, 272, 256, 0),
    (3, 8, 64, 256, 272, -1),
    (640, 3, 8, 1040, 384, -1),
    (1100, 8, 1024, 144, 144, -1),
]


@pytest.mark.parametrize("T,k,E,I,H,a_div", SWIGLU_CASES)
def test_swiglu(T, k, E, I, H, a_div):
    rng = np.random.default_rng(T + k + E + I)
    a_div = k if a_div < 0 else a_div
    off, ent = routing(rng, T, k, E)
    P = T * k
    aq, as_ = rows8(rng, T if a_div == k else P, H, spread=1)
    gq, gs = mats8(rng, E, I, H)
    uq, us = mats8(rng, E, I, H)
    gs *= 2.0 ** -3  # gate values of a few units
    ws = make_ws()
    q = torch.empty(P, I, dtype=FP8, device="cuda")
    s = torch.empty(P, F.blocks(I), device="cuda")
    moe.moe_grouped_swiglu_fp8(dev(aq), dev(as_), dev(gq), dev(gs), dev(uq), dev(us), dev(off), dev(ent), q, s, ws,
                               a_div=a_div)
    assert moe.moe_get_error(ws) == 0
    h, dh = swiglu_ref(F.dequant_rows(aq, as_), F.dequant_mats(gq, gs), F.dequant_mats(uq, us), off, ent, a_div, H)
    check_codes(q, s, h, dh)


@pytest.mark.parametrize("rows", [3, 150])
def test_swiglu_one_group(rows):
    """offsets None: one matrix pair over all rows (a shared expert); extreme
    gates (silu near 0 and near the identity)."""
    rng = np.random.default_rng(rows)
    I, H = 272, 256
    aq, as_ = rows8(rng, rows, H, spread=8)
    gq, gs = mats8(rng, 1, I, H)
    uq, us = mats8(rng, 1, I, H)
    q = torch.empty(rows, I, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, F.blocks(I), device="cuda")
    ws = make_ws()
    moe.moe_grouped_swiglu_fp8(dev(aq), dev(as_), dev(gq), dev(gs), dev(uq), dev(us), None, None, q, s, ws)
    assert moe.moe_get_error(ws) == 0
    off, ent = np.array([0, rows]), np.arange(rows)
    h, dh = swiglu_ref(F.dequant_rows(aq, as_), F.dequant_mats(gq, gs), F.dequant_mats(uq, us), off, ent, 0, H)
    check_codes(q, s, h, dh)


# --------------------------------------------------------- bad device data ---
@pytest.mark.parametrize("off", [[0, 5, 3, 8], [-1, 2, 4, 8], [0, 2, 4, 9]])
@pytest.mark.parametrize("N", [128, 20000])
def test_bad_offsets_are_latched_and_nothing_is_written(off, N):
    rng = np.random.default_rng(2)
    K, P = 256, 8
    aq, as_ = rows8(rng, P, K)
    wq = torch.zeros(3, N, K, dtype=torch.uint8, device="cuda")
    ws_ = torch.ones(3, F.blocks(N), 2, device="cuda")
    out = torch.full((P, N), 5.0, device="cuda")
    ws = make_ws()
    moe.moe_grouped_gemm_fp8(dev(aq), dev(as_), wq, ws_, dev(np.array(off, np.int32)), dev(np.arange(P, dtype=np.int32)),
                             out, ws, scatter=True)
    assert moe.moe_get_error(ws) == moe.MOE_ERR_DEVICE_DATA
    assert (out == 5.0).all()
    assert moe.moe_get_error(ws) == 0


@pytest.mark.parametrize("P", [6, 400])
def test_bad_entries_skip_their_rows(P):
    rng = np.random.default_rng(3)
    E, N, K, T = 2, 136, 144, P
    aq, as_ = rows8(rng, T, K)
    wq, ws_ = mats8(rng, E, N, K)
    off = np.array([0, P // 2, P], np.int32)
    ent = np.arange(P, dtype=np.int32)
    bad = {1: -3, P - 2: P + 5}
    for p, v in bad.items():
        ent[p] = v
    out = torch.full((P, N), 5.0, device="cuda")
    ws = make_ws()
    moe.moe_grouped_gemm_fp8(dev(aq), dev(as_), dev(wq), dev(ws_), dev(off), dev(ent), out, ws, a_div=1, scatter=True)
    assert moe.moe_get_error(ws) == moe.MOE_ERR_DEVICE_DATA
    fine = np.setdiff1d(np.arange(P), list(bad))
    want, mag = F.grouped(F.dequant_rows(aq, as_), F.dequant_mats(wq, ws_), off, np.arange(P), 1)
    check_prod(out[dev(fine)], want[fine], mag[fine], K, F32)
    assert (out[dev(np.array(list(bad)))] == 5.0).all()
    q = torch.full((P, 144), 0x11, dtype=torch.uint8, device="cuda")
    s = torch.full((P, 2), -1.0, device="cuda")
    gq, gs = mats8(rng, E, 144, K)
    moe.moe_grouped_swiglu_fp8(dev(aq), dev(as_), dev(gq), dev(gs), dev(gq), dev(gs), dev(off), dev(ent), q, s, ws,
                               a_div=1)
    assert moe.moe_get_error(ws) == moe.MOE_ERR_DEVICE_DATA
    at = dev(np.array(list(bad)))
    assert (q[at] == 0x11).all() and (s[at] == -1.0).all()
    h, dh = swiglu_ref(F.dequant_rows(aq, as_), F.dequant_mats(gq, gs), F.dequant_mats(gq, gs), off, np.arange(P), 1, K)
    check_codes(q[dev(fine)], s[dev(fine)], h[fine], dh[fine])


# ------------------------------------------------- streams, graphs, repeats ---
def _prefill(seed, rows=300, N=700, K=640):
    rng = np.random.default_rng(seed)
    aq, as_ = rows8(rng, rows, K)
    wq, ws_ = mats8(rng, 1, N, K)
    return [dev(t) for t in (aq, as_, wq[0], ws_[0])], torch.empty(rows, N, device="cuda")


@pytest.mark.parametrize("rows", [1, 300, 3000])
def test_repeated_and_captured_calls_are_identical(rows):
    args, out = _prefill(3, rows)
    ws = make_ws()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.moe_gemm_fp8(*args, out, ws)
        torch.cuda.synchronize()
        first = out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            moe.moe_gemm_fp8(*args, out, ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    assert moe.moe_get_error(ws) == 0


def test_two_streams_share_a_workspace():
    """Only status words live in the workspace: calls on two streams, and two
    graphs captured over it, do not touch each other."""
    ws = make_ws()
    work = [_prefill(k, rows) for k, rows in ((1, 4), (2, 500))]
    want = []
    for args, out in work:
        moe.moe_gemm_fp8(*args, out, ws)
        torch.cuda.synchronize()
        want.append(out.clone())
    streams = [torch.cuda.Stream() for _ in work]
    graphs = []
    for (args, out), st in zip(work, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(4):
                moe.moe_gemm_fp8(*args, out, ws, stream=st)
        graphs.append(g)
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for (args, out), st, g in zip(work, streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
                moe.moe_gemm_fp8(*args, out, ws, stream=st)
    torch.cuda.synchronize()
    for (_, out), w in zip(work, want):
        assert torch.equal(out, w)
    assert moe.moe_get_error(ws) == 0


@pytest.mark.parametrize("rows,N", [(200, 8192), (2, 256)])
def test_expired_wait_latches_timeout_and_next_call_recovers(rows, N):
    rng = np.random.default_rng(6)
    K = 1024
    aq, as_ = rows8(rng, rows, K)
    gq, gs = mats8(rng, 1, N, K)
    q = torch.empty(rows, N, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, F.blocks(N), device="cuda")
    args = [dev(t) for t in (aq, as_, gq, gs, gq, gs)]
    ws = make_ws()
    moe.moe_workspace_set_limits(ws, 1000, moe.MOE_DEBUG_STARVE_FIRST_WAIT)
    moe.moe_grouped_swiglu_fp8(*args, None, None, q, s, ws)
    assert moe.moe_get_error(ws) == moe.MOE_ERR_TIMEOUT
    moe.moe_workspace_set_limits(ws, 0, 0)
    moe.moe_grouped_swiglu_fp8(*args, None, None, q, s, ws)
    assert moe.moe_get_error(ws) == 0
    off, ent = np.array([0, rows]), np.arange(rows)
    a, w = F.dequant_rows(aq, as_), F.dequant_mats(gq, gs)
    h, dh = swiglu_ref(a, w, w, off, ent, 0, K)
    check_codes(q, s, h, dh)


# ----------------------------------------------------------- run together ---
@pytest.mark.parametrize("T,shared", [(1, False), (5, True), (260, True)])
def test_layer_norm_route_experts_combine(T, shared):
    """norm -> router -> bucket -> 8-bit experts -> combine, as a layer runs
    them.  The oracle starts from the operators' own 8-bit rows; h is quantised
    on both sides, so a value next to a rounding border may take the other
    code: rows within 5e-3 (the bar of the MXFP4 activation path)."""
    rng = np.random.default_rng(T)
    H, I, E, k = 512, 272 + 16 * 1, 16, 4   # I = 288: the last block of h is short
    x = dev(rng.standard_normal((T, H)), BF16)
    r = dev(2 * rng.standard_normal((T, H)), BF16)
    w = dev(1 + 0.1 * rng.standard_normal(H), F32)
    W_r = dev(rng.standard_normal((E, H)) * 0.05, F32)

    def experts(n):
        g, u, d = mats8(rng, n, I, H), mats8(rng, n, I, H), mats8(rng, n, H, I)
        parts = dict(gate_q=g[0], gate_s=g[1] / 8, up_q=u[0], up_s=u[1], down_q=d[0], down_s=d[1])
        return parts, moe.Fp8Experts(**{n_: dev(t) for n_, t in parts.items()})

    ex_np, ex = experts(E)
    sh_np, sh = experts(1) if shared else (None, None)
    shape = moe.shape_of(T, H, I, E, k)
    n_bytes = max(moe.moe_workspace_bytes(shape, moe.MOE_PATH_GEMV),
                  moe.load_library().moe_expert_ffn_fp8_workspace_bytes(shape, int(shared)))
    ws = make_ws(n_bytes)
    q = torch.empty(T, H, dtype=FP8, device="cuda")
    s = torch.empty(T, F.blocks(H), device="cuda")
    res, y = torch.empty_like(x), torch.empty_like(x)
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    tw = torch.empty((T, k), device="cuda")
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    ent = torch.empty(T * k, dtype=torch.int32, device="cuda")
    partial = torch.empty((T * (k + shared), H), device="cuda")
    out = torch.empty((T, H), dtype=torch.int16, device="cuda")

    def layer():
        moe.moe_rmsnorm_quant_fp8(x, w, 1e-6, q, s, residual=r, residual_out=res, y_out=y)
        moe.moe_route_topk(y, W_r, None, shape, idx, tw, ws)
        moe.moe_bucket(idx, shape, counts, off, ent, ws)
        moe.moe_expert_ffn_fp8(ex, sh, q, s, off, ent, shape, partial, ws)
        moe.moe_combine(partial, tw, shape, shared, out)

    layer()
    torch.cuda.synchronize()
    assert moe.moe_get_error(ws) == 0
    first, first_q = bits_np(out).copy(), codes_np(q).copy()

    a = F.dequant_rows(codes_np(q), f64(s))
    offn, entn = off.cpu().numpy(), ent.cpu().numpy()
    want = np.zeros((T * (k + shared), H))

    def ffn(parts, rows_of, offs, ents, div):
        m = {n_: F.dequant_mats(parts[n_ + "_q"], parts[n_ + "_s"]) for n_ in ("gate", "up", "down")}
        g, _ = F.grouped(a, m["gate"], offs, ents, div)
        u, _ = F.grouped(a, m["up"], offs, ents, div)
        hq, hs = F.quantise(F.silu(g) * u)
        o, _ = F.grouped(F.dequant_rows(hq, hs), m["down"], offs, ents, 0)
        want[rows_of] = o

    ffn(ex_np, entn, offn, entn, k)
    if shared:
        ffn(sh_np, np.arange(T * k, T * k + T), np.array([0, T]), np.arange(T), 0)
    assert rel_l2_rows(f64(partial), want).max() < 5e-3
    comb = (want[:T * k].reshape(T, k, H) * f64(tw)[:, :, None]).sum(axis=1)
    if shared:
        comb = comb + want[T * k:]
    assert rel_l2_rows(O.bf16_bits_to_f64(first), comb).max() < 5e-3 + half(BF16)

    # the same captured and replayed
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        layer()
    for t in (out, partial, q):
        t.view(torch.uint8).zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits_np(out), first)
    np.testing.assert_array_equal(codes_np(q), first_q)
    assert moe.moe_get_error(ws) == 0


# ------------------------------------------------- codes at rounding borders ---
def around_borders(rng, n, top):
    """n float32 values of a block whose largest is `top`: `top` first, then
    values within two units of the middle between neighbouring codes, times the
    block's scale, in the upper half of the range."""
    s = np.float32(top) / np.float32(F.MAX)
    mags = F.decode(np.arange(127))
    mid = (mags[1:] + mags[:-1]) / 2
    mid = mid[(mid > 226) & (mid < 440)]
    v = (rng.choice(mid, n) * np.float64(s)).astype(np.float32)
    for _ in range(2):
        way = rng.integers(-1, 2, n)
        v = np.where(way == 0, v, np.nextafter(v, np.where(way < 0, 0, np.inf).astype(np.float32)))
    v[0] = top
    return v


def quotient_codes(v):
    """Codes and scales of float32 rows as the header defines them: float32
    quotients, rounded to E4M3."""
    blocks = np.abs(v).reshape(v.shape[0], -1, 128).max(axis=2)
    s = np.maximum(blocks / np.float32(F.MAX), np.float32(F.MIN_SCALE))
    assert s.dtype == np.float32 and v.dtype == np.float32
    return F.encode(v / np.repeat(s, 128, axis=1)), s


def test_norm_codes_are_rounded_quotients():
    """Rows of +-1 with eps = 0 have norm 1, so n is the weight exactly."""
    rng = np.random.default_rng(21)
    H = 16384
    for _ in range(4):
        w = np.concatenate([around_borders(rng, 128, rng.uniform(1, 2) * 2.0 ** rng.integers(-115, 120))
                            for _ in range(H // 128)]).astype(np.float32)
        w[5::128] = 0.0                          # the sign of a zero stays
        sign = rng.choice(np.array([-1, 1], np.float32), (3, H))
        q, s, _, y = run_norm(dev(sign), None, dev(w), F32, eps=0.0)
        n = sign * w
        np.testing.assert_array_equal(y.cpu().numpy(), n)
        want_q, want_s = quotient_codes(n)
        np.testing.assert_array_equal(s.cpu().numpy(), want_s)
        np.testing.assert_array_equal(codes_np(q), want_q)


@pytest.mark.parametrize("rows,blocks", [(3, 16), (3, 60), (3, 100), (40, 16), (150, 18), (150, 37), (150, 80)])
def test_swiglu_codes_are_rounded_quotients(rows, blocks):
    """Gates of 32, whose silu is 32 exactly, and ups put together from six
    K blocks of four bits each, so h = 32 u exactly.  The column blocks run over
    clusters of 4, 2 and 1 on each side of the tile heights."""
    rng = np.random.default_rng(rows + blocks)
    I, H = 128 * blocks, 7 * 128
    u = np.stack([around_borders(rng, 128, np.float32(2 ** 24 - rng.integers(1, 2 ** 15))) for _ in range(blocks)])
    u = u.reshape(-1).astype(np.int64)
    assert (u >= 2 ** 23).all() and (u < 2 ** 24).all()   # 24-bit whole numbers, each a float32
    uq, gq = np.zeros((1, I, H)), np.zeros((1, I, H))
    gq[0, :, 0] = 32.0
    us = np.ones((1, blocks, 7), np.float32)
    for b in range(6):
        uq[0, :, 128 * (b + 1)] = (u >> (20 - 4 * b)) & 15
        us[0, :, b + 1] = 2.0 ** -(4 * b)
    gs = np.ones((1, blocks, 7), np.float32)
    aq = np.zeros((rows, H))
    aq[:, ::128] = 1.0
    power = rng.integers(-3, 4, rows)           # rows at their own power of two
    as_ = np.ones((rows, 7), np.float32)
    as_[:, 1:] = 2.0 ** power[:, None]
    q = torch.empty(rows, I, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, blocks, device="cuda")
    ws = make_ws()
    moe.moe_grouped_swiglu_fp8(*(dev(t) for t in (F.encode(aq), as_, F.encode(gq), gs, F.encode(uq), us)), None, None,
                               q, s, ws)
    assert moe.moe_get_error(ws) == 0
    h = (32.0 * u[None] * 2.0 ** -20 * 2.0 ** power[:, None]).astype(np.float32)
    want_q, want_s = quotient_codes(h)
    np.testing.assert_array_equal(s.cpu().numpy(), want_s)
    np.testing.assert_array_equal(codes_np(q), want_q)


@pytest.mark.parametrize("rows", [3, 40, 150])
def test_swiglu_silu_over_the_range(rows):
    """silu against 64 bits through the block maxima: one column of every block
    has a gate, exactly known (code 1 times a scale and a power of two), and an
    up of 2^20, so s 448 = |silu(g)| 2^20.  Within 16 units of 2^-24 in all, two
    of them for the scale's division and this test's own product."""
    rng = np.random.default_rng(rows)
    blocks, H = 400, 128
    g = np.concatenate([np.linspace(-88, 88, 340), 10.0 ** rng.uniform(-6, 0, 60) * rng.choice([-1, 1], 60)])
    gs = np.abs(g).astype(np.float32).reshape(1, blocks, 1)
    gq, uq = np.zeros((1, blocks * 128, H)), np.zeros((1, blocks * 128, H))
    at = np.arange(blocks) * 128 + rng.integers(0, 128, blocks)
    gq[0, at, 5] = np.sign(g)
    uq[0, at, 5] = 1.0
    us = np.full((1, blocks, 1), 2.0 ** 20, np.float32)
    aq = np.zeros((rows, H))
    aq[:, 5] = 1.0
    down = 2.0 ** -(np.arange(rows) % 5)        # the row's own power of two, in gate and up
    q = torch.empty(rows, blocks * 128, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, blocks, device="cuda")
    ws = make_ws()
    moe.moe_grouped_swiglu_fp8(*(dev(t) for t in (F.encode(aq), down[:, None].astype(np.float32), F.encode(gq), gs,
                                                  F.encode(uq), us)), None, None, q, s, ws)
    assert moe.moe_get_error(ws) == 0
    gate = (np.sign(g) * gs.reshape(-1).astype(np.float64))[None] * down[:, None]
    want = np.abs(F.silu(gate)) * 2.0 ** 20 * down[:, None]
    err = np.abs(f64(s) * F.MAX / want - 1)
    assert err.max() <= 16 * U, (float(err.max() / U), float(gate.reshape(-1)[err.argmax()]))


# ------------------------------------------------------- paths of few calls ---
@pytest.mark.parametrize("T,k,E,N,K", [
    (5, 8, 256, 1000, 512),    # 128-column tiles, two K blocks a stage
    (5, 8, 256, 1000, 640),    # the same, a short last stage
    (12, 4, 64, 136, 640),     # 64-column tiles, four K blocks a stage, a short last stage
    (12, 4, 64, 136, 1024),    # the same, whole stages
    (40, 1, 5, 200, 384),      # buckets of several tiles
])
@pytest.mark.parametrize("scatter", [False, True])
def test_grouped_rows_in_order_several_blocks_per_copy(T, k, E, N, K, scatter):
    """Small buckets of rows in bucket order, K of whole blocks: a stage's rows
    are one copy, at the tile's first row."""
    rng = np.random.default_rng(T + E + K)
    off, ent = routing(rng, T, k, E)
    P = T * k
    assert 16 <= P <= 8 * E and K % 128 == 0
    aq, as_ = rows8(rng, P, K)
    wq, ws_ = mats8(rng, E, N, K)
    ws = make_ws()
    out = torch.empty(P, N, device="cuda")
    moe.moe_grouped_gemm_fp8(dev(aq), dev(as_), dev(wq), dev(ws_), dev(off), dev(ent), out, ws, scatter=scatter)
    assert moe.moe_get_error(ws) == 0
    want, mag = F.grouped(F.dequant_rows(aq, as_), F.dequant_mats(wq, ws_), off, ent, 0)
    check_prod(out[dev(ent).long()] if scatter else out, want, mag, K, F32)


@pytest.mark.parametrize("P,E,I,H", [(20, 4, 256, 640), (24, 4, 1280, 384), (40, 5, 4096, 512), (16, 1, 272, 640),
                                     (16, 1, 8192, 256)])
def test_swiglu_rows_in_order_several_blocks_per_copy(P, E, I, H):
    """The same for the pair, in clusters of 4, 2 and 1; E = 1 without offsets."""
    rng = np.random.default_rng(P + I)
    off, ent = routing(rng, P, 1, E)
    aq, as_ = rows8(rng, P, H, spread=1)
    gq, gs = mats8(rng, E, I, H)
    uq, us = mats8(rng, E, I, H)
    gs *= 2.0 ** -3
    ws = make_ws()
    q = torch.empty(P, I, dtype=torch.uint8, device="cuda")
    s = torch.empty(P, F.blocks(I), device="cuda")
    moe.moe_grouped_swiglu_fp8(*(dev(t) for t in (aq, as_, gq, gs, uq, us)), dev(off) if E > 1 else None, None, q, s, ws)
    assert moe.moe_get_error(ws) == 0
    h, dh = swiglu_ref(F.dequant_rows(aq, as_), F.dequant_mats(gq, gs), F.dequant_mats(uq, us), off, ent, 0, H)
    check_codes(q, s, h, dh)


@pytest.mark.parametrize("T,k", [(5, 4), (16, 2)])
def test_expert_ffn_whole_blocks(T, k):
    """I and H of whole blocks, with the shared expert: the down projection's
    rows, and at T = 16 the shared expert's, come several K blocks per copy."""
    rng = np.random.default_rng(T)
    H, I, E = 384, 256, 16
    x, xs = rows8(rng, T, H, spread=1)
    off, ent = routing(rng, T, k, E)
    parts = []
    for n in (E, 1):
        g, u, d = mats8(rng, n, I, H), mats8(rng, n, I, H), mats8(rng, n, H, I)
        parts.append(dict(gate_q=g[0], gate_s=g[1] / 8, up_q=u[0], up_s=u[1], down_q=d[0], down_s=d[1]))
    ex, sh = (moe.Fp8Experts(**{n: dev(t) for n, t in p.items()}) for p in parts)
    shape = moe.shape_of(T, H, I, E, k)
    ws = moe.fp8_workspace(shape, True)
    partial = torch.empty(T * (k + 1), H, device="cuda")
    moe.moe_expert_ffn_fp8(ex, sh, dev(x), dev(xs), dev(off), dev(ent), shape, partial, ws)
    assert moe.moe_get_error(ws) == 0
    a, want = F.dequant_rows(x, xs), np.zeros((T * (k + 1), H))
    groups = ((parts[0], off, ent, k, ent), (parts[1], np.array([0, T]), np.arange(T), 0, np.arange(T * k, T * k + T)))
    for p, offs, ents, div, rows in groups:
        g, u, d = (F.dequant_mats(p[n + "_q"], p[n + "_s"]) for n in ("gate", "up", "down"))
        h = F.silu(F.grouped(a, g, offs, ents, div)[0]) * F.grouped(a, u, offs, ents, div)[0]
        want[rows] = F.grouped(F.dequant_rows(*F.quantise(h)), d, offs, ents, 0)[0]
    # h is quantised on both sides: a value next to a border may take the other
    # code, the bar of the layer test above
    assert rel_l2_rows(f64(partial), want).max() < 5e-3


@pytest.mark.parametrize("rows,N,K", [(3, 200, 65536), (16, 72, 7168), (40, 136, 16400), (150, 136, 7168)])
def test_gemm_long_k(rows, N, K):
    rng = np.random.default_rng(K)
    aq, as_ = rows8(rng, rows, K)
    wq, ws_ = mats8(rng, 1, N, K)
    out = torch.empty(rows, N, device="cuda")
    ws = make_ws()
    moe.moe_gemm_fp8(dev(aq), dev(as_), dev(wq[0]), dev(ws_[0]), out, ws)
    assert moe.moe_get_error(ws) == 0
    want, mag = F.gemm(F.dequant_rows(aq, as_), F.dequant_mats(wq[0], ws_[0]))
    check_prod(out, want, mag, K, F32)


@pytest.mark.parametrize("T,k,E,K", [(5, 2, 8, 7168), (90, 2, 4, 7184)])
def test_grouped_and_swiglu_long_k(T, k, E, K):
    rng = np.random.default_rng(T + K)
    off, ent = routing(rng, T, k, E)
    aq, as_ = rows8(rng, T, K, spread=1)
    gq, gs = mats8(rng, E, 144, K)
    uq, us = mats8(rng, E, 144, K)
    gs *= 2.0 ** -5
    ws = make_ws()
    a, g, u = F.dequant_rows(aq, as_), F.dequant_mats(gq, gs), F.dequant_mats(uq, us)
    args = [dev(t) for t in (aq, as_, gq, gs, uq, us)]
    out = torch.empty(T * k, 144, device="cuda")
    moe.moe_grouped_gemm_fp8(*args[:4], dev(off), dev(ent), out, ws, a_div=k, scatter=True)
    q = torch.empty(T * k, 144, dtype=torch.uint8, device="cuda")
    s = torch.empty(T * k, 2, device="cuda")
    moe.moe_grouped_swiglu_fp8(*args, dev(off), dev(ent), q, s, ws, a_div=k)
    assert moe.moe_get_error(ws) == 0
    want, mag = F.grouped(a, g, off, ent, k)
    check_prod(out[dev(ent).long()], want, mag, K, F32)
    check_codes(q, s, *swiglu_ref(a, g, u, off, ent, k, K))


# --------------------------------------------------------------- non-finite ---
@pytest.mark.parametrize("T,k,E,N,K", [(5, 8, 256, 200, 512), (6, 2, 16, 136, 272), (77, 2, 8, 200, 400),
                                       (300, 4, 8, 136, 272)])
def test_grouped_nan_stays_in_its_rows(T, k, E, N, K):
    """Rows full of NaN beside clean ones, in 16-row tiles (whose MMAs read past
    their rows), half tiles and full ones: every clean row is right."""
    rng = np.random.default_rng(T + K)
    off, ent = routing(rng, T, k, E)
    P = T * k
    aq, as_ = rows8(rng, P, K)
    sick = rng.random(P) < 0.6
    aq[sick] = 0x7F
    as_[sick & (np.arange(P) % 2 == 0)] = np.inf
    wq, ws_ = mats8(rng, E, N, K)
    ws = make_ws()
    out = torch.empty(P, N, device="cuda")
    moe.moe_grouped_gemm_fp8(dev(aq), dev(as_), dev(wq), dev(ws_), dev(off), dev(ent), out, ws)
    assert moe.moe_get_error(ws) == 0
    aq[sick], as_[sick] = 0, 0
    want, mag = F.grouped(F.dequant_rows(aq, as_), F.dequant_mats(wq, ws_), off, ent, 0)
    check_prod(out[dev(~sick)], want[~sick], mag[~sick], K, F32)
    assert np.isnan(f64(out)[sick]).all()


@pytest.mark.parametrize("rows", [3, 40, 150])
def test_swiglu_nonfinite_gates(rows):
    """NaN and infinite gates and ups, block by block, and gates far below zero.
    A NaN stays in its place and out of the maximum; an infinite maximum makes
    the scale infinite, finite codes 0 and the infinite ones NaN."""
    I, H = 7 * 128, 128
    gq, uq = np.zeros((1, I, H)), np.zeros((1, I, H))
    j = np.arange(128)
    col = lambda b: slice(128 * b, 128 * b + 128)  # noqa: E731
    gate = np.stack([(j % 7 - 3.0) / 2] * 7)       # gates of the blocks
    up = np.stack([(j % 9 - 4.0) / 4] * 7)
    gs, us = np.ones((1, 7, 1), np.float32), np.ones((1, 7, 1), np.float32)
    gate[1, 17] = np.nan
    up[2, 90] = np.nan
    gs[0, 3] = np.inf            # +inf, -inf and, where the gate's code is 0, NaN
    us[0, 4] = np.inf
    gate[5] = -1.0
    gs[0, 5] = 200.0             # silu counts as 0, beside ...
    gate[5, 3], up[5, 3] = 0.25, 1.0  # ... one gate of 50
    gate[6] = 1.0
    gs[0, 6] = 3e38              # silu the identity, h infinite where |up| exceeds 1
    up[6, 100] = 1.5
    up[6, 101] = 0.5
    aq = np.zeros((rows, H))
    aq[:, 3] = 1.0
    for b in range(7):
        gq[0, col(b), 3], uq[0, col(b), 3] = gate[b], up[b]
    args = [F.encode(aq), np.ones((rows, 1), np.float32), F.encode(gq), gs, F.encode(uq), us]
    q = torch.empty(rows, I, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, 7, device="cuda")
    ws = make_ws()
    moe.moe_grouped_swiglu_fp8(*(dev(t) for t in args), None, None, q, s, ws)
    assert moe.moe_get_error(ws) == 0
    with np.errstate(all="ignore"):
        g = F.decode(args[2])[0, :, 3] * np.repeat(gs.reshape(-1).astype(np.float64), 128)
        u = F.decode(args[4])[0, :, 3] * np.repeat(us.reshape(-1).astype(np.float64), 128)
        h = F.silu(g) * u
        h = np.where(np.abs(h) > np.finfo(np.float32).max, np.copysign(np.inf, h), h)
        h = np.where(g < -88.8, h * 0, h)          # silu counts as 0 there
        want_s = F.scales(h[None])[0]
        t = h / np.repeat(want_s, 128)
    assert np.isinf(want_s[[3, 4, 6]]).all() and np.isfinite(want_s[[0, 1, 2, 5]]).all()
    got_s, got = f64(s), F.decode(codes_np(q))
    for r in range(rows):
        assert (np.abs(got_s[r, [0, 1, 2, 5]] / want_s[[0, 1, 2, 5]] - 1) <= 18 * U).all()
        assert np.isposinf(got_s[r, [3, 4, 6]]).all()
        np.testing.assert_array_equal(np.isnan(got[r]), np.isnan(t))
        fine = ~np.isnan(t)
        # half a step, and the quotient's own 20 units
        tol = np.maximum(np.abs(t[fine]) * (2.0 ** -4 + 20 * U), 2.0 ** -10)
        assert (np.abs(got[r][fine] - t[fine]) <= tol).all()


def test_norm_rows_past_float32_come_out_as_zeros():
    rng = np.random.default_rng(7)
    for dt in (BF16, F32):
        x = dev(rng.standard_normal((4, 512)), dt)
        x[1] *= 1e30
        x[2, 40] = 3e38
        q, s, _, y = run_norm(x, None, torch.ones(512, device="cuda"), dt)
        for r in (1, 2):
            assert (f64(y)[r] == 0).all() and (f64(s)[r] == F.MIN_SCALE).all()
            assert (F.decode(codes_np(q))[r] == 0).all()
        good = [0, 3]
        _, n = F.rmsnorm(f64(x)[good], None, np.ones(512), 1e-6)
        check_codes(q[good], s[good], n, 40 * U * np.abs(n))


def test_first_call_of_a_process_may_be_captured():
    """No call before the captured one: whatever is set up once is set up under
    capture."""
    code = """
import torch
from routed_expert_ffn_fp32_b200 import moe
g = torch.Generator(device="cuda").manual_seed(1)
ints = lambda *s: torch.randint(0, 96, s, generator=g, dtype=torch.uint8, device="cuda")
ones = lambda *s: torch.ones(s, device="cuda")
aq, w, u = ints(5, 256), ints(1, 256, 256), ints(1, 256, 256)
ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
x, nq, ns = torch.randn(5, 256, generator=g, device="cuda"), ints(5, 256), ones(5, 2)
out, q, s = ones(5, 256), ints(5, 256), ones(5, 2)

def calls():
    moe.moe_rmsnorm_quant_fp8(x, weight, 1e-6, nq, ns)
    moe.moe_gemm_fp8(aq, sc, w[0], wsc[0], out, ws)
    moe.moe_grouped_swiglu_fp8(aq, sc, w, wsc, u, wsc, None, None, q, s, ws)

weight, sc, wsc = ones(256), ones(5, 2), ones(1, 2, 2)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls()
graph.replay()
torch.cuda.synchronize()
first = [t.clone() for t in (nq, ns, out, q, s)]
calls()
assert moe.moe_get_error(ws) == 0
assert all(torch.equal(a, b) for a, b in zip(first, (nq, ns, out, q, s)))
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("rows,N,dt", [(40, 256, F32), (700, 1600, BF16), (1300, 4096, F16), (3, 256, BF16)])
def test_gemm_output_at_16_byte_alignment(rows, N, dt):
    """Rows of whole 32-byte sectors that start in the middle of one; the values
    around the output are left alone."""
    rng = np.random.default_rng(rows)
    K = 256
    aq, as_ = rows8(rng, rows, K)
    wq, ws_ = mats8(rng, 1, N, K)
    shift = 16 // torch.empty(0, dtype=dt).element_size()
    buf = torch.full((rows * N + 2 * shift,), 7.0, dtype=dt, device="cuda")
    out = buf[shift:shift + rows * N].view(rows, N)
    assert out.data_ptr() % 32 == 16
    ws = make_ws()
    moe.moe_gemm_fp8(dev(aq), dev(as_), dev(wq[0]), dev(ws_[0]), out, ws)
    assert moe.moe_get_error(ws) == 0
    want, mag = F.gemm(F.dequant_rows(aq, as_), F.dequant_mats(wq[0], ws_[0]))
    check_prod(out, want, mag, K, dt)
    assert (buf[:shift] == 7.0).all() and (buf[-shift:] == 7.0).all()


@pytest.mark.parametrize("P,E", [(6, 4), (400, 4)])
def test_empty_buckets_write_nothing(P, E):
    """Pairs that lie in no bucket (a rank that holds none of their experts)."""
    N, K = 256, 128
    ints = torch.full((E, N, K), 0x38, dtype=torch.uint8, device="cuda")
    one = torch.ones(E, 2, 1, device="cuda")
    a, as_ = ints.view(-1, K)[:P].contiguous(), torch.ones(P, 1, device="cuda")
    ent = torch.arange(P, dtype=torch.int32, device="cuda")
    out = torch.full((P, N), 5.0, device="cuda")
    q, s = torch.full((P, N), 0x11, dtype=torch.uint8, device="cuda"), torch.full((P, 2), -1.0, device="cuda")
    ws = make_ws()
    for at in (0, P // 2, P):
        off = torch.full((E + 1,), at, dtype=torch.int32, device="cuda")
        moe.moe_grouped_gemm_fp8(a, as_, ints, one, off, ent, out, ws, scatter=True)
        moe.moe_grouped_swiglu_fp8(a, as_, ints, one, ints, one, off, ent, q, s, ws, a_div=1)
    assert moe.moe_get_error(ws) == 0
    assert (out == 5.0).all() and (q == 0x11).all() and (s == -1.0).all()


def test_swiglu_results_repeat_beside_other_calls():
    """The same call alone, again, and while calls of other shapes run on a second
    stream over the same workspace: the same bits."""
    rng = np.random.default_rng(31)
    T, k, E, I, H = 300, 4, 16, 640, 384
    aq, as_ = rows8(rng, T, H, spread=1)
    mats = [dev(t) for t in (*mats8(rng, E, I, H), *mats8(rng, E, I, H))]
    mats[1] /= 8
    ws = make_ws()
    other = _prefill(5, 40, 512, 512)
    calls = []
    for rows in (T, 2):   # full tiles, and a cluster's
        o, e = routing(rng, rows, k, E)
        args = [dev(aq[:rows]), dev(as_[:rows]), *mats, dev(o), dev(e)]
        q = torch.empty(rows * k, I, dtype=torch.uint8, device="cuda")
        calls.append((args, q, torch.empty(rows * k, 5, device="cuda")))
    first = []
    for args, q, s in calls:
        moe.moe_grouped_swiglu_fp8(*args, q, s, ws, a_div=k)
        torch.cuda.synchronize()
        first.append((q.clone(), s.clone()))
    side = torch.cuda.Stream()
    for _ in range(20):
        for (args, q, s), (q0, s0) in zip(calls, first):
            q.zero_()
            s.zero_()
            with torch.cuda.stream(side):
                moe.moe_gemm_fp8(*other[0], other[1], ws)
            moe.moe_grouped_swiglu_fp8(*args, q, s, ws, a_div=k)
            with torch.cuda.stream(side):
                moe.moe_gemm_fp8(*other[0], other[1], ws)
            torch.cuda.synchronize()
            assert torch.equal(q, q0) and torch.equal(s, s0)
    assert moe.moe_get_error(ws) == 0
