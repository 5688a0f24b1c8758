"""GPU parity of the dense operators (residual norm with 8-bit output, dense
product, sampling) against their float64 oracle.

Tolerances (u = 2^-24, half an fp32 step relative to the value):
* codes, tokens: equal. fp32 z: equal.
* scales: a row's fp32 sum of squares has at most 32 + 5 + 16 roundings of
  positive terms in a chain, halved by the square root; rsqrtf is off by two
  steps (4 u), and the mean, eps, product and quotient round: (27 + 4 + 4) u,
  below 40 u = 2.4e-6.
* bf16 outputs: half a step, 2^-8 relative to the value, on top of those.
* products: int32 sums are exact, then three roundings and the bias; bf16
  products are exact in fp32 and summed in K / 16 steps whose alignment may
  truncate by a step (2 u) of at most sum |a w|. Activations have a slope of at
  most 1.13 and are formed to 2e-6 of |v|.
"""
import ctypes
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import quantised_expert_decode_b200 as q
from oracle import dense
from quantised_expert_decode_b200.model import DecodeStack, TokenHead
from synth import configs, gen
from synth.workload import device_layers
from tests.gpu_util import status_word, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8
TORCH = {q.F32: torch.float32, q.BF16: torch.bfloat16}


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


# -------------------------------------------------------------------- norm --
def run_norm(x, y, dtype, gain, group, eps=1e-6, want_norm=True, want_codes=True, z=None):
    T, H = x.shape
    z = z if z is not None else torch.full_like(x, float("nan"))
    norm = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda") if want_norm else None
    codes = torch.full((T + 1, H), 99, dtype=torch.int8, device="cuda") if want_codes else None
    scales = torch.full((T + 1, H // group if group else 1), -7.0, device="cuda") if want_codes else None
    q.qmoe_rmsnorm_residual_q8(x, y, dtype, gain, eps, T, H, group, z, norm, codes, scales)
    torch.cuda.synchronize()
    if want_codes:   # the row behind the last stays as it was
        assert (codes[T] == 99).all() and (scales[T] == -7.0).all()
        codes, scales = codes[:T], scales[:T]
    return z, norm, codes, scales


def check_norm(x, y, dtype, gain, group, eps=1e-6):
    z, norm, codes, scales = run_norm(x, y, dtype, gain, group, eps)
    xs = to_np(x.float())
    ys = None if y is None else to_np(y.float())
    zo, no, co, so = dense.norm_q8(xs, ys, None if gain is None else to_np(gain), eps, group)
    want_z = torch.from_numpy(zo).to(z.dtype)
    assert torch.equal(torch.nan_to_num(z.cpu(), nan=3.0), torch.nan_to_num(want_z, nan=3.0))
    assert np.array_equal(to_np(codes), co)
    s = f64(scales)
    assert np.array_equal(np.isnan(s), np.isnan(so))
    ok = ~np.isnan(so)
    assert (np.abs(s[ok] - so[ok]) <= 40 * U * so[ok] + 1e-45).all()
    n = f64(norm)
    fine = np.isfinite(no) & (np.abs(no) < 3e38)
    assert np.array_equal(np.isnan(n), np.isnan(no))
    assert (np.abs(n[fine] - no[fine]) <= (BF + 41 * U) * np.abs(no[fine]) + 1e-40).all()


@pytest.mark.parametrize("T,H,group", [(1, 16, 0), (1, 2048, 0), (8, 2048, 128), (3, 2064, 0), (5, 256, 32), (37, 1152, 64),
                                       (2, 4224, 32), (9, 5248, 128), (2, 16384, 0), (1, 16384, 64), (401, 128, 128),
                                       (3001, 272, 0)])
@pytest.mark.parametrize("dtype", [q.F32, q.BF16])
def test_norm_matches_oracle(T, H, group, dtype):
    rs = np.random.default_rng(T * 31 + H + group + dtype)
    x = dev((rs.standard_normal((T, H)) * np.exp(rs.standard_normal(H))).astype(np.float32), TORCH[dtype])
    y = dev(rs.standard_normal((T, H)).astype(np.float32), TORCH[dtype])
    gain = dev((1 + 0.3 * rs.standard_normal(H)).astype(np.float32))
    check_norm(x, y, dtype, gain, group)
    check_norm(x, None, dtype, None, group)


def test_codes_at_rounding_borders():
    """Values that are exact multiples of half a step (ties to even) and their fp32 neighbours."""
    H = 512
    base = np.concatenate([np.arange(-127, 128, 0.5), [127.0, -127.0]])[:H].astype(np.float32)
    base[0] = 127.0
    rows = [base, np.nextafter(base, np.float32(np.inf)), np.nextafter(base, np.float32(-np.inf))]
    for r in rows:
        r[0] = 127.0
    x = dev(np.stack(rows + [r * np.float32(0.37) for r in rows]))
    for group in (0, 32):
        check_norm(x, None, q.F32, None, group, eps=0.0)
    # a gain whose products need more than 24 bits
    gain = dev(np.full(H, 1.0 / 3.0, dtype=np.float32))
    check_norm(x, None, q.F32, gain, 0)


@pytest.mark.parametrize("group", [0, 32])
def test_norm_extreme_rows(group):
    """Zero, tiny, huge, infinite and NaN rows, one among ordinary ones."""
    H = 288
    rs = np.random.default_rng(group)
    x = rs.standard_normal((9, H)).astype(np.float32)
    x[0] = 0
    x[1] *= np.float32(1e-42)
    x[2] *= np.float32(1e37)
    x[3] *= np.float32(1e-22)
    x[4, 7] = np.inf
    x[5, 3] = np.nan
    x[6, :32] = 0
    x[7] = np.finfo(np.float32).max
    gain = np.ones(H, dtype=np.float32)
    check_norm(dev(x), None, q.F32, dev(gain), group, eps=0.0)
    check_norm(dev(x), None, q.F32, None, group)
    gain[40] = np.nan
    gain[41] = np.inf
    _, _, codes, scales = run_norm(dev(x[8:]), None, q.F32, dev(gain), group)
    _, _, co, so = dense.norm_q8(x[8:], None, gain, 1e-6, group)
    assert np.array_equal(to_np(codes), co) and np.array_equal(np.isnan(to_np(scales)), np.isnan(so))


@pytest.mark.parametrize("T", [3, 700])
@pytest.mark.parametrize("size,gains", [(1e10, 1e30), (1e-10, 1e-32), (1.0, 1e37), (1e10, None), (1e-11, None)])
@pytest.mark.parametrize("group", [None, 0, 64])
def test_norm_rows_of_gains_far_from_one(T, size, gains, group):
    """z times gain leaves the fp32 range although the normed row does not; with codes and without."""
    H = 576
    rs = np.random.default_rng(T)
    x = (size * rs.standard_normal((T, H))).astype(np.float32)
    # (None: gains of many sizes side by side)
    gain = (np.exp2(rs.integers(-100, 110, H)) if gains is None else gains * (0.5 + rs.random(H))).astype(np.float32)
    xd, gd = dev(x), dev(gain)
    z, no, co, so = dense.norm_q8(x, None, gain, 1e-30, group or 0)
    _, norm, codes, scales = run_norm(xd, None, q.F32, gd, group or 0, eps=1e-30, want_codes=group is not None)
    n = f64(norm)
    # with codes z gain is rounded first: where it lies below 2^-126, to a multiple of 2^-149, so that r times half
    # of that adds to the error
    r = 1 / np.sqrt((x.astype(np.float64) ** 2).mean(1, keepdims=True) + 1e-30)
    tol = (BF + 41 * U) * np.abs(no) + 1e-40 + (0 if group is None else 2.0 ** -150 * r)
    fine = np.abs(no) < 3e38
    assert (np.abs(n - no) <= tol)[fine].all()
    if group is not None:
        assert np.array_equal(to_np(codes), co)
        assert (np.abs(f64(scales) - so) <= 40 * U * so + 1e-45).all()


@pytest.mark.parametrize("T,H,group", [(2500, 272, 0), (2500, 1056, 32), (700, 4112, 0), (700, 5248, 64), (149, 2048, 128)])
@pytest.mark.parametrize("dtype", [q.F32, q.BF16])
def test_norm_many_rows(T, H, group, dtype):
    """CTAs that loop over rows, with rows that are redone or mended among the ordinary ones."""
    rs = np.random.default_rng(T + H)
    x = (2 * rs.standard_normal((T, H))).astype(np.float32)
    half = np.concatenate([np.arange(-127, 128, 0.5), np.zeros(H)])[:H].astype(np.float32)
    half[-1] = 127.0
    x[1::7] = half                               # codes at rounding borders
    x[2::31] *= np.float32(1e-41)
    x[3::31] = 0
    x[4::31, 5] = np.inf
    x[5::31, 6] = np.nan
    y = (rs.standard_normal((T, H)) * (rs.random((T, 1)) < 0.5)).astype(np.float32)
    y[1::7] = 0
    gain = dev((0.2 + rs.random(H)).astype(np.float32))
    xd, yd = dev(x, TORCH[dtype]), dev(y, TORCH[dtype])
    check_norm(xd, yd, dtype, gain, group)
    check_norm(xd, None, dtype, dev(np.full(H, 1.0 / 3.0, dtype=np.float32)), group)
    check_norm(xd, None, dtype, None, group)


@pytest.mark.parametrize("T,H,group", [(1, 16384, 0), (200, 16384, 128), (330, 8192, 0), (160, 14080, 0), (160, 14096, 0)])
def test_norm_wide_rows(T, H, group):
    """Rows in turn in a CTA's shared memory, and rows too wide for that."""
    rs = np.random.default_rng(H + T)
    x, y = (rs.standard_normal((T, H)).astype(np.float32) for _ in range(2))
    x[T // 2] = 0
    y[T // 2] *= np.float32(1e-40)
    x[T - 1, H - 1] = 0.5
    gain = dev((0.2 + rs.random(H)).astype(np.float32))
    check_norm(dev(x), dev(y), q.F32, gain, group)
    check_norm(dev(x, torch.bfloat16), None, q.BF16, gain, group)


def test_norm_in_place_and_partial_outputs():
    rs = np.random.default_rng(3)
    T, H = 6, 640
    x, y = dev(rs.standard_normal((T, H)).astype(np.float32)), dev(rs.standard_normal((T, H)).astype(np.float32))
    want = run_norm(x, y, q.F32, None, 128)
    for alias in ("x", "y"):
        x2, y2 = x.clone(), y.clone()
        got = run_norm(x2, y2, q.F32, None, 128, z=x2 if alias == "x" else y2)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    only_norm = run_norm(x, y, q.F32, None, 0, want_codes=False)
    assert torch.equal(only_norm[1], want[1])
    only_codes = run_norm(x, y, q.F32, None, 128, want_norm=False)
    assert torch.equal(only_codes[2], want[2])
    # the existing fp32 norm on the same rows
    plain = torch.empty_like(x)
    q.qmoe_rmsnorm_residual(x, y, 1e-6, plain, T, H)
    assert (only_norm[1].float() - plain).abs().le(plain.abs() * (BF + 41 * U)).all()


@pytest.mark.parametrize("rows,H,group", [(1, 16, 0), (300, 768, 0), (70, 1024, 64), (5, 16384, 0)])
def test_quantise_rows(rows, H, group):
    rs = np.random.default_rng(rows)
    x = rs.standard_normal((rows, H)).astype(np.float32)
    x[0, :16] = 0
    if rows > 4:
        x[3, 5] = np.inf
        x[4] *= np.float32(1e-40)
    for dtype in (q.F32, q.BF16):
        xd = dev(x, TORCH[dtype])
        codes = torch.empty((rows, H), dtype=torch.int8, device="cuda")
        scales = torch.empty((rows, H // group if group else 1), device="cuda")
        q.qmoe_quantise_rows(xd, dtype, rows, H, group, codes, scales)
        co, so = dense.quantise(f64(xd), 1.0, group)
        assert np.array_equal(to_np(codes), co)
        s = f64(scales)
        assert np.array_equal(np.isnan(s), np.isnan(so))
        ok = ~np.isnan(so)
        assert (np.abs(s - so)[ok] <= 2 * U * so[ok] + 1e-45).all()


# ------------------------------------------------------------------ linear --
def make_linear(M, N, K, in_dtype, out_dtype, bias, residual, seed, lda=None, ldw=None, ldo=None, ldr=None):
    rs = np.random.default_rng(seed)
    step = 8 if in_dtype == q.BF16 else 16
    lda = lda or (K + step - 1) // step * step
    ldw = ldw or (K + step - 1) // step * step
    ldo, ldr = ldo or N, ldr or N
    d = {"M": M, "N": N, "K": K, "in": in_dtype, "od": out_dtype, "lda": lda, "ldw": ldw, "ldo": ldo, "ldr": ldr}
    if in_dtype == q.BF16:
        # columns past K hold NaN: they must not be read into a sum
        a = np.full((M, lda), np.nan, np.float32)
        w = np.full((N, ldw), np.nan, np.float32)
        a[:, :K], w[:, :K] = rs.standard_normal((M, K)), rs.standard_normal((N, K)) / np.sqrt(K)
        d["a"], d["w"] = dev(a, torch.bfloat16), dev(w, torch.bfloat16)
        d["sa"] = d["sw"] = None
    else:
        d["a"], d["w"] = (dev(rs.integers(-128, 128, (r, c), dtype=np.int8)) for r, c in ((M, lda), (N, ldw)))
        d["sa"] = dev(((0.5 + rs.random(M)) / 70).astype(np.float32))
        d["sw"] = dev(((0.5 + rs.random(N)) / (70 * np.sqrt(K))).astype(np.float32))
    d["bias"] = dev(rs.standard_normal(N).astype(np.float32)) if bias else None
    d["res"] = dev(rs.standard_normal((M, ldr)).astype(np.float32), TORCH[out_dtype]) if residual else None
    d["out"] = torch.full((M + 1, ldo), -77.0, dtype=TORCH[out_dtype], device="cuda")
    return d


def call_linear(d, act=q.ACT_NONE, out=None, st=None, stream=None):
    st = status_word() if st is None else st
    q.qmoe_linear(d["a"], d["in"], d["w"], d["M"], d["N"], d["K"], d["sa"], d["sw"], d["bias"], act, d["res"],
                  d["out"] if out is None else out, d["od"], st, d["lda"], d["ldw"], d["ldr"], d["ldo"], stream)
    return st


NAMES = {q.ACT_NONE: "none", q.ACT_RELU: "relu", q.ACT_SILU: "silu", q.ACT_GELU: "gelu"}


def check_linear(d, act):
    M, N, K = d["M"], d["N"], d["K"]
    st = call_linear(d, act)
    torch.cuda.synchronize()
    assert q.qmoe_read_status(st) == 0
    out = f64(d["out"])
    assert (out[M] == -77.0).all() and (out[:, N:] == -77.0).all()      # behind the last row and column
    a, w = f64(d["a"])[:, :K], f64(d["w"])[:, :K]
    res = None if d["res"] is None else f64(d["res"])[:, :N]
    want, pre, mag = dense.linear(a, w, None if d["sa"] is None else f64(d["sa"]), None if d["sw"] is None else f64(d["sw"]),
                                  None if d["bias"] is None else f64(d["bias"]), NAMES[act], res)
    acc = 3 * U * mag if d["in"] == q.I8 else (K / 16 + 2) * 2 * U * mag
    tol = 1.13 * (acc + U * (np.abs(pre) + mag)) + 2e-6 * np.abs(pre) + 2 * U * np.abs(want)
    tol += (BF if d["od"] == q.BF16 else 0) * (np.abs(want) + tol)
    err = np.abs(out[:M, :N] - want)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol).all(), (worst, out[worst], want[worst], tol[worst])


SHAPES = [(1, 1, 1), (1, 128, 64), (1, 2048, 2048), (2, 77, 200), (8, 1000, 512), (16, 130, 1501), (17, 256, 128), (33, 2048, 768),
          (64, 300, 2048), (65, 64, 96), (77, 1000, 1501), (128, 129, 64), (129, 128, 320), (200, 513, 136), (300, 272, 2064),
          (515, 1000, 72), (1030, 520, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("in_dtype", [q.BF16, q.I8])
def test_linear_matches_oracle(M, N, K, in_dtype):
    for n, (od, act, bias, res) in enumerate([(q.F32, q.ACT_NONE, False, False), (q.BF16, q.ACT_SILU, True, True),
                                              (q.F32, q.ACT_GELU, True, False), (q.BF16, q.ACT_RELU, False, True)]):
        check_linear(make_linear(M, N, K, in_dtype, od, bias, res, M + N + K + n), act)


@pytest.mark.parametrize("M", [5, 90, 300])
@pytest.mark.parametrize("in_dtype", [q.BF16, q.I8])
def test_linear_strides(M, in_dtype):
    N, K = 200, 176
    for ldo, ldr in ((208, 216), (201, 203), (256, 200)):
        check_linear(make_linear(M, N, K, in_dtype, q.F32, True, True, M, 192, 208, ldo, ldr), q.ACT_SILU)
        check_linear(make_linear(M, N, K, in_dtype, q.BF16, True, True, M, 192, 208, ldo, ldr), q.ACT_NONE)


@pytest.mark.parametrize("M,N,K", [(700, 1700, 200), (1300, 1000, 72), (2100, 2600, 200), (4097, 1288, 136), (300, 9000, 64)])
@pytest.mark.parametrize("in_dtype", [q.BF16, q.I8])
def test_linear_large_tiles_with_ragged_ends(M, N, K, in_dtype):
    """Tiles of 128 and pairs of 256 rows that end inside the matrix, padded rows, each output type."""
    for n, (od, act, bias, res) in enumerate([(q.F32, q.ACT_SILU, True, True), (q.BF16, q.ACT_NONE, True, True),
                                              (q.BF16, q.ACT_GELU, False, False), (q.F32, q.ACT_NONE, False, False)]):
        check_linear(make_linear(M, N, K, in_dtype, od, bias, res, M + n, ldo=N + 8 * (n % 2) + (-N) % 8, ldr=N + 24 + (-N) % 8), act)


def test_linear_residual_in_place_and_repeatable():
    for M, N in ((3, 256), (40, 256), (200, 256), (700, 1704), (2100, 2600)):
        d = make_linear(M, N, 512, q.BF16, q.F32, False, True, M)
        call_linear(d)
        first = d["out"][:M].clone()
        again = d["res"].clone()
        d2 = dict(d, res=again)
        call_linear(d2, out=again)          # the residual is overwritten by the result
        assert torch.equal(again, first)
        for _ in range(3):
            call_linear(d)
            assert torch.equal(d["out"][:M], first)


def test_linear_infinities_and_nan_stay_in_their_rows():
    d = make_linear(70, 140, 256, q.BF16, q.F32, False, False, 1)
    d["a"][3, 5] = float("nan")
    d["a"][69, 255] = float("inf")
    call_linear(d)
    out = d["out"][:70, :140]
    bad = ~torch.isfinite(out).all(dim=1)
    assert bad.nonzero().flatten().tolist() == [3, 69] and torch.isnan(out[3]).all()


def test_linear_int8_sums_are_exact_at_the_limits():
    """All codes -128 over the longest K: |sum| = 2^30, and one code less in a row."""
    K, M, N = 65536, 3, 70
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    a[1, 7] = 0
    one = torch.ones(128, device="cuda")
    out = torch.empty((M, N), device="cuda")
    st = status_word()
    q.qmoe_linear(a, q.I8, w, M, N, K, one, one, None, q.ACT_NONE, None, out, q.F32, st)
    want = torch.tensor([2.0 ** 30, 2.0 ** 30 - 2.0 ** 14, 2.0 ** 30], device="cuda").unsqueeze(1).expand(M, N)
    assert torch.equal(out, want) and q.qmoe_read_status(st) == 0


def test_linear_full_size_chunk():
    """4096 x 2048 x 768 in 8 bits and 2048 x 2048 x 2048 in bf16, against torch in float64."""
    for M, N, K, dt in ((4096, 2048, 768, q.I8), (2048, 2048, 2048, q.BF16)):
        d = make_linear(M, N, K, dt, q.BF16, True, True, 5)
        st = call_linear(d, q.ACT_SILU)
        a, w = d["a"].double(), d["w"].double()
        if dt == q.I8:
            a, w = a * d["sa"].double()[:, None], w * d["sw"].double()[:, None]
        pre = a @ w.T + d["bias"].double()
        mag = a.abs() @ w.abs().T
        want = pre * torch.sigmoid(pre) + d["res"].double()
        tol = 1.13 * (K / 16 + 4) * 2 * U * mag + 3e-6 * pre.abs()
        tol = tol + BF * (want.abs() + tol)
        assert ((d["out"][:M].double() - want).abs() <= tol).all()
        assert q.qmoe_read_status(st) == 0


def test_linear_that_takes_seconds():
    """The longest rows by 200000 x 200000 results: more than 4e9 SM cycles in one launch, which is no reason for
    a timeout. (1.2e6 products and sums a cycle at most on 148 SMs; both operands are the same matrix.)"""
    M, K = 200_000, 65536
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 125 << 30:
        pytest.skip("needs 106 GB")
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    a = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for i in range(0, M, 20_000):
        a[i:i + 20_000].normal_(generator=g)
    out, st = torch.empty((M, M), dtype=torch.bfloat16, device="cuda"), status_word()
    q.qmoe_linear(a, q.BF16, a, M, M, K, None, None, None, q.ACT_NONE, None, out, q.BF16, st)
    torch.cuda.synchronize()
    assert q.qmoe_read_status(st) == 0
    rows = torch.tensor([0, 77, 128, 100_001, M - 1], device="cuda")
    cols = torch.cat([rows, torch.randint(0, M, (100,), generator=g, device="cuda")])
    x, y = a[rows].double(), a[cols].double()
    want, mag = x @ y.T, x.abs() @ y.abs().T
    tol = (K / 16 + 2) * 2 * U * mag
    tol = tol + BF * (want.abs() + tol)
    assert ((out[rows][:, cols].double() - want).abs() <= tol).all()
    del a, out
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ sample --
def run_sample(logits, dtype=q.F32, ld=0, V=None, temperature=None, top_k=None, top_p=None, min_p=None, u=None, st=None):
    T = logits.shape[0]
    V = V or logits.shape[1]
    f = lambda v, t: None if v is None else dev(np.asarray(v, dtype=t))  # noqa: E731
    token = torch.full((T + 1,), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((T + 1,), -9.0, device="cuda")
    own = st is None
    st = status_word() if own else st
    q.qmoe_sample(logits, dtype, T, V, f(temperature, np.float32), f(top_k, np.int32), f(top_p, np.float32),
                  f(min_p, np.float32), f(u, np.float32), token, prob, st, ld)
    torch.cuda.synchronize()
    assert not own or q.qmoe_read_status(st) == 0
    assert token[T] == -9 and prob[T] == -9.0
    return to_np(token)[:T], f64(prob)[:T]


def check_sample(l, dtype=q.F32, **kw):
    t = dev(np.asarray(l, dtype=np.float32), TORCH[dtype])
    token, prob = run_sample(t, dtype, **kw)
    kw = {k: None if v is None else np.asarray(v, dtype=np.int32 if k == "top_k" else np.float32) for k, v in kw.items()}
    want, p = dense.sample(f64(t), **{k: kw.get(k) for k in ("temperature", "top_k", "top_p", "min_p", "u")})
    assert np.array_equal(token, want), (np.nonzero(token != want)[0], token, want)
    assert (np.abs(prob - p) <= 2 * U * p).all()


def uniforms(rs, T):
    u = rs.random(T).astype(np.float32)
    return np.minimum(u, np.float32(1 - U))


@pytest.mark.parametrize("V", [1, 2, 7, 31, 33, 1000, 4097, 32003, 131072])
@pytest.mark.parametrize("dtype", [q.F32, q.BF16])
def test_sample_matches_oracle(V, dtype):
    rs = np.random.default_rng(V + dtype)
    T = 12
    l = (2.5 * rs.standard_normal((T, V))).astype(np.float32)
    l[rs.random((T, V)) < 0.2] = -np.inf
    l[:, 0] = 1.0                                            # at least one candidate
    u = uniforms(rs, T)
    u[0], u[1] = 0.0, 1 - U
    temp = (0.3 + 1.5 * rs.random(T)).astype(np.float32)
    temp[2] = 0
    check_sample(l, dtype, u=u)
    check_sample(l, dtype, u=u, temperature=temp)
    k = rs.integers(1, max(2, V), T)
    k[:6] = [1, 0, -3, V, V + 5, min(V, 50)]
    check_sample(l, dtype, u=u, temperature=temp, top_k=k)
    p = rs.random(T).astype(np.float32)
    p[:5] = [0.0, 1.0, 1.5, -1.0, 1 - U]
    check_sample(l, dtype, u=u, temperature=temp, top_p=p)
    mp = (rs.random(T) ** 4).astype(np.float32)
    mp[:4] = [0.0, 1.0, -1.0, 1e-30]
    check_sample(l, dtype, u=u, temperature=temp, min_p=mp)
    check_sample(l, dtype, u=u, temperature=temp, top_k=k, top_p=p, min_p=mp)


def test_sample_large_batch():
    rs = np.random.default_rng(11)
    T, V = 300, 5003
    l = (3 * rs.standard_normal((T, V))).astype(np.float32)
    check_sample(l, u=uniforms(rs, T), top_p=np.full(T, 0.9), temperature=0.5 + rs.random(T))
    check_sample(l, u=uniforms(rs, T), top_p=0.3 + 0.7 * rs.random(T), top_k=rs.integers(1, 3000, T))


def test_sample_ties():
    """Equal logits: the lower indices rank first, in the list and past its size."""
    rs = np.random.default_rng(2)
    V = 5000
    l = np.zeros((6, V), dtype=np.float32)
    l[1] = rs.integers(0, 3, V)                              # thousands of equals per value
    l[2] = rs.integers(0, 40, V)
    l[3, 2500:] = 1
    l[4] = np.finfo(np.float32).min                          # a mask of the type's lowest value, everywhere
    l[5] = np.finfo(np.float32).min
    l[5, 4321] = 0.0
    for u in (0.0, 0.3, 0.77, 1 - U):
        us = np.full(6, u)
        check_sample(l, u=us)
        for k in (1, 2, 700, 2600, 4999):
            check_sample(l, u=us, top_k=np.full(6, k))
        for p in (0.1, 0.5, 0.7501, 0.999):
            check_sample(l, u=us, top_p=np.full(6, p))
            check_sample(l, u=us, top_p=np.full(6, p), top_k=np.full(6, 2600))
    bf = np.round(rs.standard_normal((4, 131072)) * 4) / 4   # few distinct bf16 values
    check_sample(bf, q.BF16, u=uniforms(rs, 4), top_p=[0.2, 0.5, 0.9, 0.99])
    check_sample(bf, q.BF16, u=uniforms(rs, 4), top_k=[3, 600, 60000, 131071])


@pytest.mark.parametrize("T,V", [(6, 700), (6, 40000), (170, 3000)])
@pytest.mark.parametrize("dtype", [q.F32, q.BF16])
def test_sample_zeros_of_either_sign_are_equal(T, V, dtype):
    """-0 and 0 are one logit: the lower index ranks first, whichever sign it has."""
    rs = np.random.default_rng(V + dtype)
    l = np.where(rs.random((T, V)) < 0.5, np.float32(0.0), np.float32(-0.0))
    l[rs.random((T, V)) < 0.95] = -40.0
    l[1::3] = np.round(1.2 * rs.standard_normal((len(l[1::3]), V)))       # values -4 .. 4, with zeros of either sign
    l[2::3, V // 3] = 0.25
    u = uniforms(rs, T)
    check_sample(l, dtype, u=u, top_k=rs.integers(2, 30, T))
    check_sample(l, dtype, u=u, top_p=0.2 + 0.6 * rs.random(T))
    check_sample(l, dtype, u=u, top_k=rs.integers(2, 600, T), top_p=0.3 + 0.7 * rs.random(T), min_p=np.full(T, 0.01))
    check_sample(l, dtype, u=u, temperature=np.zeros(T))


def test_sample_empty_rows_and_infinities():
    l = np.full((5, 300), -np.inf, dtype=np.float32)
    l[1, 7] = np.nan
    l[2, [3, 9]] = np.inf
    l[2, 4] = 1e30
    l[3] = np.nan
    l[3, 299] = -5.0
    l[4, [0, 299]] = [np.finfo(np.float32).min, np.finfo(np.float32).max]
    for kw in ({}, dict(top_k=[2] * 5), dict(top_p=[0.7] * 5), dict(min_p=[0.5] * 5), dict(temperature=[0.0] * 5),
               dict(temperature=[1e30] * 5, top_p=[0.9] * 5)):
        check_sample(l, u=[0.6] * 5, **kw)
    token, prob = run_sample(dev(l), u=[0.6] * 5)
    assert token.tolist()[:2] == [-1, -1] and prob[:2].tolist() == [0, 0]


@pytest.mark.parametrize("temp", [1e-30, 1e-3, 30.0, 1e6, 1e15, 1e38])
def test_sample_temperatures(temp):
    """Far from 1: one candidate left, or weights so flat that thresholds sit within a few float64 steps."""
    rs = np.random.default_rng(4)
    l = (3 * rs.standard_normal((5, 3000))).astype(np.float32)
    t = np.full(5, temp, dtype=np.float32)
    check_sample(l, u=uniforms(rs, 5), temperature=t)
    check_sample(l, u=uniforms(rs, 5), temperature=t, top_p=[0.1, 0.4, 0.5, 0.9, 0.99])
    check_sample(l, u=uniforms(rs, 5), temperature=t, min_p=[0.01, 0.5, 0.9, 0.999, 1.0])
    check_sample(l, u=uniforms(rs, 5), temperature=t, top_k=[1, 5, 300, 1500, 2999])


def test_sample_values_over_many_octaves():
    """Bins of equal width separate these slowly; the range is cut again and again."""
    rs = np.random.default_rng(6)
    V = 4000
    l = np.stack([-np.exp2(rs.uniform(-140, 120, V)), np.exp2(rs.uniform(-140, 120, V)) * rs.choice([-1, 1], V),
                  1 + rs.integers(0, 2000, V) * 2.0 ** -23]).astype(np.float32)
    t = np.full(3, 1e36, dtype=np.float32)
    for kw in (dict(top_k=[900, 1800, 1000]), dict(top_p=[0.3, 0.6, 0.5]), dict(top_p=[0.9, 0.99, 0.999])):
        check_sample(l, u=uniforms(rs, 3), temperature=t, **kw)


def test_sample_strides_and_largest_vocabulary():
    rs = np.random.default_rng(8)
    wide = dev((2 * rs.standard_normal((3, 1501))).astype(np.float32))
    for dtype in (q.F32, q.BF16):
        w = wide.to(TORCH[dtype])
        token, _ = run_sample(w, dtype, ld=1501, V=1403, u=[0.2, 0.5, 0.8], top_p=[0.9] * 3)
        want, _ = dense.sample(f64(w)[:, :1403], u=[0.2, 0.5, 0.8], top_p=np.float32([0.9] * 3))
        assert token.tolist() == want.tolist()
    V = 393216
    l = (2.5 * rs.standard_normal((2, V))).astype(np.float32)
    check_sample(l, u=uniforms(rs, 2), top_p=[0.95, 0.2], top_k=[0, 5000])


@pytest.mark.parametrize("V", [131072, 262145, 300001])
@pytest.mark.parametrize("dtype", [q.F32, q.BF16])
def test_sample_large_vocabulary(V, dtype):
    """Few rows of a large vocabulary: masked, with and without each filter, and filters that keep most of it."""
    rs = np.random.default_rng(V + dtype)
    T = 4
    l = (3 * rs.standard_normal((T, V))).astype(np.float32)
    l[1, rs.random(V) < 0.99] = -np.inf
    l[2, rs.random(V) < 0.5] = np.finfo(np.float32).min
    l[3] *= np.float32(0.01)                                 # flat: every filter keeps tens of thousands
    u = uniforms(rs, T)
    for kw in ({}, dict(min_p=[0.05, 0.1, 0.02, 0.97]), dict(top_p=[0.95] * T), dict(top_k=[40, 1000, 5000, 100000]),
               dict(temperature=[0.7, 1.0, 2.5, 0.5], top_k=[50, 0, 2000, 0], top_p=[0.9, 0.5, 0.99, 0.9], min_p=[0, 0.01, 0, 0]),
               dict(temperature=[0.0, 0.0, 1e-3, 0.0])):
        check_sample(l, dtype, u=u, **kw)


def test_sample_unaligned_rows_of_a_large_vocabulary():
    rs = np.random.default_rng(31)
    V, ld = 60001, 60007
    for dtype in (q.F32, q.BF16):
        wide = dev((2 * rs.standard_normal((3, ld))).astype(np.float32), TORCH[dtype])
        u = uniforms(rs, 3)
        for kw in (dict(top_p=np.float32([0.9] * 3)), dict(top_k=[50] * 3, min_p=np.float32([0.02] * 3))):
            token, _ = run_sample(wide, dtype, ld=ld, V=V, u=u, **kw)
            want, _ = dense.sample(f64(wide)[:, :V], u=u, **kw)
            assert token.tolist() == want.tolist()


@pytest.mark.parametrize("dtype", [q.F32, q.BF16])
def test_sample_more_rows_than_sms(dtype):
    """One CTA per row, rows of every kind among them."""
    rs = np.random.default_rng(17 + dtype)
    T, V = 160, 20011
    l = (rs.uniform(0.01, 6, (T, 1)) * rs.standard_normal((T, V))).astype(np.float32)
    l[3] = -np.inf
    l[4, rs.random(V) < 0.999] = -np.inf
    l[5] = 7.0
    l[6] = np.nan
    l[7, 100] = np.inf
    u = uniforms(rs, T)
    check_sample(l, dtype, u=u)
    check_sample(l, dtype, u=u, top_p=rs.random(T))
    check_sample(l, dtype, u=u, top_k=rs.integers(0, V, T), temperature=2 * rs.random(T))
    check_sample(l, dtype, u=u, min_p=rs.random(T) ** 3, top_p=0.5 + 0.5 * rs.random(T), top_k=rs.integers(0, 3000, T))


@pytest.mark.parametrize("T,V", [(1, 8192), (61, 9001), (61, 32003), (3, 16384), (36, 20011), (2, 32768), (15, 33001)])
@pytest.mark.parametrize("dtype", [q.F32, q.BF16])
def test_sample_by_clusters_of_every_size(T, V, dtype):
    """Rows by two, four and eight CTAs with short slices; greedy and masked rows, and each filter."""
    rs = np.random.default_rng(T * 7 + V + dtype)
    l = (2.5 * rs.standard_normal((T, V))).astype(np.float32)
    l[rs.random((T, V)) < 0.3] = -np.inf
    l[:, V // 2] = 1.0                                       # at least one candidate
    if T > 10:
        l[4], l[9] = -np.inf, 3.0                            # nothing, and all the same
        l[7, :V - 5] = -np.inf                               # all of it in the last slice
    temp = (0.5 + rs.random(T)).astype(np.float32)
    temp[::4] = 0
    u = uniforms(rs, T)
    check_sample(l, dtype, u=u, temperature=temp, min_p=0.05 * rs.random(T))
    check_sample(l, dtype, u=u, temperature=temp, top_p=0.5 + 0.5 * rs.random(T))
    check_sample(l, dtype, u=u, top_k=rs.integers(1, 60, T), top_p=np.full(T, 0.9), min_p=np.full(T, 0.01))


@pytest.mark.parametrize("T,V,dtype", [(160, 131072, q.F32), (151, 111601, q.F32), (150, 262145, q.BF16)])
def test_sample_streamed_clusters_in_turns(T, V, dtype):
    """More rows than SMs, too large for L2 together: two CTAs per row, more clusters than run at once."""
    rs = np.random.default_rng(V + T)
    l = (2.5 * rs.standard_normal((T, V), dtype=np.float32)).astype(np.float32)
    l[3] = -np.inf
    l[5, rs.random(V) < 0.99] = -np.inf
    l[6] *= np.float32(0.01)
    temp = (0.5 + rs.random(T)).astype(np.float32)
    temp[::16] = 0
    check_sample(l, dtype, u=uniforms(rs, T), temperature=temp, top_p=0.5 + 0.5 * rs.random(T))
    check_sample(l, dtype, u=uniforms(rs, T), top_k=rs.integers(0, 1500, T), min_p=0.02 * rs.random(T))


def test_sample_is_repeatable():
    rs = np.random.default_rng(9)
    l = dev((2 * rs.standard_normal((7, 60000))).astype(np.float32))
    u = uniforms(rs, 7)
    first = run_sample(l, u=u, top_p=[0.9] * 7)
    for _ in range(5):
        again = run_sample(l, u=u, top_p=[0.9] * 7)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_sample_parameters_out_of_range_are_reported():
    l = dev(np.zeros((2, 100), dtype=np.float32))
    for bad in (dict(temperature=[1.0, -1.0]), dict(temperature=[1.0, np.nan]), dict(temperature=[1.0, np.inf]),
                dict(top_p=[0.5, np.nan]), dict(min_p=[0.5, 1.5]), dict(min_p=[0.5, np.nan])):
        st = status_word()
        token, prob = run_sample(l, u=[0.5, 0.5], st=st, **bad)
        assert token[0] >= 0 and token[1] == -1 and prob[1] == 0, bad
        assert q.qmoe_read_status(st) == 1, bad
    for u in (1.0, -0.1, np.nan):
        st = status_word()
        assert run_sample(l, u=[0.5, u], st=st)[0].tolist() == [50, -1]
        assert q.qmoe_read_status(st) == 1


# ------------------------------------------------------------- other streams --
def test_captured_and_on_another_stream():
    """The three operators on a side stream and replayed from a graph give what eager calls give."""
    rs = np.random.default_rng(12)
    T, H, V = 4, 512, 3001
    x, y = (dev(rs.standard_normal((T, H)).astype(np.float32)) for _ in range(2))
    w = dev((127 * rs.uniform(-1, 1, (V, H))).astype(np.int8))
    sw = dev((rs.random(V) / 1000).astype(np.float32))
    u = dev(uniforms(rs, T))
    p = torch.full((T,), 0.9, device="cuda")
    z, codes = torch.empty_like(x), torch.empty((T, H), dtype=torch.int8, device="cuda")
    scales, logits = torch.empty(T, device="cuda"), torch.empty((T, V), device="cuda")
    token, st = torch.empty(T, dtype=torch.int32, device="cuda"), status_word()

    def step():
        q.qmoe_rmsnorm_residual_q8(x, y, q.F32, None, 1e-6, T, H, 0, z, None, codes, scales)
        q.qmoe_linear(codes, q.I8, w, T, V, H, scales, sw, None, q.ACT_NONE, None, logits, q.F32, st)
        q.qmoe_sample(logits, q.F32, T, V, None, None, p, None, u, token, None, st)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (z, codes, scales, logits, token)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    for how in ("side", "graph"):
        for t in (z, codes, scales, logits, token):
            t.zero_()
        torch.cuda.synchronize()
        if how == "side":
            with torch.cuda.stream(side):
                step()
        else:
            with torch.cuda.graph(graph):
                step()
            graph.replay()
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((z, codes, scales, logits, token), want):
            assert torch.equal(a, b), how
    assert q.qmoe_read_status(st) == 0


def test_two_streams_at_once():
    """No shared scratch: calls that overlap on two streams do not disturb one another."""
    rs = np.random.default_rng(13)
    ds = [make_linear(8, 4096, 1024, q.BF16, q.F32, False, False, s) for s in range(2)]
    ls = [dev((2 * rs.standard_normal((16, 50000))).astype(np.float32)) for _ in range(2)]
    u = dev(uniforms(rs, 16))
    toks = [torch.empty(16, dtype=torch.int32, device="cuda") for _ in range(2)]
    st = status_word()
    for d, l, t in zip(ds, ls, toks):
        call_linear(d, st=st)
        q.qmoe_sample(l, q.F32, 16, 50000, None, None, None, None, u, t, None, st)
    torch.cuda.synchronize()
    want = [(d["out"].clone(), t.clone()) for d, t in zip(ds, toks)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for s, d, l, t in zip(streams, ds, ls, toks):
            with torch.cuda.stream(s):
                call_linear(d, st=st)
                q.qmoe_sample(l, q.F32, 16, 50000, None, None, None, None, u, t, None, st)
    torch.cuda.synchronize()
    for d, t, (o, k) in zip(ds, toks, want):
        assert torch.equal(d["out"], o) and torch.equal(t, k)
    assert q.qmoe_read_status(st) == 0


@pytest.mark.parametrize("op", ["norm", "quantise", "sample"])
def test_two_host_threads_with_calls_of_different_sizes(op):
    """Neither thread's calls are refused for the size of the other's, and each gets its own results. (The C calls
    themselves: between two calls of the binding the threads hardly ever meet.)"""
    rs, lib, p = np.random.default_rng(14), q.lib(), ctypes.c_void_p
    u, st = dev(np.float32([0.4])), status_word()
    keep, calls = [], []
    for n in range(2):
        stream = torch.cuda.Stream()
        size = ((8000, 131072) if op == "sample" else (11008, 16384))[n]
        x = dev(rs.standard_normal((1, size)).astype(np.float32))
        out = torch.zeros((1, size), dtype=torch.int8, device="cuda")
        value = torch.zeros(1, dtype=torch.int32 if op == "sample" else torch.float32, device="cuda")
        px, po, pv, ps = (p(t) for t in (x.data_ptr(), out.data_ptr(), value.data_ptr(), stream.cuda_stream))
        if op == "sample":
            args = (lib.qmoe_sample, px, q.F32, 1, size, 0, None, None, None, None, p(u.data_ptr()), pv, None, p(st.data_ptr()), ps)
        elif op == "quantise":
            args = (lib.qmoe_quantise_rows, px, q.F32, 1, size, 0, po, pv, ps)
        else:
            args = (lib.qmoe_rmsnorm_residual_q8, px, None, q.F32, None, 1e-6, 1, size, 0, None, None, po, pv, ps)
        keep.append((x, stream, out, value))
        calls.append(args)
    torch.cuda.synchronize()
    want = []
    for args, (_, _, out, value) in zip(calls, keep):
        assert args[0](*args[1:]) == 0
        torch.cuda.synchronize()
        want.append((out.clone(), value.clone()))
        out.zero_(), value.zero_()
    torch.cuda.synchronize()
    go, refused = threading.Barrier(2), [0, 0]

    def work(n):
        torch.cuda.set_device(0)
        call, args = calls[n][0], calls[n][1:]
        go.wait(20)
        for i in range(8000):
            refused[n] += call(*args) != 0
            if i % 500 == 0:
                keep[n][1].synchronize()

    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0, 0]
    for (_, _, out, value), (o, v) in zip(keep, want):
        assert torch.equal(out, o) and torch.equal(value, v)
    assert q.qmoe_read_status(st) == 0


ORDER = """
import hashlib, sys, torch
import quantised_expert_decode_b200 as q
g = torch.Generator(device="cuda")
g.manual_seed(3)
st = torch.zeros(1, dtype=torch.int32, device="cuda")
a, w = (torch.randn(r, 2048, generator=g, device="cuda").bfloat16() for r in (5, 2048))
logits, u = torch.randn(18, 131072, generator=g, device="cuda"), torch.rand(18, generator=g, device="cuda")
out, token, prob = torch.empty(5, 2048, device="cuda"), torch.empty(18, dtype=torch.int32, device="cuda"), torch.empty(18, device="cuda")
for op in sys.argv[1]:
    if op == "p":
        q.qmoe_linear(a, q.BF16, w, 5, 2048, 2048, None, None, None, q.ACT_NONE, None, out, q.F32, st)
    else:
        q.qmoe_sample(logits, q.F32, 18, 131072, None, None, u, None, u, token, prob, st)
assert q.qmoe_read_status(st) == 0
print(hashlib.sha256(b"".join(t.cpu().numpy().tobytes() for t in (out, token, prob))).hexdigest())
"""


def test_results_do_not_depend_on_which_operator_ran_first():
    """How a call is spread over the chip is not decided by another operator's earlier calls."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = [subprocess.run([sys.executable, "-c", ORDER, order], cwd=root, capture_output=True, text=True, timeout=300, check=True).stdout
           for order in ("ps", "sp")]
    assert got[0] == got[1] and len(got[0].strip()) == 64


@pytest.mark.parametrize("T,H", [(1, 256), (70, 512), (600, 2048)])
def test_chained_calls_wait_for_one_another(T, H):
    """A call may be set up while the one before it runs: every result read or buffer overwritten by the next
    call, and by other libraries' kernels in between, is as if each had been waited for."""
    rs = np.random.default_rng(T)
    x0 = dev(rs.standard_normal((T, H)).astype(np.float32))
    w = dev((127 * rs.uniform(-1, 1, (H, H))).astype(np.int8))
    sw = dev((rs.random(H) / 3000).astype(np.float32))
    wb = dev((rs.standard_normal((H, H)) / H ** 0.5).astype(np.float32), torch.bfloat16)
    u = dev(uniforms(rs, T))

    def run(wait):
        x, st = x0.clone(), status_word()
        norm = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        codes, scales = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        y, tokens = torch.empty_like(x), []
        for i in range(12):
            token = torch.empty(T, dtype=torch.int32, device="cuda")
            q.qmoe_rmsnorm_residual_q8(x, None, q.F32, None, 1e-6, T, H, 0, None, norm, codes, scales)
            wait()
            q.qmoe_linear(codes, q.I8, w, T, H, H, scales, sw, None, q.ACT_SILU, x, x, q.F32, st)   # residual in place
            wait()
            codes.zero_()
            q.qmoe_linear(norm, q.BF16, wb, T, H, H, None, None, None, q.ACT_NONE, None, y, q.F32, st)
            wait()
            norm.zero_()
            q.qmoe_sample(y, q.F32, T, H, None, None, None, None, u, token, None, st)
            wait()
            y.mul_(0.5)
            q.qmoe_rmsnorm_residual_q8(x, y, q.F32, None, 1e-6, T, H, 0, x, None, codes, scales)
            wait()
            tokens.append(token)
        torch.cuda.synchronize()
        assert q.qmoe_read_status(st) == 0
        return x, torch.stack(tokens)

    want = run(torch.cuda.synchronize)
    for _ in range(3):
        got = run(lambda: None)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("how", ["route", "residual_route", "route_fixed"])
@pytest.mark.parametrize("captured", [False, True])
def test_router_weights_written_by_the_call_before(how, captured):
    """The router reads the weights that a product on the same stream has just written, and its inputs too."""
    rs = np.random.default_rng(21)
    E, H, K, T, k = 256, 512, 65536, 4, 8
    w = dev(rs.standard_normal((H, K), dtype=np.float32), torch.bfloat16)
    a = dev(rs.standard_normal((E, K), dtype=np.float32) / 256, torch.bfloat16)
    sides = [a, -a, a.flip(0).contiguous()]
    x, y = (dev(rs.standard_normal((T, H)).astype(np.float32)) for _ in range(2))
    ws, st = torch.zeros(q.qmoe_route_workspace_bytes(T, E), dtype=torch.uint8, device="cuda"), status_word()
    Wr, x_out = torch.empty((E, H), device="cuda"), torch.empty_like(x)

    def run(wait):
        got = []
        for i in range(9):
            idx, gate = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
            q.qmoe_linear(sides[i % 3], q.BF16, w, E, H, K, None, None, None, q.ACT_NONE, None, Wr, q.F32, st)
            wait()
            if how == "route":
                q.qmoe_route(Wr, None, x, q.F32, T, H, E, k, idx, gate, ws, st)
            elif how == "route_fixed":
                q.qmoe_route_fixed(Wr, None, x, T, H, E, k, idx, gate, st)
            else:
                q.qmoe_residual_route(x, y, 1e-6, x_out, Wr, None, T, H, E, k, idx, gate, ws, st)
            wait()
            got.append((idx, gate))
        return got

    want = run(torch.cuda.synchronize)
    assert not torch.equal(want[0][0], want[1][0])
    for _ in range(3):
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = run(lambda: None)
            graph.replay()
        else:
            got = run(lambda: None)
        torch.cuda.synchronize()
        for (i, g), (wi, wg) in zip(got, want):
            assert torch.equal(i, wi) and torch.equal(g, wg)
    assert q.qmoe_read_status(st) == 0


# ---------------------------------------------------- behind a layer stack --
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("T", [1, 8])
def test_token_head_behind_a_stack(bits, T):
    """Stack -> norm -> head product -> token: the same eagerly, on a side stream and captured, and the oracle's."""
    cfg = configs.get(0).with_(L=2, T=T, residual=True)
    layers, routers, _ = device_layers(0, cfg, 2)
    stack = DecodeStack(layers, routers, None, T, cfg.k, cfg.eps)
    rs = np.random.default_rng(40 + bits + T)
    V = 5003
    weight = dev(rs.standard_normal((V, cfg.H)).astype(np.float32), torch.bfloat16 if bits == 16 else None)
    gain, bias = dev((0.5 + rs.random(cfg.H)).astype(np.float32)), dev(rs.standard_normal(V).astype(np.float32))
    head = TokenHead(weight, T, gain, bias, bits=bits)
    u = uniforms(rs, T)
    kw = dict(temperature=np.full(T, 4.0), top_k=np.full(T, 400), top_p=np.full(T, 0.9), min_p=np.full(T, 0.001))
    kw = {k: v.astype(np.int32 if k == "top_k" else np.float32) for k, v in kw.items()}
    ud, kd = dev(u), {k: dev(v) for k, v in kw.items()}
    stack.x_in.copy_(dev(gen.tokens(0, cfg, 0)))
    stack.decode()
    head.step(stack.x_out, ud, **kd)
    torch.cuda.synchronize()
    assert stack.status() == 0 and head.status() == 0
    x = to_np(stack.x_out)
    _, no, co, so = dense.norm_q8(x, None, to_np(gain), 1e-6, 0)
    if bits == 8:
        wc, ws = dense.quantise(f64(weight), 1.0, 0)
        assert np.array_equal(to_np(head.weight), wc) and np.array_equal(to_np(head.codes), co)
        want, pre, mag = dense.linear(co, wc, so[:, 0], ws[:, 0], f64(bias))
        tol = (3 + 40 + 2) * U * mag + 2 * U * (np.abs(pre) + mag)
    else:
        want, pre, mag = dense.linear(no, f64(weight), bias=f64(bias))
        tol = (BF + 41 * U) * mag + (cfg.H / 16 + 2) * 2 * U * mag + 2 * U * (np.abs(pre) + mag)
    logits = f64(head.logits)
    assert (np.abs(logits - want) <= tol).all()
    token, prob = dense.sample(logits, u=u, **kw)
    assert np.array_equal(to_np(head.token), token) and (np.abs(f64(head.prob) - prob) <= 2 * U * prob).all()

    keep = [t.clone() for t in (head.logits, head.token, head.prob)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    for how in ("side", "graph"):
        for t in (head.logits, head.token, head.prob):
            t.zero_()
        torch.cuda.synchronize()
        if how == "side":
            stack.decode(side)
            head.step(stack.x_out, ud, stream=side, **kd)
        else:
            with torch.cuda.graph(graph):
                head.step(stack.x_out, ud, **kd)
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((head.logits, head.token, head.prob), keep):
            assert torch.equal(a, b), how
    stack.close()


@pytest.mark.parametrize("bits,dtype", [(8, torch.float32), (16, torch.float32), (16, torch.bfloat16)])
@pytest.mark.parametrize("handle", ["stream", "address", "default"])
def test_token_head_built_on_another_stream(bits, dtype, handle):
    """The current stream is busy, with the weights' own values among its work; the head is built and used on
    another without a wait between, and the weights are dropped at once."""
    rs = np.random.default_rng(60 + bits)
    V, H, T = 5003, 512, 3
    values = rs.standard_normal((V, H)).astype(np.float32)
    x, u = dev(rs.standard_normal((T, H)).astype(np.float32)), dev(uniforms(rs, T))
    want = TokenHead(dev(values, dtype), T, bits=bits)
    want.step(x, u)
    torch.cuda.synchronize()
    source = dev(values, dtype)
    side = torch.cuda.default_stream() if handle == "default" else torch.cuda.Stream()
    busy = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(busy):
            weight = torch.full_like(source, 3.0)
            torch.cuda._sleep(20_000_000)
            weight.copy_(source)
            head = TokenHead(weight, T, bits=bits, stream=side.cuda_stream if handle == "address" else side)
            del weight
            junk = [torch.full_like(source, 7.0) for _ in range(3)]   # takes the weights' memory over
        head.step(x, u, stream=side)
        torch.cuda.synchronize()
        assert head.status() == 0
        assert torch.equal(head.logits, want.logits) and torch.equal(head.token, want.token)
        del head, junk


def test_token_head_refusals():
    w = torch.zeros((100, 64), device="cuda")
    for bad in (dict(weight=w[0]), dict(weight=w.double()), dict(weight=w, bits=4), dict(weight=w, T=0),
                dict(weight=w[:, :40])):
        with pytest.raises(q.QmoeError):
            TokenHead(**{"T": 1, **bad})
    head, u = TokenHead(w, 2), torch.zeros(2, device="cuda")
    for x, uu in ((torch.zeros((1, 64), device="cuda"), u), (torch.zeros((2, 64), device="cuda").double(), u),
                  (torch.zeros((2, 64), device="cuda"), u[:0])):
        with pytest.raises(q.QmoeError):
            head.step(x, uu)
    with pytest.raises(q.QmoeError):
        TokenHead(w, 2, gain=torch.ones(32, device="cuda")).step(torch.zeros((2, 64), device="cuda"), u)
    assert head.step(torch.zeros((2, 64), device="cuda"), u).tolist() == [0, 0] and head.status() == 0
