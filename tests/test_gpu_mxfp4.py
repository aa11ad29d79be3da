"""MXFP4 quantizers and products on the GPU against the float64 oracle.

Tolerances.  Quantizer codes, scale words and read-back values are exact.  A
product's BF16 result o is within 2^-8 |o| of the exact value by its rounding,
plus the FP32 accumulation: K/64 tensor-core steps of 64 products each; a step
aligns its terms and adds to the accumulator with at least 23 bits kept, so each
of the K/64 + 64 roundings of an element loses at most 2^-23 of the sum S of its
terms' magnitudes.
"""

import contextlib
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import moe_grouped_gemm_act_b200 as dg
from moe_grouped_gemm_act_b200 import inputs
from oracle import mxfp4
from tests._helpers import dev

pytestmark = pytest.mark.gpu
SENTINEL = 0x7FC1


def sentinel(*shape):
    return torch.full(shape, SENTINEL, dtype=torch.int16, device="cuda").view(torch.bfloat16)


def untouched(d):
    return bool((d.view(torch.int16) == SENTINEL).all())


def operand(x):
    """(q, sf) on the device and the values in float64 on the device, from the oracle."""
    codes, byte = mxfp4.quantize(x)
    if x.ndim == 3:
        sf = np.stack([mxfp4.scale_words(b) for b in byte])
    else:
        sf = mxfp4.scale_words(byte)
    return dev(mxfp4.pack(codes)), dev(sf), dev(mxfp4.values(codes, byte))


def check(d, a, b, what=""):
    want, s = a @ b.T, a.abs() @ b.abs().T
    steps = a.shape[1] / 64 + 64
    diff = (d.double() - want).abs()
    bound = 2.0 ** -8 * want.abs() + steps * 2.0 ** -23 * s
    assert bool(torch.isfinite(d).all()), what
    assert bool((diff <= bound).all()), f"{what}: {(diff - bound).max()}"


def rnd(shape, seed, outliers=False):
    return inputs.activations(int(np.prod(shape[:-1])), shape[-1], seed, outliers).reshape(shape)


def blocked(byte):
    """mxfp4.scale_words on the device, for large operands: [R, K/32] -> words."""
    r, kg = byte.shape
    full = torch.zeros((-(-r // 128) * 128, -(-kg // 4) * 4), dtype=torch.uint8, device="cuda")
    full[:r, :kg] = byte
    w = full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    return w.view(torch.int32).squeeze(-1)


def random_operand(rows, k, seed):
    """(q, sf) with random codes and scales, and the values in FP32 (exact)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 256, (rows, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    byte = torch.randint(120, 135, (rows, k // 32), generator=gen, device="cuda",
                         dtype=torch.uint8)
    v = dev(mxfp4.VALUES).float()[torch.stack([q & 15, q >> 4], -1).flatten(1).int()]
    v *= torch.exp2(byte.float() - 127).repeat_interleave(32, 1)
    return q, blocked(byte), v


def test_blocked_is_scale_words():
    byte = np.random.default_rng(0).integers(0, 256, (300, 13)).astype(np.uint8)
    assert np.array_equal(blocked(dev(byte)).cpu().numpy(), mxfp4.scale_words(byte))


# ------------------------------------------------------------------ quantizers
def special_rows(m, k, seed):
    x = rnd((m, k), seed, outliers=True)
    g = x.reshape(m, -1, 32)
    g[0, 0] = 0
    g[-1, -1] = -0.0
    g[m // 2, 0] *= np.float32(1e-40)              # subnormal values
    g[m // 2, -1] *= np.float32(1e37)
    g[0, -1] = np.tile(np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6], np.float32), 4)
    g[-1, 0] = np.float32(2.0 ** -126)
    if m > 3:
        g[1, 0, 5] = np.inf
        g[2, 0, 7] = np.nan
        g[3, 0, 1] = -np.inf
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,k", [(1, 32), (3, 64), (5, 96), (33, 160), (128, 128), (129, 1024),
                                 (200, 2112), (64, 7168)])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_is_exact(m, k, dtype, transpose):
    x = torch.from_numpy(special_rows(m, k, seed=m + k)).to(dtype)
    codes, byte = mxfp4.quantize(x.float().numpy())
    src = (x.t() if transpose else x).contiguous().cuda()
    q, sf = dg.dg_quantize_mxfp4(src, transpose=transpose)
    words = mxfp4.scale_words(byte)
    assert np.array_equal(sf.cpu().numpy(), words)
    assert np.array_equal(q.cpu().numpy(), mxfp4.pack(codes))
    want = mxfp4.values(codes, byte)
    for out in (torch.float32, torch.bfloat16):
        y = dg.dg_dequantize_mxfp4(q, sf, out)
        assert y.dtype == out
        # values below the type's smallest subnormal aside, both types are exact
        assert np.array_equal(y.double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_strided(dtype, transpose):
    """A view with a row stride and an offset; odd column counts when transposed."""
    for cols, off, ld in [(96, 8, 136), (97 if transpose else 160, 8, 264), (32, 0, 40)]:
        rows = 64
        base = torch.from_numpy(rnd((rows, ld), 5)).to(dtype).cuda()
        x = base[:, off:off + cols]
        q, sf = dg.dg_quantize_mxfp4(x, transpose=transpose)
        xx = x.float().cpu().numpy()
        codes, byte = mxfp4.quantize(np.ascontiguousarray(xx.T if transpose else xx))
        assert np.array_equal(q.cpu().numpy(), mxfp4.pack(codes))
        assert np.array_equal(sf.cpu().numpy(), mxfp4.scale_words(byte))
    # a base that only has the element's alignment
    base = torch.from_numpy(rnd((64, 41), 6)).to(dtype).cuda()
    if transpose:
        x = base[:, 1:40]
        q, sf = dg.dg_quantize_mxfp4(x, transpose=True)
        codes, byte = mxfp4.quantize(np.ascontiguousarray(x.float().cpu().numpy().T))
        assert np.array_equal(q.cpu().numpy(), mxfp4.pack(codes))
    else:
        with pytest.raises(dg.DGError):
            dg.dg_quantize_mxfp4(base[:, 1:33])


def test_quantize_batch_and_empty():
    x = rnd((3, 70, 96), 7)
    q, sf = dg.dg_quantize_mxfp4(torch.from_numpy(x).cuda())
    assert sf.shape == (3, 1, 1, 32, 4)
    y = dg.dg_dequantize_mxfp4(q, sf, torch.float32).cpu().numpy()
    for b in range(3):
        codes, byte = mxfp4.quantize(x[b])
        assert np.array_equal(q[b].cpu().numpy(), mxfp4.pack(codes))
        assert np.array_equal(sf[b].cpu().numpy(), mxfp4.scale_words(byte))
        assert np.array_equal(y[b], mxfp4.values(codes, byte))
    q, sf = dg.dg_quantize_mxfp4(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 32) and dg.dg_dequantize_mxfp4(q, sf).shape == (0, 64)


@pytest.mark.parametrize("batch,m", [(70000, 2), (1, 600000)])
def test_quantize_past_the_grid(batch, m):
    """More matrices and more rows than a grid has blocks for."""
    k = 32
    x = torch.randn(batch, m, k, device="cuda")
    q, sf = dg.dg_quantize_mxfp4(x)
    y = dg.dg_dequantize_mxfp4(q, sf, torch.float32)
    for i in (0, 1, 65535, 65536, 524287, 524288, batch * m - 1):
        b, r = divmod(i, m)
        if b < batch:
            codes, byte = mxfp4.quantize(x[b, r:r + 1].cpu().numpy())
            assert np.array_equal(q[b, r:r + 1].cpu().numpy(), mxfp4.pack(codes))
            assert np.array_equal(y[b, r:r + 1].cpu().numpy(), mxfp4.values(codes, byte))
    # the worst element is 5 2^e, halfway between 4 and 6: a fifth of it, and so of amax at most
    assert bool(((y - x).abs() <= 0.2001 * x.abs().amax(-1, keepdim=True)).all())


def test_quantize_columns_past_the_grid():
    k, m = 65536 * 256 + 96, 3
    x = torch.randn(k, m, device="cuda").to(torch.bfloat16)
    q, sf = dg.dg_quantize_mxfp4(x, transpose=True)
    for at in (0, 65535 * 256, k - 96):
        codes, byte = mxfp4.quantize(x[at:at + 96].float().cpu().numpy().T.copy())
        assert np.array_equal(q[:, at // 2:at // 2 + 48].cpu().numpy(), mxfp4.pack(codes))
    y = dg.dg_dequantize_mxfp4(q, sf)
    assert bool(((y.t().float() - x.float()).abs() <=
                 0.2001 * x.float().view(-1, 32, m).abs().amax(1).repeat_interleave(32, 0)).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_read_back_into_wider_rows(dtype):
    """The C call's row stride: what lies past K stays."""
    m, k, ld = 37, 96, 136
    codes, byte = mxfp4.quantize(rnd((m, k), 8))
    q, sf = dev(mxfp4.pack(codes)), dev(mxfp4.scale_words(byte))
    y = torch.full((m + 1, ld), -3.0, dtype=dtype, device="cuda")
    rc = dg.load_library().dg_dequantize_mxfp4(
        q.data_ptr(), sf.data_ptr(), 1, m, k, y.data_ptr(),
        dg.DG_DTYPE_F32 if dtype == torch.float32 else dg.DG_DTYPE_BF16, ld,
        torch.cuda.current_stream().cuda_stream)
    assert rc == dg.DG_OK
    assert np.array_equal(y[:m, :k].double().cpu().numpy(), mxfp4.values(codes, byte))
    assert bool((y[:m, k:] == -3).all()) and bool((y[m] == -3).all())


# ------------------------------------------------------------------ dense product
@pytest.mark.parametrize("m,n,k", [
    (1, 8, 32), (1, 2112, 7168), (2, 136, 96), (5, 128, 128), (16, 256, 288), (17, 1000, 544),
    (33, 264, 1056), (64, 7168, 2048), (100, 264, 160), (128, 256, 512), (129, 512, 1056),
    (255, 384, 800), (256, 128, 64), (257, 1048, 1024), (300, 200, 224), (513, 2112, 736),
    (1031, 1544, 2080), (40, 24576, 512), (4096, 2112, 512),
    (2500, 4104, 544), (1024, 7168, 96)])
def test_gemm(m, n, k):
    qa, sa, a = operand(rnd((m, k), m + n, outliers=True))
    qb, sb, b = operand(inputs.weights((n, k), k + 1))
    big = sentinel(m + 2, n)  # rows around D stay as they are
    d = big[1:m + 1]
    assert dg.dg_mxfp4_gemm_nt(qa, sa, qb, sb, d) is d
    check(d, a, b, f"{m}x{n}x{k}")
    assert untouched(big[0]) and untouched(big[-1])
    again = torch.empty_like(d)
    dg.dg_mxfp4_gemm_nt(qa, sa, qb, sb, again)
    assert torch.equal(again.view(torch.int16), d.contiguous().view(torch.int16))
    assert dg.dg_get_device_status() == 0


@pytest.mark.parametrize("m,n,k", [
    (2500, 2008, 3328),     # CTA pairs, a last wave of few tiles
    (2350, 2008, 800),      # the same, half a tile past the rows
    (100, 24576, 4096),     # the same with single CTAs
    (17, 20000, 1312),      # two CTAs per SM
    (700, 7168, 7168), (4096, 4096, 1056)])
def test_gemm_large(m, n, k):
    qa, sa, a = random_operand(m, k, 1)
    qb, sb, b = random_operand(n, k, 2)
    big = sentinel(m + 2, n)
    d = big[1:m + 1]
    for _ in range(2):
        d.view(torch.int16).fill_(SENTINEL)
        dg.dg_mxfp4_gemm_nt(qa, sa, qb, sb, d)
        rows = torch.unique(torch.cat([torch.arange(0, m, 37), torch.tensor([m - 1])])).cuda()
        check(d[rows], a[rows].double(), b.double(), f"{m}x{n}x{k}")
        assert not bool((d.view(torch.int16) == SENTINEL).any())
    assert untouched(big[0]) and untouched(big[-1])
    assert dg.dg_get_device_status() == 0


def test_overlapping_launches_are_ordered():
    """Every kernel starts before the one ahead of it has finished: each must still
    see all that came before it on the stream."""
    m, n, k = 2500, 2008, 3328
    qb, sb, b = random_operand(n, k, 3)
    a32 = [torch.randn(m, k, device="cuda") for _ in range(3)]
    d = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((m, k // 2), dtype=torch.uint8, device="cuda")
    sf = torch.empty((20, 26, 32, 4), dtype=torch.int32, device="cuda")
    want = []
    for x in a32:
        dg.dg_quantize_mxfp4(x, q=q, sf=sf)
        dg.dg_mxfp4_gemm_nt(q, sf, qb, sb, d)
        torch.cuda.synchronize()
        want.append(d.clone())
    for _ in range(5):
        got = []
        for x in a32:
            dg.dg_quantize_mxfp4(x, q=q, sf=sf)
            dg.dg_mxfp4_gemm_nt(q, sf, qb, sb, d)
            got.append(d.clone())
        assert all(torch.equal(u, v) for u, v in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dg_quantize_mxfp4(a32[1], q=q, sf=sf)
        dg.dg_mxfp4_gemm_nt(q, sf, qb, sb, d)
        copy = d.clone()
    for _ in range(3):
        d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(copy, want[1])


def test_quantizer_behind_a_running_product():
    """A quantizer that overwrites a product's operands directly behind it, with nothing
    between the two on the stream: it must not start on them before the product is
    done; nor a product on what the quantizer has not written yet."""
    m, n, k = 2500, 2008, 3328
    qb, sb, b = random_operand(n, k, 3)
    xs = [torch.randn(m, k, device="cuda") for _ in range(4)]
    q = torch.empty((m, k // 2), dtype=torch.uint8, device="cuda")
    sf = torch.empty((20, 26, 32, 4), dtype=torch.int32, device="cuda")
    new = lambda rows: [torch.empty((rows, n), dtype=torch.bfloat16, device="cuda") for _ in xs]
    for rows in (m, 100, 5):      # CTA pairs; K split, for the first rows
        want, got = new(rows), new(rows)
        blocks = -(-rows // 128)
        ops = (q[:rows], sf[:blocks], qb, sb)
        for x, d in zip(xs, want):
            dg.dg_quantize_mxfp4(x, q=q, sf=sf)
            torch.cuda.synchronize()
            dg.dg_mxfp4_gemm_nt(*ops, d)
            torch.cuda.synchronize()
        for _ in range(5):
            for x, d in zip(xs, got):
                dg.dg_quantize_mxfp4(x, q=q, sf=sf)
                dg.dg_mxfp4_gemm_nt(*ops, d)
            assert all(torch.equal(u, v) for u, v in zip(got, want)), rows


def test_offsets_past_32_bits():
    """An input and an output of more than 2^32 bytes (2.3e9 elements each)."""
    m, n, k = 70000, 32768, 64
    qa, sa, a = random_operand(m, k, 4)
    qb, sb, b = random_operand(n, k, 5)
    d = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    dg.dg_mxfp4_gemm_nt(qa, sa, qb, sb, d)
    rows = torch.tensor([0, 1, 32767, 65536, 65537, 69887, 69999], device="cuda")
    check(d[rows], a[rows].double(), b.double())
    q, sf = dg.dg_quantize_mxfp4(d)       # rows of D as an operand
    x = d[rows].float().cpu().numpy()
    codes, byte = mxfp4.quantize(x)
    assert np.array_equal(q[rows].cpu().numpy(), mxfp4.pack(codes))
    y = dg.dg_dequantize_mxfp4(q, sf)
    assert np.array_equal(y[rows].double().cpu().numpy(), mxfp4.values(codes, byte))
    del y
    cut = d[:69984, 32700:]               # the operand's rows are d's last columns
    q, sf = dg.dg_quantize_mxfp4(cut, transpose=True)
    codes, byte = mxfp4.quantize(cut[-96:].float().cpu().numpy().T.copy())
    assert np.array_equal(q[:, -48:].cpu().numpy(), mxfp4.pack(codes))


@pytest.mark.parametrize("m,n,k", [(3, 264, 7168), (64, 256, 4096), (200, 256, 7168),
                                   (600, 768, 1024)])
def test_gemm_exact_integers(m, n, k):
    """Unit scales and whole codes: the FP32 sums are exact, so the result is the
    exact value's one rounding, bit for bit."""
    g = np.random.default_rng(m)
    ca = g.choice([0, 2, 4, 5, 10, 12], (m, k)).astype(np.uint8)
    cb = g.choice([0, 2, 4, 10, 12, 13], (n, k)).astype(np.uint8)
    one = lambda r: dev(mxfp4.scale_words(np.full((r, k // 32), 127, np.uint8)))
    d = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    dg.dg_mxfp4_gemm_nt(dev(mxfp4.pack(ca)), one(m), dev(mxfp4.pack(cb)), one(n), d)
    want = dev(mxfp4.VALUES[ca]) @ dev(mxfp4.VALUES[cb]).T
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(d, want.float().to(torch.bfloat16))


def test_gemm_every_scale_byte_lands_on_its_group():
    """One nonzero product per output, with its own scales: a scale taken from
    another row, group or operand shows."""
    m, n, k = 130, 264, 544
    g = np.random.default_rng(0)
    ea, eb = g.integers(100, 150, (m, k // 32)), g.integers(100, 150, (n, k // 32))
    for grp in (0, 1, 2, 3, 5, 8, 15, 16):
        ca, cb = np.zeros((m, k), np.uint8), np.zeros((n, k), np.uint8)
        ca[:, 32 * grp + 7] = 2  # 1.0
        cb[:, 32 * grp + 7] = 4  # 2.0
        d = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        dg.dg_mxfp4_gemm_nt(dev(mxfp4.pack(ca)), dev(mxfp4.scale_words(ea.astype(np.uint8))),
                            dev(mxfp4.pack(cb)), dev(mxfp4.scale_words(eb.astype(np.uint8))), d)
        want = np.ldexp(2.0, ea[:, grp][:, None] + eb[:, grp][None, :] - 254)
        assert np.array_equal(d.double().cpu().numpy(), want), grp


def test_gemm_nan_group_reaches_its_row_only():
    x, w = rnd((40, 96), 1), inputs.weights((72, 96), 2)
    x[7, 40] = np.nan
    w[11, 3] = np.inf
    qa, sa = dg.dg_quantize_mxfp4(dev(x))
    qb, sb = dg.dg_quantize_mxfp4(dev(w))
    d = torch.empty((40, 72), dtype=torch.bfloat16, device="cuda")
    dg.dg_mxfp4_gemm_nt(qa, sa, qb, sb, d)
    nan = torch.isnan(d).cpu().numpy()
    assert nan[7].all() and nan[:, 11].all()
    nan[7], nan[:, 11] = False, False
    assert not nan.any()


def test_gemm_zero_rows_and_sm_cap():
    qa, sa, a = operand(rnd((70, 512), 3))
    qb, sb, b = operand(inputs.weights((520, 512), 4))
    d0 = torch.empty((0, 520), dtype=torch.bfloat16, device="cuda")
    e, es = dg.dg_quantize_mxfp4(torch.empty(0, 512, device="cuda"))
    dg.dg_mxfp4_gemm_nt(e, es, qb, sb, d0)
    try:
        for cap in (1, 7, 60):
            dg.dg_set_num_sms(cap)
            d = torch.empty((70, 520), dtype=torch.bfloat16, device="cuda")
            dg.dg_mxfp4_gemm_nt(qa, sa, qb, sb, d)
            check(d, a, b, f"cap {cap}")
    finally:
        dg.dg_set_num_sms(0)


@pytest.mark.parametrize("cap", [1, 2, 7, 60, 147])
def test_every_form_under_an_sm_cap(cap):
    """Pairs, tiles past one per SM, K split, and the grouped forms, on fewer SMs."""
    cases = [(2500, 1032, 800), (17, 20000, 96), (5, 256, 2048)]
    ops = [(random_operand(m, k, 1), random_operand(n, k, 2)) for m, n, k in cases]
    counts = np.array([130, 0, 300, 5], np.int32)
    idx, qc, sc, ac, qb, sb, b = contiguous(counts, 392, 160, 31)
    qm, sm, am = operand(rnd((4, 300, 160), 32))
    try:
        dg.dg_set_num_sms(cap)
        for (qa, sa, a), (qw, sw, w) in ops:
            d = torch.empty((len(a), len(w)), dtype=torch.bfloat16, device="cuda")
            dg.dg_mxfp4_gemm_nt(qa, sa, qw, sw, d)
            check(d, a.double(), w.double(), f"cap {cap}")
        dc = sentinel(len(idx), 392)
        dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(qc, sc, qb, sb, dc, dev(idx))
        dm = sentinel(4, 300, 392)
        dg.dg_m_grouped_mxfp4_gemm_nt_masked(qm, sm, qb, sb, dm, dev(counts))
    finally:
        dg.dg_set_num_sms(0)
    assert untouched(dc[torch.from_numpy(idx < 0).cuda()])
    for e, c in enumerate(counts):
        if c:
            rows = torch.from_numpy(np.flatnonzero(idx == e)).cuda()
            check(dc[rows], ac[rows], b[e], f"contiguous, cap {cap}")
            check(dm[e, :c], am[e, :c], b[e], f"masked, cap {cap}")
        assert untouched(dm[e, c:])
    assert dg.dg_get_device_status() == 0


# ------------------------------------------------------------------ grouped products
def contiguous(counts, n, k, seed, extra=0):
    idx = []
    for e, c in enumerate(counts):
        idx += [e] * c + [-1] * (-c % 128)
    idx += [-1] * extra
    idx = np.array(idx, np.int32)
    x = rnd((len(idx), k), seed)
    x[idx < 0] = np.nan  # padding rows may hold anything
    qa, sa, a = operand(x)
    qb, sb, b = operand(inputs.weights((len(counts), n, k), seed + 1))
    return idx, qa, sa, a, qb, sb, b


@pytest.mark.parametrize("counts,n,k,extra", [
    ([128], 128, 64, 0), ([1, 0, 300], 264, 160, 0), ([256, 256], 384, 512, 0),
    ([130, 0, 0, 5, 700], 1000, 544, 256), ([0, 127, 129, 128], 72, 1056, 128),
    ([1000, 900], 2112, 736, 0), ([130, 1, 384, 0, 700, 128, 515], 4872, 288, 128)])
def test_contiguous(counts, n, k, extra):
    idx, qa, sa, a, qb, sb, b = contiguous(counts, n, k, 11, extra)
    d = sentinel(len(idx), n)
    dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(qa, sa, qb, sb, d, dev(idx))
    for e in range(len(counts)):
        rows = torch.from_numpy(np.flatnonzero(idx == e)).cuda()
        if len(rows):
            check(d[rows], a[rows], b[e], f"expert {e}")
    assert untouched(d[torch.from_numpy(idx < 0).cuda()])
    assert dg.dg_get_device_status() == 0


def test_contiguous_many_rows():
    """More 128-row blocks than one launch's table holds, every expert's run cut."""
    rows, n, k, g = 262144 + 640, 16, 32, 3
    idx = torch.arange(rows, device="cuda", dtype=torch.int32) // 128 % (g + 1)
    idx = torch.where(idx == g, -1, idx)
    idx[-384:] = 1
    gen = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randint(0, 256, (rows, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    qb, sb, b = operand(inputs.weights((g, n, k), 4))
    sf = torch.full((rows // 128, 1, 32, 4), 0x7F, device="cuda", dtype=torch.int32)
    a = dev(mxfp4.VALUES)[torch.stack([q & 15, q >> 4], -1).flatten(1).long()]
    d = sentinel(rows, n)
    dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(q, sf, qb, sb, d, idx)
    for e in range(g):
        check(d[idx == e], a[idx == e], b[e], f"expert {e}")
    assert untouched(d[idx < 0])
    assert dg.dg_get_device_status() == 0


def test_contiguous_bad_indices_are_reported():
    idx, qa, sa, a, qb, sb, b = contiguous([256, 200], 136, 96, 13)
    bad = idx.copy()
    bad[5] = 1          # a block of expert 0 with a row of expert 1
    bad[256:384] = 7    # no such expert
    d = sentinel(len(idx), 136)
    dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(qa, sa, qb, sb, d, dev(bad))
    assert dg.dg_get_device_status() == dg.DG_ERR_DEVICE_DATA
    rows = torch.from_numpy(np.flatnonzero(bad == 0)).cuda()
    check(d[rows], a[rows], b[0])
    assert untouched(d[5]) and untouched(d[256:384])
    assert dg.dg_get_device_status() == 0
    d = sentinel(len(idx), 136)
    none = np.full_like(idx, -1)
    dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(qa, sa, qb, sb, d, dev(none))
    assert untouched(d) and dg.dg_get_device_status() == 0


@pytest.mark.parametrize("counts,m_max,n,k", [
    ([1], 1, 8, 32), ([0, 0], 5, 72, 96), ([3, 0, 16, 9], 16, 264, 160),
    ([100, 1, 0, 57, 99], 100, 1000, 544), ([256, 0, 128, 129, 17], 256, 512, 1056),
    ([300, 257, 0, 1], 300, 136, 288), ([700, 0, 129, 513, 256], 700, 392, 544), ([7] * 40, 30, 128, 256),
    (list(range(40)), 40, 520, 96), ([64, 0, 33] * 10, 64, 1032, 160)])
def test_masked(counts, m_max, n, k):
    g = len(counts)
    x = rnd((g, m_max, k), 17)
    for e, c in enumerate(counts):
        x[e, c:] = np.nan
    qa, sa, a = operand(x)
    qb, sb, b = operand(inputs.weights((g, n, k), 18))
    d = sentinel(g, m_max, n)
    dg.dg_m_grouped_mxfp4_gemm_nt_masked(qa, sa, qb, sb, d, dev(np.array(counts, np.int32)))
    for e, c in enumerate(counts):
        if c:
            check(d[e, :c], a[e, :c], b[e], f"expert {e}")
        assert untouched(d[e, c:])
    assert dg.dg_get_device_status() == 0


@pytest.mark.parametrize("m_max,n", [(8, 72), (130, 40), (300, 264)])
def test_masked_1024_experts(m_max, n):
    """The largest table of tiles, most experts empty."""
    g, k = 1024, 96
    gen = torch.Generator(device="cuda").manual_seed(n)
    qa = torch.randint(0, 256, (g, m_max, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    qb = torch.randint(0, 256, (g, n, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    # unit scales, zero bytes for the group past K
    one = lambda r: torch.full((g, -(-r // 128), 1, 32, 4), 0x7F7F7F, dtype=torch.int32, device="cuda")
    val = lambda q: dev(mxfp4.VALUES)[torch.stack([q & 15, q >> 4], -1).flatten(-2).long()]
    counts = np.random.default_rng(n).integers(0, m_max + 1, g).astype(np.int32)
    counts[np.random.default_rng(1).random(g) < 0.6] = 0
    counts[[0, 31, 32, 1023]] = m_max, 0, 1, m_max
    d = sentinel(g, m_max, n)
    dg.dg_m_grouped_mxfp4_gemm_nt_masked(qa, one(m_max), qb, one(n), d, dev(counts))
    live = torch.arange(m_max, device="cuda") < dev(counts)[:, None]
    assert untouched(d[~live])
    for e in np.flatnonzero(counts):
        c = int(counts[e])
        want = val(qa[e, :c]) @ val(qb[e]).T       # whole quarters below 2^24: exact in FP32
        assert torch.equal(d[e, :c], want.float().to(torch.bfloat16)), e
    assert dg.dg_get_device_status() == 0


def test_contiguous_many_experts():
    g, n, k = 300, 40, 64
    counts = np.random.default_rng(7).integers(0, 200, g)
    counts[::3] = 0
    idx, qa, sa, a, qb, sb, b = contiguous(counts.tolist(), n, k, 33)
    d = sentinel(len(idx), n)
    dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(qa, sa, qb, sb, d, dev(idx))
    for e in np.flatnonzero(counts):
        rows = torch.from_numpy(np.flatnonzero(idx == e)).cuda()
        check(d[rows], a[rows], b[e], f"expert {e}")
    assert untouched(d[torch.from_numpy(idx < 0).cuda()])
    assert dg.dg_get_device_status() == 0


def test_masked_bad_counts_and_graph_replay():
    g, m_max, n, k = 4, 40, 264, 160
    qa, sa, a = operand(rnd((g, m_max, k), 19))
    qb, sb, b = operand(inputs.weights((g, n, k), 20))
    mm = dev(np.array([-3, 41, 40, 0], np.int32))
    d = sentinel(g, m_max, n)
    dg.dg_m_grouped_mxfp4_gemm_nt_masked(qa, sa, qb, sb, d, mm)
    assert dg.dg_get_device_status() == dg.DG_ERR_DEVICE_DATA
    assert untouched(d[0]) and untouched(d[3])
    check(d[1], a[1], b[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dg_m_grouped_mxfp4_gemm_nt_masked(qa, sa, qb, sb, d, mm)
    for counts in ([1, 2, 3, 4], [40, 0, 17, 33], [0, 0, 0, 0]):
        mm.copy_(torch.tensor(counts, dtype=torch.int32))
        d.view(torch.int16).fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        for e, c in enumerate(counts):
            if c:
                check(d[e, :c], a[e, :c], b[e])
            assert untouched(d[e, c:])
    assert dg.dg_get_device_status() == 0


def test_streams_side_by_side():
    """Products of different shapes on two streams at once, one of them given by
    argument; quantizers allocate for the stream they run on."""
    s = torch.cuda.Stream()
    x = rnd((60, 2048), 21)
    qa, sa, a = operand(x)
    qb, sb, b = operand(inputs.weights((1544, 2048), 22))
    xd = dev(x)
    d1 = [torch.empty((60, 1544), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    d2 = [torch.empty((60, 1544), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for i in range(4):
        q2, s2 = dg.dg_quantize_mxfp4(xd, stream=s)
        dg.dg_mxfp4_gemm_nt(q2, s2, qb, sb, d2[i], stream=s)
        del q2, s2
        dg.dg_mxfp4_gemm_nt(qa, sa, qb, sb, d1[i])
    torch.cuda.synchronize()
    for d in d1 + d2:
        check(d, a, b)
    assert dg.dg_get_device_status() == 0


@contextlib.contextmanager
def starved(stage):
    """CTA 0 leaves out the loads of its `stage`-th stage; waits run out after 20 ms."""
    names = {"DG_TEST_STARVE_LOAD": str(stage), "DG_TEST_WAIT_LIMIT_US": "20000"}
    os.environ.update(names)
    try:
        yield
    finally:
        for name in names:
            del os.environ[name]


@pytest.mark.parametrize("stage", [0, 2])
@pytest.mark.parametrize("m,n,k", [
    (5, 256, 2048),         # K split over a cluster (one stage for each CTA: stage 0 alone)
    (5, 256, 7168),         # the same, several stages each
    (17, 20000, 1312),      # two CTAs per SM
    (100, 20000, 1056),     # single CTAs
    (2500, 2008, 3328)])    # CTA pairs
def test_lost_load_times_out_and_the_next_product_is_right(m, n, k, stage):
    """Nothing completes a stage that was left out: the bounded waits run out, the CTAs
    leave after the copies that are still in flight, and the call reports it."""
    qa, sa, a = random_operand(m, k, 6)
    qb, sb, b = random_operand(n, k, 7)
    d = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    dg.dg_get_device_status()
    with starved(stage):
        dg.dg_mxfp4_gemm_nt(qa, sa, qb, sb, d)
        torch.cuda.synchronize()
    lost = stage == 0 or k != 2048
    assert dg.dg_get_device_status() == (dg.DG_ERR_TIMEOUT if lost else 0)
    for _ in range(2):
        d.view(torch.int16).fill_(SENTINEL)
        dg.dg_mxfp4_gemm_nt(qa, sa, qb, sb, d)
        check(d, a.double(), b.double())
    assert dg.dg_get_device_status() == 0


@pytest.mark.parametrize("m,n", [(256, 264), (4096, 4872)])
def test_lost_load_of_grouped_products(m, n):
    """The contiguous and the masked form, single CTAs and CTA pairs (masked: also two
    CTAs per SM)."""
    k, g = 1056, 2
    qb, sb = (torch.stack(t) for t in zip(*(random_operand(n, k, s)[:2] for s in (1, 2))))
    b = [random_operand(n, k, s)[2].double() for s in (1, 2)]
    qa, sa, a = random_operand(m, k, 3)
    idx = torch.arange(m, device="cuda", dtype=torch.int32) // (m // 2)
    d = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    with starved(1):
        dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(qa, sa, qb, sb, d, idx)
        torch.cuda.synchronize()
    assert dg.dg_get_device_status() == dg.DG_ERR_TIMEOUT
    dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(qa, sa, qb, sb, d, idx)
    for e in range(g):
        check(d[idx == e], a[idx == e].double(), b[e])
    for m_max, groups in ((40, 64), (100, 2), (256, 2)):   # (64 experts' tiles outnumber the SMs)
        ops = [random_operand(m_max, k, 10 + e) for e in range(groups)]
        qm, sm = (torch.stack(t) for t in zip(*(o[:2] for o in ops)))
        rep = lambda t: t.repeat(groups // g, *[1] * (t.dim() - 1))
        mm = torch.full((groups,), m_max, dtype=torch.int32, device="cuda")
        dm = torch.empty((groups, m_max, n), dtype=torch.bfloat16, device="cuda")
        args = (qm, sm, rep(qb), rep(sb), dm, mm)
        with starved(1):
            dg.dg_m_grouped_mxfp4_gemm_nt_masked(*args)
            torch.cuda.synchronize()
        assert dg.dg_get_device_status() == dg.DG_ERR_TIMEOUT
        dg.dg_m_grouped_mxfp4_gemm_nt_masked(*args)
        for e in range(groups):
            check(dm[e], ops[e][2].double(), b[e % g])
    assert dg.dg_get_device_status() == 0


FIRST_CALLS = """
import threading, torch
import moe_grouped_gemm_act_b200 as dg

gen = torch.Generator(device="cuda").manual_seed(5)
def operand(*shape):
    return dg.dg_quantize_mxfp4(torch.randn(*shape, device="cuda", generator=gen))
# one product for each form: K split, two CTAs per SM, CTA pairs, single CTAs
dense = [(operand(m, k), operand(n, k)) for m, n, k in
         [(5, 256, 2048), (17, 20000, 96), (2500, 2008, 160), (300, 200, 224)]]
masked = [(operand(4, m, 160), operand(4, 264, 160)) for m in (40, 300)]
mm = torch.tensor([1, 0, 40, 17], dtype=torch.int32, device="cuda")
cont = [(operand(m, 160), operand(2, 4872, 160)) for m in (256, 4096)]
new = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()

def run():
    out = []
    for (a, sa), (b, sb) in dense:
        out.append(dg.dg_mxfp4_gemm_nt(a, sa, b, sb, new(len(a), len(b))))
    for (a, sa), (b, sb) in masked:
        out.append(dg.dg_m_grouped_mxfp4_gemm_nt_masked(a, sa, b, sb, new(4, a.shape[1], 264), mm))
    for (a, sa), (b, sb) in cont:
        idx = torch.arange(len(a), device="cuda", dtype=torch.int32) // 128 % 2
        out.append(dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(a, sa, b, sb, new(len(a), 4872), idx))
    return out

start, got = threading.Barrier(4), {}
def work(i):
    with torch.cuda.stream(torch.cuda.Stream()):
        start.wait()
        got[i] = run()
        torch.cuda.current_stream().synchronize()
threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
[t.start() for t in threads]
[t.join() for t in threads]
want = run()
torch.cuda.synchronize()
assert sorted(got) == [0, 1, 2, 3]
assert all(torch.equal(u, v) for g in got.values() for u, v in zip(g, want))
assert dg.dg_get_device_status() == 0
"""


def test_first_calls_from_several_threads():
    """What the library asks of a device once, asked by four threads at once (in a
    process of its own, where no product has run)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_refused_launch_leaves_no_error_behind():
    """A launch that CUDA refuses (the default stream while a stream that waits for it
    is being captured) is that call's error alone."""
    cudart = ctypes.CDLL("libcudart.so.12")   # torch's, already loaded
    lib = dg.load_library()
    x = torch.randn(32, 128, device="cuda")
    q, sf = dg.dg_quantize_mxfp4(x)
    d = torch.empty((32, 32), dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    out = dg.dg_moe_route(x, 4)
    codes = torch.empty((32, 128), dtype=torch.uint8, device="cuda")
    scales = torch.empty((1, 32), device="cuda")
    dlog = dg.dg_moe_route_backward(x, out[0], out[1], out[2], out[4])
    P = lambda t: t.data_ptr()
    calls = {
        "quantize": (lib.dg_quantize_mxfp4, P(x), 0, 1, 32, 128, 128, 0, P(q), P(sf)),
        "dequantize": (lib.dg_dequantize_mxfp4, P(q), P(sf), 1, 32, 128, P(y), 0, 128),
        "product": (lib.dg_mxfp4_gemm_nt, P(q), P(sf), P(q), P(sf), P(d), 32, 32, 128),
        "route": (lib.dg_moe_route, P(x), 0, 32, 128, 128, 4, 1, None, *map(P, out), None, 0),
        "gradient": (lib.dg_moe_route_backward, P(x), 0, 32, 128, 128, 4, 1, P(out[0]), P(out[1]),
                     P(out[2]), P(out[4]), None, None, P(dlog)),
    }
    for name, (fn, *args) in calls.items():
        assert fn(*args, None) == dg.DG_OK, name
    torch.cuda.synchronize()
    for name, (fn, *args) in calls.items():
        stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
        assert cudart.cudaStreamCreate(ctypes.byref(stream)) == 0   # it waits for the default one
        assert cudart.cudaStreamBeginCapture(stream, 2) == 0        # relaxed
        rc = fn(*args, None)
        cudart.cudaStreamEndCapture(stream, ctypes.byref(graph))    # (the capture is void)
        assert cudart.cudaStreamDestroy(stream) == 0
        cudart.cudaGetLastError()
        assert rc == dg.DG_ERR_CUDA, name
        after = lib.dg_quantize_1x128(P(x), 0, 1, 32, 128, 128, P(codes), 128, P(scales), 32, 0,
                                      None)
        assert after == dg.DG_OK, name
        assert fn(*args, None) == dg.DG_OK, name
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == 0


def test_backward_products_of_a_linear_layer():
    """Y = X W^T in MXFP4; its backward products dX = dY W and dW = dY^T X with the
    operands quantized along the axis each product contracts."""
    m, n, k = 192, 264, 160
    x, w, dy = rnd((m, k), 23), inputs.weights((n, k), 24), rnd((m, n), 25)
    dy[:, 256:] = 0
    dyd = torch.zeros(m, 288, device="cuda")      # N padded to the group size
    dyd[:, :n] = dev(dy)
    wt = torch.zeros(288, k, device="cuda")
    wt[:n] = dev(w)
    vals = lambda z: dev(mxfp4.values(*mxfp4.quantize(z)))
    pad = lambda z, r: np.concatenate([z, np.zeros((r - z.shape[0],) + z.shape[1:], z.dtype)])
    q1, s1 = dg.dg_quantize_mxfp4(dyd)
    q2, s2 = dg.dg_quantize_mxfp4(wt, transpose=True)           # W^T [K, N]
    dx = torch.empty((m, k), dtype=torch.bfloat16, device="cuda")
    dg.dg_mxfp4_gemm_nt(q1, s1, q2, s2, dx)
    check(dx, vals(pad(dy.T.copy(), 288).T.copy()), vals(pad(w, 288).T.copy()), "dX")
    q3, s3 = dg.dg_quantize_mxfp4(dev(dy), transpose=True)      # dY^T [N, M]
    q4, s4 = dg.dg_quantize_mxfp4(dev(x), transpose=True)       # X^T [K, M]
    dw = torch.empty((n, k), dtype=torch.bfloat16, device="cuda")
    dg.dg_mxfp4_gemm_nt(q3, s3, q4, s4, dw)
    check(dw, vals(dy.T.copy()), vals(x.T.copy()), "dW")
