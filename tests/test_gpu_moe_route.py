"""MoE routing on the GPU against the float64 oracle.

Tolerances (u = 2^-24, one FP32 rounding): x - max is rounded once, which moves
exp by up to u |x - max|; exp itself, the division and the sum over E experts
(E/32 + 5 additions in a row) add (E/32 + 16) u, all relative.  The loss adds sums
over at most T/16 + 16 + 148 + E positive terms in a row.  Choices and counts are
exact.  A gradient is bounded by the same factor times the sum of its terms'
magnitudes, and BF16 gradients by 2^-8 of the value more.
"""

import threading

import numpy as np
import pytest
import torch

import moe_grouped_gemm_act_b200 as dg
from oracle import mxfp4, route
from tests._helpers import dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def logits(t, e, seed, dtype=torch.float32, closed=False):
    g = np.random.default_rng(seed)
    x = g.normal(0, 2, (t, e)).astype(np.float32)
    if closed:
        x[g.random((t, e)) < 0.5] = -np.inf
        x[g.random(t) < 0.1] = -np.inf
    x = torch.from_numpy(x).to(dtype)
    return x.cuda(), x.double().numpy()


def rel_bound(x, e):
    f = np.where(np.isfinite(x), x, 0)
    return (np.ptp(f, axis=1, keepdims=True) + e / 32 + 16) * U if len(x) else 0


def check_forward(out, x, k, normalize, mask):
    idx, w, counts, loss, n = (v.cpu().numpy() for v in out)
    oi, ow, oc, ol, on, p = route.route(x, k, normalize, mask)
    assert np.array_equal(idx, oi)
    assert np.array_equal(counts, oc) and n[0] == on
    t, e = x.shape
    r = rel_bound(x, e)
    assert (np.abs(w - ow) <= (2 if normalize else 1) * r * ow + 2.0 ** -149).all()
    worst = (float(np.max(r)) if t else 0) + (t / 16 + 180 + e) * U
    assert abs(loss[0] - ol) <= worst * ol
    return oi, ow, oc, on, p


def check_backward(got, x, p, oi, ow, oc, on, dw, dl, normalize, bf16):
    t, e = x.shape
    k = oi.shape[1]
    want = route.route_backward(p, oi, ow, oc, on, dw, dl, normalize)
    c = (abs(dl) * e / (k * max(on, 1) ** 2) * oc) if dl is not None else np.zeros(e)
    a = np.abs(dw) if dw is not None else np.zeros((t, k))
    wdw = (ow * a).sum(1, keepdims=True)
    size = p * (c + (p @ c)[:, None] + (0 if normalize else wdw))
    own = ow * (a + (wdw if normalize else 0))
    for j in range(k):
        rows = np.flatnonzero(oi[:, j] >= 0)
        size[rows, oi[rows, j]] += own[rows, j]
    bound = 4 * rel_bound(x, e) * size + (2.0 ** -8 * np.abs(want) if bf16 else 0) + 2.0 ** -126
    # the oracle's own rounding: it forms p (dp - <p, dp>), whose <p, dp> cancels exactly for
    # normalized weights but only to E + k additions of 2^-53 relative in float64, the terms'
    # magnitudes adding up to at most 2 <w, |dw|> + <p, c>
    bound = bound + (e + k + 8) * 2.0 ** -53 * p * (2 * wdw + (p @ c)[:, None])
    assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (64, 32, 8), (65, 33, 4),
                                   (127, 72, 6), (300, 128, 8), (200, 160, 6), (130, 256, 8),
                                   (70, 257, 32), (90, 512, 16), (40, 1000, 8), (20, 1024, 32),
                                   (3000, 16, 2),
                                   (256, 64, 4), (257, 64, 4)])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_and_gradient(t, e, k, dtype, normalize):
    g = np.random.default_rng(t * e)
    for closed, masked in [(False, False), (True, True)]:
        xd, x = logits(t, e, t + e + k, dtype, closed)
        mask = g.random(t) < 0.8 if masked else None
        out = dg.dg_moe_route(xd, k, normalize, None if mask is None else dev(mask))
        oi, ow, oc, on, p = check_forward(out, x, k, normalize, mask)
        dw, dl = g.normal(size=(t, k)).astype(np.float32), np.float32(0.3)
        for use_w, use_l in [(True, True), (True, False), (False, True), (False, False)]:
            d = dg.dg_moe_route_backward(xd, *(out[i] for i in (0, 1, 2, 4)),
                                         dev(dw) if use_w else None,
                                         dev(np.array([dl])) if use_l else None, normalize)
            assert d.dtype == dtype
            check_backward(d, x, p, oi, ow, oc, on, dw if use_w else None,
                           float(dl) if use_l else None, normalize, dtype == torch.bfloat16)
        if not masked:
            d0 = dg.dg_moe_route(xd, k, normalize)
            assert all(torch.equal(a, b) for a, b in zip(out, d0))  # same bits again
    assert dg.dg_get_device_status() == 0



@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e,k", [(1, 1), (7, 2), (8, 8), (9, 3), (127, 5), (255, 8), (257, 8),
                                 (511, 4), (512, 32), (1000, 6), (1023, 1), (1024, 32)])
def test_joined_blocks(e, k, dtype):
    """Many tokens: the blocks' sums are joined by a second kernel, for every
    split of the E + 1 columns."""
    for t in (257, 2500):
        xd, x = logits(t, e, t + e, dtype, closed=e > 7)
        mask = np.random.default_rng(e).random(t) < 0.9
        a, b = (dg.dg_moe_route(xd, k, True, dev(mask)) for _ in range(2))
        check_forward(a, x, k, True, mask)
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert dg.dg_get_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [160, 256, 500, 1024])
@pytest.mark.parametrize("t", [100, 256, 5000])
def test_last_token_of_a_warp_does_not_route(t, e, dtype):
    """The keys of a warp's last token lie where its probability sums go: left out
    by the mask, by closed experts or by a NaN, it must leave nothing there."""
    xd, x = logits(t, e, t + e, dtype)
    first = t // 2                       # every warp's tokens ascend
    mask = np.arange(t) < first
    check_forward(dg.dg_moe_route(xd, 8, True, dev(mask)), x, 8, True, mask)
    assert dg.dg_get_device_status() == 0
    for hole, status in ((-np.inf, 0), (np.nan, dg.DG_ERR_DEVICE_DATA)):
        xd[first:], x[first:] = hole, hole
        check_forward(dg.dg_moe_route(xd, 8), x, 8, True, None)
        assert dg.dg_get_device_status() == status


def test_ties_signed_zeros_and_lowest_values():
    low = torch.finfo(torch.float32).min
    x = np.array([[0.0, -0.0, 0.0, -0.0, 1.0, 1.0, 1.0, 1.0],
                  [low] * 8,
                  [low, low, 3.0, low, low, low, low, low],
                  [-np.inf, low, -np.inf, low, -np.inf, -np.inf, -np.inf, -np.inf]], np.float32)
    for k in (1, 3, 6, 8):
        for normalize in (True, False):
            out = dg.dg_moe_route(dev(x), k, normalize)
            check_forward(out, x.astype(np.float64), k, normalize, None)
    assert dg.dg_moe_route(dev(x), 6)[0][0].tolist() == [4, 5, 6, 7, 0, 1]


def test_bad_rows_are_left_out_and_reported():
    x = np.random.default_rng(3).normal(size=(70, 24)).astype(np.float32)
    x[4, 3], x[9, 0], x[11, 5] = np.nan, np.inf, np.nan
    mask = np.ones(70, bool)
    mask[11] = False
    xd = dev(x)
    out = dg.dg_moe_route(xd, 4, token_mask=dev(mask))
    assert dg.dg_get_device_status() == dg.DG_ERR_DEVICE_DATA
    oi, ow, oc, on, p = check_forward(out, x.astype(np.float64), 4, True, mask)
    assert on == 67 and (oi[[4, 9, 11]] == -1).all()
    d = dg.dg_moe_route_backward(xd, *(out[i] for i in (0, 1, 2, 4)),
                                 torch.ones(70, 4, device="cuda"), torch.ones(1, device="cuda"))
    assert bool((d[[4, 9, 11]] == 0).all()) and bool(torch.isfinite(d).all())
    # the mask hides the NaN of a padded batch altogether
    mask[[4, 9]] = False
    dg.dg_moe_route(xd, 4, token_mask=dev(mask.astype(np.uint8)))
    assert dg.dg_get_device_status() == 0


@pytest.mark.parametrize("t", [0, 5, 200])
def test_no_token_routes(t):
    x = torch.randn(t, 40, device="cuda")
    idx, w, counts, loss, n = out = dg.dg_moe_route(
        x, 3, token_mask=torch.zeros(t, dtype=torch.bool, device="cuda"))
    assert bool((idx == -1).all()) and bool((w == 0).all()) and bool((counts == 0).all())
    assert float(loss) == 0 and int(n) == 0
    d = dg.dg_moe_route_backward(x, idx, w, counts, n, torch.ones(t, 3, device="cuda"),
                                 torch.ones(1, device="cuda"))
    assert d.shape == (t, 40) and bool((d == 0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_logits(dtype):
    for e, ld, off in [(64, 80, 8), (64, 67, 1), (33, 50, 3), (256, 260, 2)]:
        base = torch.randn(100, ld, device="cuda").to(dtype)
        x = base[:, off:off + e]
        a, b = dg.dg_moe_route(x, 4), dg.dg_moe_route(x.contiguous(), 4)
        assert all(torch.equal(u, v) for u, v in zip(a, b))
        dw = torch.randn(100, 4, device="cuda")
        ga = dg.dg_moe_route_backward(x, a[0], a[1], a[2], a[4], dw)
        gb = dg.dg_moe_route_backward(x.contiguous(), a[0], a[1], a[2], a[4], dw)
        assert torch.equal(ga, gb)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_offsets_past_32_bits(dtype):
    """Rows so far apart that the last ones lie past 2^32 bytes and 2^31 elements."""
    t, e, ld = 40000, 60, 1 << 16
    base = torch.empty((t, ld), dtype=dtype, device="cuda")
    x = base[:, 4:4 + e]
    x.copy_(torch.randn(t, e, device="cuda"))
    a, b = dg.dg_moe_route(x, 4), dg.dg_moe_route(x.contiguous(), 4)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    dw = torch.randn(t, 4, device="cuda")
    ga = dg.dg_moe_route_backward(x, a[0], a[1], a[2], a[4], dw, a[3])
    gb = dg.dg_moe_route_backward(x.contiguous(), a[0], a[1], a[2], a[4], dw, a[3])
    assert torch.equal(ga, gb)


def test_padded_batch_with_garbage():
    """A padded batch: what the left-out tokens hold (NaN, infinities) in logits and in
    the incoming gradient reaches nothing."""
    t, e, k = 700, 72, 6
    xd, x = logits(t, e, 80)
    mask = np.random.default_rng(2).random(t) < 0.7
    md = dev(mask)
    xd[~md] = torch.tensor([np.nan, np.inf, -np.inf] * (e // 3), device="cuda")
    x[~mask] = 0.0
    for normalize in (True, False):
        out = dg.dg_moe_route(xd, k, normalize, md)
        oi, ow, oc, on, p = check_forward(out, x, k, normalize, mask)
        dw = np.random.default_rng(3).normal(size=(t, k)).astype(np.float32)
        dwd = dev(dw)
        dwd[~md] = float("nan")
        d = dg.dg_moe_route_backward(xd, *(out[i] for i in (0, 1, 2, 4)), dwd,
                                     torch.full((1,), 0.5, device="cuda"), normalize)
        check_backward(d, x, p, oi, ow, oc, on, dw, 0.5, normalize, False)
        assert bool((d[~md] == 0).all())
    assert dg.dg_get_device_status() == 0


def test_gradient_against_differences():
    """The kernels' own weights and loss, in differences of the logits."""
    t, e, k = 12, 16, 3
    xd, x = logits(t, e, 5)
    out = dg.dg_moe_route(xd, k)
    dw = torch.randn(t, k, device="cuda")
    dl = torch.full((1,), 2.0, device="cuda")
    d = dg.dg_moe_route_backward(xd, out[0], out[1], out[2], out[4], dw, dl)
    f = lambda z: float((dg.dg_moe_route(z, k)[1].double() * dw.double()).sum() +
                        dl.double() * dg.dg_moe_route(z, k)[3].double())
    h = 2.0 ** -8
    for i, j in [(0, int(out[0][0, 0])), (3, int(out[0][3, 2])), (5, 1), (11, 15)]:
        up, dn = xd.clone(), xd.clone()
        up[i, j] += h
        dn[i, j] -= h
        if not (torch.equal(dg.dg_moe_route(up, k)[0], out[0]) and
                torch.equal(dg.dg_moe_route(dn, k)[0], out[0])):
            continue  # a choice changes here: no derivative
        # FP32 sums of ~t*k terms of size ~1: 2^-20 / 2h, and h^2/6 of the third derivative (< 4)
        assert abs((f(up) - f(dn)) / (2 * h) - float(d[i, j])) < 2.0 ** -11


def test_workspace_and_the_sm_cap():
    """The size holds under every cap, so a cap that changes between the two calls does
    no harm; results under a cap differ in the loss's rounding alone."""
    t, e, k = 4000, 96, 4
    xd, x = logits(t, e, 77)
    size = dg.dg_moe_route_workspace_size(t, e)
    try:
        for cap in (1, 3, 60, 147):
            dg.dg_set_num_sms(cap)
            assert dg.dg_moe_route_workspace_size(t, e) == size
            out = dg.dg_moe_route(xd, k)
            oi, ow, oc, on, p = check_forward(out, x, k, True, None)
            dw = np.random.default_rng(1).normal(size=(t, k)).astype(np.float32)
            d = dg.dg_moe_route_backward(xd, *(out[i] for i in (0, 1, 2, 4)), dev(dw))
            check_backward(d, x, p, oi, ow, oc, on, dw, None, True, False)
    finally:
        dg.dg_set_num_sms(0)
    assert dg.dg_get_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_threads_with_different_experts(dtype):
    """From 513 experts on, one kernel serves every E with shared memory of its own
    size: threads that route different E at once must not take each other's."""
    t, k, lib, rcs = 2, 4, dg.load_library(), {}
    code = {torch.float32: dg.DG_DTYPE_F32, torch.bfloat16: dg.DG_DTYPE_BF16}[dtype]
    cases = {e: logits(t, e, e, dtype)[0] for e in (513, 600, 1024)}
    want = {e: dg.dg_moe_route(x, k) for e, x in cases.items()}
    bufs = {e: [torch.zeros_like(v) for v in want[e]] for e in cases}
    streams = {e: torch.cuda.Stream() for e in cases}
    torch.cuda.synchronize()
    start = threading.Barrier(len(cases))

    def work(e):
        i, w, c, ls, n = (v.data_ptr() for v in bufs[e])
        args = (cases[e].data_ptr(), code, t, e, e, k, 1, None, i, w, c, ls, n, None, 0,
                streams[e].cuda_stream)
        start.wait()
        rcs[e] = {lib.dg_moe_route(*args) for _ in range(50000)}

    threads = [threading.Thread(target=work, args=(e,)) for e in cases]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert rcs == {e: {dg.DG_OK} for e in cases}
    for e in cases:
        assert all(torch.equal(u, v) for u, v in zip(bufs[e], want[e]))


def test_sm_cap_changed_by_another_thread():
    """The scratch that is enough for one SM, while another thread moves the cap: a
    call either has enough or is refused, and nothing behind the scratch is written."""
    t, e, k = 4000, 64, 4
    xd, x = logits(t, e, 78)
    lib = dg.load_library()
    need = 4 * (e + 1) * 8               # four blocks: what one SM takes
    ws = torch.full((4 << 20,), 0x5A, dtype=torch.uint8, device="cuda")
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    idx, w, counts, loss, num = i32(t * k), i32(t * k), i32(e), i32(1), i32(1)
    assert ws.numel() >= dg.dg_moe_route_workspace_size(t, e)
    stop = threading.Event()

    def toggle():
        while not stop.is_set():
            lib.dg_set_num_sms(1)
            lib.dg_set_num_sms(0)

    th = threading.Thread(target=toggle)
    th.start()
    try:
        rcs = {lib.dg_moe_route(xd.data_ptr(), 0, t, e, e, k, 1, None, idx.data_ptr(),
                                w.data_ptr(), counts.data_ptr(), loss.data_ptr(), num.data_ptr(),
                                ws.data_ptr(), need, None) for _ in range(3000)}
    finally:
        stop.set()
        th.join()
        dg.dg_set_num_sms(0)
    torch.cuda.synchronize()
    assert rcs <= {dg.DG_OK, dg.DG_ERR_WORKSPACE}
    assert bool((ws[need:] == 0x5A).all())
    if dg.DG_OK in rcs:
        out = (idx.view(t, k), w.view(torch.float32).view(t, k), counts,
               loss.view(torch.float32), num)
        check_forward(out, x, k, True, None)


def test_graph_replay_and_two_graphs():
    t, e, k = 500, 48, 4
    xs = [logits(t, e, s)[0] for s in (1, 2)]
    dg.dg_moe_route(xs[0], k)
    graphs, outs, ins = [], [], []
    for x in xs:
        buf = x.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = dg.dg_moe_route(buf, k)
            dlog = dg.dg_moe_route_backward(buf, o[0], o[1], o[2], o[4], o[1], o[3])
        graphs.append(g)
        outs.append((*o, dlog))
        ins.append(buf)
    for x in (xs[1], xs[0], logits(t, e, 9)[0]):
        for buf in ins:
            buf.copy_(x)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        o = dg.dg_moe_route(x, k)
        want = (*o, dg.dg_moe_route_backward(x, o[0], o[1], o[2], o[4], o[1], o[3]))
        for got in outs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_on_a_forked_stream():
    """A graph whose calls are given a stream that forks from the captured one."""
    t, e, k = 900, 40, 3
    xs = [logits(t, e, s)[0] for s in (81, 82)]
    side = torch.cuda.Stream()
    dg.dg_moe_route(xs[0], k)
    buf = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        temp = buf[:, :32].contiguous()
        side.wait_stream(torch.cuda.current_stream())
        out = dg.dg_moe_route(buf, k, stream=side)
        dlog = dg.dg_moe_route_backward(buf, out[0], out[1], out[2], out[4], out[1], out[3],
                                        stream=side)
        q, sf = dg.dg_quantize_mxfp4(temp, stream=side)
        del temp                          # (and its memory must not serve the next line)
        other = torch.full((t, 32), float("nan"), device="cuda")
        torch.cuda.current_stream().wait_stream(side)
    for x in (xs[1], xs[0]):
        buf.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        o = dg.dg_moe_route(x, k)
        want = (*o, dg.dg_moe_route_backward(x, o[0], o[1], o[2], o[4], o[1], o[3]),
                *dg.dg_quantize_mxfp4(x[:, :32].contiguous()))
        assert all(torch.equal(a, b) for a, b in zip((*out, dlog, q, sf), want))


def test_two_streams_at_once():
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    xs = [logits(2000, 64, s)[0] for s in (1, 2)]
    want = [dg.dg_moe_route(x, 4) for x in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [dg.dg_moe_route(x, 4, stream=s) for x, s in zip(xs, (s1, s2))]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_temporaries_with_a_given_stream():
    """A mask and logits that are dropped right after the call, while the stream that
    was given has not come to it yet: their memory is not handed out before."""
    t, e, k = 70000, 40, 4
    xd, x = logits(200, e, 79)
    xd = xd.repeat(t // 200, 1)
    keep = torch.arange(t, device="cuda") % 3 > 0
    want = dg.dg_moe_route(xd, k, token_mask=keep)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)             # some 10 ms
        temps = xd + 0.0, keep.clone()
        torch.cuda.current_stream().synchronize()     # (they are ready)
        got = dg.dg_moe_route(temps[0], k, token_mask=temps[1], stream=side)
        del temps
        refill = [torch.full((t,), False, device="cuda"),
                  torch.full((t, e), float("nan"), device="cuda")]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del refill
    assert dg.dg_get_device_status() == 0


def test_a_layer_of_experts():
    """Routing, the experts' MXFP4 products on both layouts, and the weighted sum:
    counts feed masked_m, and the two layouts give the same rows."""
    t, e, k, kk, n = 150, 6, 2, 256, 136
    xd, _ = logits(t, e, 31)
    tok = torch.randn(t, kk, device="cuda")
    w = torch.randn(e, n, kk, device="cuda") * 0.02
    idx, weights, counts, loss, _ = dg.dg_moe_route(xd, k)
    qw, sw = dg.dg_quantize_mxfp4(w)
    flat = idx.flatten().long()
    order = torch.argsort(flat, stable=True)          # pairs by expert, tokens in order
    start = torch.cumsum(counts, 0) - counts
    slot = torch.empty_like(flat)
    slot[order] = torch.arange(t * k, device="cuda") - start[flat[order]]
    token = torch.arange(t, device="cuda").repeat_interleave(k)
    m_max = int(counts.max())
    buf = torch.zeros(e, m_max, kk, device="cuda")
    buf[flat, slot] = tok[token]
    qa, sa = dg.dg_quantize_mxfp4(buf)
    d = torch.zeros(e, m_max, n, dtype=torch.bfloat16, device="cuda")
    dg.dg_m_grouped_mxfp4_gemm_nt_masked(qa, sa, qw, sw, d, counts)
    y1 = (d[flat, slot].float().view(t, k, n) * weights[..., None]).sum(1)
    padded = (counts + 127) // 128 * 128
    base = torch.cumsum(padded, 0) - padded
    row = base[flat] + slot
    total = int(padded.sum())
    m_indices = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    m_indices[row] = idx.flatten()
    rows = torch.zeros(total, kk, device="cuda")
    rows[row] = tok[token]
    qc, sc = dg.dg_quantize_mxfp4(rows)
    dc = torch.zeros(total, n, dtype=torch.bfloat16, device="cuda")
    dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(qc, sc, qw, sw, dc, m_indices)
    assert torch.equal(dc[row], d[flat, slot])
    # against float64 on the quantized values
    va = mxfp4.values(*mxfp4.quantize(tok.cpu().numpy()))
    vw = np.stack([mxfp4.values(*mxfp4.quantize(z)) for z in w.cpu().numpy()])
    want = np.zeros((t, n))
    size = np.zeros((t, n))
    for i in range(t):
        for j in range(k):
            ee, g = int(idx[i, j]), float(weights[i, j])
            want[i] += g * (vw[ee] @ va[i])
            size[i] += g * (np.abs(vw[ee]) @ np.abs(va[i]))
    # BF16 of each expert's row (2^-8) and FP32 sums
    assert (np.abs(y1.double().cpu().numpy() - want) <= (2.0 ** -8) * size + 1e-30).all()
    assert dg.dg_get_device_status() == 0
