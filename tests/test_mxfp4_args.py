"""Refusals of the MXFP4 and routing entry points, on the CPU: the C ABI's
argument checks with addresses that are never dereferenced (every case fails
before any CUDA call), and the binding's checks of types, shapes and strides."""

import subprocess
import sys

import pytest
import torch

import moe_grouped_gemm_act_b200 as dg

OK, INV, ALN = dg.DG_OK, dg.DG_ERR_INVALID_ARG, dg.DG_ERR_ALIGNMENT
P, ODD = 0x10000, 0x10004
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    return dg.load_library()


def test_quantize_checks(lib):
    q = lambda x=P, dt=0, b=1, m=4, k=64, ld=64, tr=0, qq=P, sf=P: \
        lib.dg_quantize_mxfp4(x, dt, b, m, k, ld, tr, qq, sf, None)
    for bad in (dict(x=None), dict(qq=None), dict(sf=None), dict(dt=2), dict(b=0), dict(m=-1),
                dict(k=0), dict(k=48), dict(k=-32), dict(ld=63), dict(tr=2), dict(tr=1, ld=3),
                dict(tr=1, b=2), dict(m=BIG + 1), dict(k=BIG + 32, ld=BIG + 32),
                dict(b=1 << 30, m=1 << 30, k=1 << 10, ld=1 << 10), dict(ld=BIG + 4)):
        assert q(**bad) == INV, bad
    for bad in (dict(x=ODD), dict(qq=ODD), dict(sf=ODD), dict(ld=66), dict(dt=1, ld=68),
                dict(tr=1, ld=4, x=P + 2)):
        assert q(**bad) == ALN, bad
    assert q(m=0, x=None) == OK


def test_dequantize_checks(lib):
    q = lambda qq=P, sf=P, b=1, m=4, k=64, y=P, dt=0, ld=64: \
        lib.dg_dequantize_mxfp4(qq, sf, b, m, k, y, dt, ld, None)
    for bad in (dict(qq=None), dict(sf=None), dict(y=None), dict(dt=3), dict(b=0), dict(m=-1),
                dict(k=40), dict(ld=32), dict(m=BIG + 1)):
        assert q(**bad) == INV, bad
    for bad in (dict(qq=ODD), dict(sf=ODD), dict(y=ODD), dict(dt=1, ld=68)):
        assert q(**bad) == ALN, bad
    assert q(m=0, y=None) == OK


def test_gemm_checks(lib):
    g = lambda a=P, sa=P, b=P, sb=P, d=P, m=4, n=16, k=64: \
        lib.dg_mxfp4_gemm_nt(a, sa, b, sb, d, m, n, k, None)
    bad_sizes = (dict(m=-1), dict(n=0), dict(n=12), dict(k=0), dict(k=48), dict(m=BIG),
                 dict(n=BIG), dict(k=BIG), dict(m=1 << 30, n=1 << 30))
    for bad in bad_sizes + tuple({x: None} for x in ("a", "sa", "b", "sb", "d")):
        assert g(**bad) == INV, bad
    for x in ("a", "sa", "b", "sb", "d"):
        assert g(**{x: ODD}) == ALN
    assert g(m=0, a=None) == OK

    c = lambda a=P, sa=P, b=P, sb=P, d=P, i=P, m=128, n=16, k=64, gr=2: \
        lib.dg_m_grouped_mxfp4_gemm_nt_contiguous(a, sa, b, sb, d, i, m, n, k, gr, None)
    for bad in bad_sizes[1:6] + (dict(m=100), dict(gr=0), dict(i=None), dict(a=None)):
        assert c(**bad) == INV, bad
    assert c(i=ODD) == ALN and c(m=0) == OK

    k_ = lambda a=P, sa=P, b=P, sb=P, d=P, mm=P, m=10, n=16, k=64, gr=2: \
        lib.dg_m_grouped_mxfp4_gemm_nt_masked(a, sa, b, sb, d, mm, gr, m, n, k, None)
    for bad in bad_sizes[:6] + (dict(m=0), dict(gr=0), dict(gr=1025), dict(mm=None),
                                dict(sb=None)):
        assert k_(**bad) == INV, bad
    assert k_(mm=P + 2) == ALN


def test_route_checks(lib):
    r = lambda x=P, dt=0, t=4, e=8, ld=8, k=2, nm=1, i=P, w=P, c=P, ls=P, n=P, ws=None, nb=0: \
        lib.dg_moe_route(x, dt, t, e, ld, k, nm, None, i, w, c, ls, n, ws, nb, None)
    for bad in (dict(x=None), dict(dt=2), dict(t=-1), dict(t=BIG), dict(e=0), dict(e=1025, ld=1025),
                dict(ld=7), dict(ld=BIG), dict(k=0), dict(k=9), dict(e=64, ld=64, k=33),
                dict(nm=2), dict(i=None), dict(w=None), dict(c=None), dict(ls=None),
                dict(n=None)):
        assert r(**bad) == INV, bad
    for bad in (dict(x=P + 2), dict(dt=1, x=P + 1), dict(i=P + 2), dict(w=P + 1), dict(c=P + 2),
                dict(ls=P + 2), dict(n=P + 2), dict(ws=ODD)):
        assert r(**bad) == ALN, bad
    b = lambda x=P, dt=0, t=4, e=8, ld=8, k=2, nm=1, i=P, w=P, c=P, n=P, dw=P, dl=P, y=P: \
        lib.dg_moe_route_backward(x, dt, t, e, ld, k, nm, i, w, c, n, dw, dl, y, None)
    for bad in (dict(x=None), dict(i=None), dict(w=None), dict(c=None), dict(n=None),
                dict(y=None), dict(k=9), dict(nm=-1), dict(ld=4), dict(dt=5)):
        assert b(**bad) == INV, bad
    for bad in (dict(y=P + 2), dict(dw=P + 1), dict(dl=P + 2), dict(i=P + 2)):
        assert b(**bad) == ALN, bad
    assert b(t=0, x=None) == OK
    assert dg.dg_moe_route_workspace_size(1, 256) == 0
    assert dg.dg_moe_route_workspace_size(100000, 256) >= 148 * (256 * 8 + 4)


def test_binding_refuses_host_tensors():
    x = torch.zeros(32, 64)
    q, sf = torch.zeros(32, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, dtype=torch.int32)
    d = torch.zeros(32, 32, dtype=torch.bfloat16)
    idx = torch.zeros(32, 2, dtype=torch.int32)
    w, c, n = torch.zeros(32, 2), torch.zeros(64, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: dg.dg_quantize_mxfp4(x), lambda: dg.dg_dequantize_mxfp4(q, sf),
                 lambda: dg.dg_mxfp4_gemm_nt(q, sf, q, sf, d),
                 lambda: dg.dg_moe_route(x, 2),
                 lambda: dg.dg_moe_route_backward(x, idx, w, c, n)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_refuses_shapes_and_types():
    x = torch.zeros(32, 64)
    q, sf = torch.zeros(32, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, dtype=torch.int32)
    d = torch.zeros(32, 32, dtype=torch.bfloat16)
    g3 = lambda t: t.unsqueeze(0)
    calls = [
        lambda: dg.dg_quantize_mxfp4(x.half()),
        lambda: dg.dg_quantize_mxfp4(x[:, :40]),                   # K % 32
        lambda: dg.dg_quantize_mxfp4(x.t()),                       # elements of a row apart
        lambda: dg.dg_quantize_mxfp4(x.expand(2, 32, 64), transpose=True),
        lambda: dg.dg_quantize_mxfp4(x.expand(2, 32, 64)),         # batch not contiguous
        lambda: dg.dg_quantize_mxfp4(x[:1].expand(32, 64)),        # rows overlap
        lambda: dg.dg_quantize_mxfp4(x[:, :0]),
        lambda: dg.dg_quantize_mxfp4(x, q=q[:16]),
        lambda: dg.dg_quantize_mxfp4(x, sf=sf.float()),
        lambda: dg.dg_dequantize_mxfp4(q, sf[:, :, :16]),
        lambda: dg.dg_dequantize_mxfp4(q, sf, torch.float16),
        lambda: dg.dg_dequantize_mxfp4(q[:, ::2], sf),
        lambda: dg.dg_mxfp4_gemm_nt(q, sf, q[:, :16].contiguous(), sf, d),
        lambda: dg.dg_mxfp4_gemm_nt(q, sf, q, sf, d.float()),
        lambda: dg.dg_mxfp4_gemm_nt(q, sf, q, sf, d[:, :16]),
        lambda: dg.dg_mxfp4_gemm_nt(q, sf.repeat(2, 1, 1, 1), q, sf, d),
        lambda: dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(q, sf, g3(q), g3(sf), d,
                                                         torch.zeros(32, dtype=torch.int64)),
        lambda: dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(q, sf, q, sf, d,
                                                         torch.zeros(32, dtype=torch.int32)),
        lambda: dg.dg_m_grouped_mxfp4_gemm_nt_masked(g3(q), g3(sf), g3(q), g3(sf), g3(d),
                                                     torch.zeros(2, dtype=torch.int32)),
        lambda: dg.dg_moe_route(x, 0),
        lambda: dg.dg_moe_route(x, 65),
        lambda: dg.dg_moe_route(x.double(), 2),
        lambda: dg.dg_moe_route(x, 2, token_mask=torch.ones(31, dtype=torch.bool)),
        lambda: dg.dg_moe_route(x, 2, token_mask=torch.ones(32)),
        lambda: dg.dg_moe_route(x[0], 2),
        lambda: dg.dg_moe_route_backward(x, torch.zeros(32, 2, dtype=torch.int64),
                                         torch.zeros(32, 2), torch.zeros(64, dtype=torch.int32),
                                         torch.zeros(1, dtype=torch.int32)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")


def test_route_workspace_size_of_refused_experts():
    """No scratch for a number of experts that the call refuses -- and an answer (in a
    child process: a size that never came back would hold up the others)."""
    code = ("import moe_grouped_gemm_act_b200 as dg\n"
            "print([dg.dg_moe_route_workspace_size(t, e) for t in (1, 257, 1 << 40)"
            "       for e in (-1, 0, 1025, (1 << 30) + 1, (1 << 31) - 1)])")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert set(eval(r.stdout)) == {0}
    for e in (1, 1024):
        assert dg.dg_moe_route_workspace_size(257, e) > 0


class _OnStream:
    """What the binding asks of a tensor on cuda:0."""
    device = torch.device("cuda", 0)

    def __init__(self):
        self.used_on = []

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.used_on.append(stream)


def test_tensors_are_marked_as_used_on_a_given_stream(monkeypatch):
    """A temporary passed with stream= is not handed out again while the stream still
    reads it."""
    class Stream:
        device, cuda_stream = torch.device("cuda", 0), 7

    calls = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 3)
    monkeypatch.setattr(dg, "_lib", type("Lib", (), {
        "entry": staticmethod(lambda *a: calls.append(a) or OK)}))
    s, ts = Stream(), [_OnStream(), _OnStream()]
    dg._on_device("entry", (1,), ts, None)
    assert calls == [(1, 3)] and all(t.used_on == [] for t in ts)
    dg._on_device("entry", (2,), ts, s)
    assert calls[1] == (2, 7) and all(t.used_on == [s] for t in ts)
