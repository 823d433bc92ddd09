"""Host-side checks of the prompt-stage operators (no GPU): argument refusals
of the C ABI, the binding's refusals, and the 64-bit reference the GPU tests
use against the independent oracle."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from paged_gqa_decode_07_b200 import build as pgd_build
from tests import prefill_ref
from workloads import make_case, multi_query

OK, INVALID, UNSUPPORTED = 0, 1, 2
A = ctypes.c_void_p(0x10000)       # never dereferenced: every check fails on the host
MIS = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    pgd_build.build()
    import paged_gqa_decode_07_b200 as pgd
    return pgd.load_library()


def prefill(lib, **kw):
    a = dict(q=A, qs=1024, k=A, ks=256, v=A, vs=256, cu=A, B=2, T=64, ml=0, W=0, Hq=8, Hkv=2,
             D=128, scale=0.1, out=A, lse=None, ws=None, wsb=0, ns=0)
    a.update(kw)
    return lib.pgd_prefill_attention(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["cu"],
                                     a["B"], a["T"], a["ml"], a["W"], a["Hq"], a["Hkv"], a["D"],
                                     a["scale"], a["out"], a["lse"], a["ws"], a["wsb"], a["ns"],
                                     None)


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=6, Hkv=4), INVALID), (dict(Hq=34, Hkv=2, qs=4352), UNSUPPORTED),
    (dict(D=64), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(Hkv=0), INVALID),
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(W=-1), INVALID), (dict(ml=-1), INVALID),
    (dict(ns=-1), INVALID), (dict(ns=1025), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(cu=None), INVALID), (dict(out=None), INVALID),
    (dict(q=MIS), INVALID), (dict(k=MIS), INVALID), (dict(v=MIS), INVALID),
    (dict(out=MIS), INVALID), (dict(lse=MIS), INVALID), (dict(cu=MIS), INVALID),
    (dict(qs=1016), INVALID),              # rows of 1024 elements overlap
    (dict(ks=260), INVALID),               # not a multiple of 8 elements
    (dict(vs=0), INVALID), (dict(qs=1 << 40), INVALID),
    (dict(ws=None, wsb=64), INVALID), (dict(ws=MIS, wsb=64), INVALID),
    (dict(B=0, q=None), OK), (dict(T=0, q=None), OK),
])
def test_prefill_refusals(lib, kw, status):
    assert prefill(lib, **kw) == status


def paged(lib, **kw):
    a = dict(q=A, qs=1024, k=A, v=A, bt=A, mb=8, cl=A, cu=A, B=2, T=64, mq=0, mc=0, W=0, Hq=8,
             Hkv=2, D=128, bs=16, nb=16, scale=0.1, dt=0, ks=None, vs=None, out=A, lse=None,
             ws=None, wsb=0, ns=0)
    a.update(kw)
    return lib.pgd_paged_prefill_attention(
        a["q"], a["qs"], a["k"], a["v"], a["bt"], a["mb"], a["cl"], a["cu"], a["B"], a["T"],
        a["mq"], a["mc"], a["W"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["nb"], a["scale"],
        a["dt"], a["ks"], a["vs"], a["out"], a["lse"], a["ws"], a["wsb"], a["ns"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=6, Hkv=4), INVALID), (dict(Hq=34, Hkv=2, qs=4352), UNSUPPORTED),
    (dict(D=64), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(bs=128), UNSUPPORTED),
    (dict(dt=1), INVALID),                 # FP8 without scales
    (dict(dt=1, D=256, qs=2048, ks=A, vs=A), UNSUPPORTED), (dict(dt=7), INVALID),
    (dict(nb=0), INVALID), (dict(mb=0), INVALID), (dict(mc=-1), INVALID),
    (dict(nb=1 << 30, Hkv=2), UNSUPPORTED), (dict(mb=1 << 28), UNSUPPORTED),
    (dict(bt=None), INVALID), (dict(cl=None), INVALID), (dict(cu=None), INVALID),
    (dict(k=MIS), INVALID), (dict(v=MIS), INVALID), (dict(bt=MIS), INVALID),
    (dict(dt=1, ks=MIS, vs=A), INVALID), (dict(qs=1020), INVALID), (dict(ns=-1), INVALID),
    (dict(B=0, q=None), OK), (dict(T=0, out=None), OK),
])
def test_paged_prefill_refusals(lib, kw, status):
    assert paged(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(D=64), UNSUPPORTED), (dict(h=0), INVALID),
    (dict(h=65537), UNSUPPORTED), (dict(acc=2), INVALID), (dict(k=None), INVALID),
    (dict(k=MIS), INVALID), (dict(ks=None), INVALID), (dict(vs=MIS), INVALID),
])
def test_quant_scales_refusals(lib, kw, status):
    a = dict(k=A, v=A, n=4, h=2, D=128, acc=0, ks=A, vs=A)
    a.update(kw)
    assert lib.pgd_kv_quant_scales(a["k"], a["v"], a["n"], a["h"], a["D"], a["acc"], a["ks"],
                                   a["vs"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(D=64), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
    (dict(h=0), INVALID), (dict(h=65537), UNSUPPORTED), (dict(nb=0), INVALID),
    (dict(dt=3), INVALID), (dict(dt=1), INVALID), (dict(k=MIS), INVALID),
    (dict(ko=MIS), INVALID), (dict(sl=ctypes.c_void_p(0x10004)), INVALID),
    (dict(dt=1, ks=A, vs=MIS), INVALID), (dict(n=0, k=None), OK),
])
def test_gather_refusals(lib, kw, status):
    a = dict(k=A, v=A, sl=A, n=4, ko=A, vo=A, h=2, D=128, bs=16, nb=4, dt=0, ks=None, vs=None)
    a.update(kw)
    assert lib.pgd_kv_gather(a["k"], a["v"], a["sl"], a["n"], a["ko"], a["vo"], a["h"], a["D"],
                             a["bs"], a["nb"], a["dt"], a["ks"], a["vs"], None) == status


def test_binding_refuses_cpu_tensors():
    import paged_gqa_decode_07_b200 as pgd
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        pgd.prefill_attention(q, k, k, cu, 8, 2, 128, 0.1)
    with pytest.raises(ValueError):
        pgd.kv_quant_scales(k, k)
    with pytest.raises(TypeError):
        pgd.prefill_attention([1], k, k, cu, 8, 2, 128, 0.1)


class _OnDevice:
    """The attributes of a tensor on a CUDA device that the binding reads."""

    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    from paged_gqa_decode_07_b200 import _binding
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    _binding._same_device("op", _OnDevice(0), None, _OnDevice(0))
    with pytest.raises(ValueError):
        _binding._same_device("op", _OnDevice(0), _OnDevice(1))


def _bf16(bits):
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16)


@pytest.mark.parametrize("dt,window,L", [("bf16", 0, 3), ("bf16", 5, 4), ("e4m3", 0, 2),
                                         ("e4m3", 33, 5)])
def test_reference_agrees_with_the_oracle(dt, window, L):
    """Paged rows with L queries per sequence: the oracle's multi-token decode."""
    w = make_case([1, 3, 17, 40, 0, 64], 6, 2, 128, 16, dt, seed=5)
    qm = multi_query(w, L, seed=2)
    want, want_lse = oracle.paged_decode_multi(qm, w.k_cache, w.v_cache, w.block_table,
                                               w.context_lens, 2, w.scale, window=window,
                                               k_scale=w.k_scale, v_scale=w.v_scale)
    if dt == "bf16":
        kc, vc, ks, vs = _bf16(w.k_cache), _bf16(w.v_cache), None, None
    else:
        kc, vc = (torch.from_numpy(c).view(torch.float8_e4m3fn) for c in (w.k_cache, w.v_cache))
        ks, vs = torch.from_numpy(w.k_scale), torch.from_numpy(w.v_scale)
    B = w.num_seqs
    out, lse, _, _ = prefill_ref.paged(_bf16(qm).reshape(B * L, 6, 128), kc, vc,
                                       torch.from_numpy(w.block_table), w.context_lens,
                                       [L * i for i in range(B + 1)], window, w.scale, ks, vs)
    np.testing.assert_allclose(out.numpy(), want.reshape(B * L, 6, 128), rtol=1e-9, atol=1e-11)
    np.testing.assert_allclose(lse.numpy(), want_lse.reshape(B * L, 6), rtol=1e-9, atol=1e-11)


def test_packed_reference_is_causal_softmax():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((9, h, 128), generator=g, dtype=torch.float64) for h in (4, 2, 2))
    out, lse, _, _ = prefill_ref.packed(q, k, v, [0, 4, 4, 9], 0, 0.3)
    for a, b in ((0, 4), (4, 9)):
        kk, vv = (x[a:b].repeat_interleave(2, 1).transpose(0, 1) for x in (k, v))
        want = torch.nn.functional.scaled_dot_product_attention(
            q[a:b].transpose(0, 1), kk, vv, is_causal=True, scale=0.3)
        torch.testing.assert_close(out[a:b].transpose(0, 1), want, rtol=1e-10, atol=1e-12)


class _Sizes:
    """pgd_prefill_workspace_bytes of a device that cannot be asked at first."""

    def __init__(self, answer):
        self.answer, self.fails, self.asked = answer, True, 0

    def pgd_prefill_workspace_bytes(self, seqs, tokens, keys, window, hq, hkv, d, ctas):
        self.asked += 1
        if self.fails:
            return 0
        return 4096 if ctas == 2 else self.answer


@pytest.mark.parametrize("answer", [1 << 20, 0], ids=["cut", "whole"])
def test_a_workspace_size_that_failed_is_asked_again(monkeypatch, answer):
    from paged_gqa_decode_07_b200 import _binding
    lib = _Sizes(answer)
    monkeypatch.setattr(_binding, "load_library", lambda: lib)
    _binding._prefill_need.cache_clear()
    sizes = (99, 3, 5000, 4000, 0, 8, 2, 128, 0)
    with pytest.raises(_binding.PGDError):
        _binding._prefill_need(*sizes)
    lib.fails = False
    assert _binding._prefill_need(*sizes) == answer
    asked = lib.asked
    assert _binding._prefill_need(*sizes) == answer
    assert lib.asked == asked, "an answer is kept"
    _binding._prefill_need.cache_clear()
