"""The staged norm-and-rotation kernels refill their shared-memory stages while
other warps still work on them (GPU): every token of a batch of many rounds
must come out as it does in small batches, which have no stages, and the same
in every run."""

import pytest
import torch

from mhc_pre_gb300 import binding as B
from tests.test_gpu_qk_norm_rope import _inputs

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda", 0)


@pytest.mark.parametrize("T,Hq,Hk,dh,rot,dtype", [
    (20000, 40, 8, 128, 128, "bf16"), (12000, 20, 4, 128, 64, "f32"), (60000, 4, 2, 64, 64, "bf16"),
    (30000, 3, 1, 128, 0, "bf16"), (15000, 16, 16, 64, 0, "f32")])
def test_stages_are_refilled_after_their_reads(T, Hq, Hk, dh, rot, dtype):
    q, k, v, w, pos, cs, g = _inputs(T, Hq, Hk, dh, rot, dtype, _dev(), seed=3)
    kw = dict(positions=pos, cos_sin=cs) if rot else {}
    r, b = B.mhc_qk_norm_rope(q, k, *w, **kw), B.mhc_qk_norm_rope_bwd(*g, q, k, *w, **kw)
    for t0 in list(range(0, T - 64, T // 40)) + [T - 64]:
        s = slice(t0, t0 + 64)
        kws = dict(positions=pos[s], cos_sin=cs) if rot else {}
        few = B.mhc_qk_norm_rope(q[s], k[s], *w, **kws)
        fewb = B.mhc_qk_norm_rope_bwd(g[0][s], g[1][s], q[s], k[s], *w, **kws)
        assert torch.equal(r.q[s], few.q) and torch.equal(r.k[s], few.k)
        assert torch.equal(b.dq[s], fewb.dq) and torch.equal(b.dk[s], fewb.dk)
    for _ in range(10):
        r2, b2 = B.mhc_qk_norm_rope(q, k, *w, **kw), B.mhc_qk_norm_rope_bwd(*g, q, k, *w, **kw)
        assert torch.equal(r.q, r2.q) and torch.equal(r.k, r2.k)
        assert all(torch.equal(x, y) for x, y in zip(b, b2))
    assert B.get_last_device_error() == B.MHC_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_with_many_tokens(dtype):
    """Outputs over the inputs, parts of a packed projection (the C entry points)."""
    T, Hq, Hk, dh = 20000, 6, 2, 64
    q, k, _, w, pos, cs, _ = _inputs(T, Hq, Hk, dh, 64, dtype, _dev(), seed=4)
    kw = dict(positions=pos, cos_sin=cs)
    want = B.mhc_qk_norm_rope(q, k, *w, **kw)
    code = B.MHC_BF16 if dtype == "bf16" else B.MHC_F32
    packed = torch.cat([q.reshape(T, -1), k.reshape(T, -1)], dim=1)
    qp, kp = packed[:, :Hq * dh], packed[:, Hq * dh:]
    s = torch.cuda.current_stream().cuda_stream
    assert B.lib().mhc_qk_norm_rope(code, qp.data_ptr(), packed.stride(0), kp.data_ptr(), packed.stride(0),
                                    w[0].data_ptr(), w[1].data_ptr(), pos.data_ptr(), cs.data_ptr(), cs.shape[0], T,
                                    Hq, Hk, dh, 64, 0, 1e-6, qp.data_ptr(), packed.stride(0), kp.data_ptr(),
                                    packed.stride(0), s) == B.MHC_OK
    assert torch.equal(qp.reshape(T, Hq, dh), want.q) and torch.equal(kp.reshape(T, Hk, dh), want.k)
    assert B.get_last_device_error() == B.MHC_OK
