"""GPU: the rotation's gradient where a warp has more room than heads."""
import pytest

from tests import _cache as C
from tests import _more as R
from tests._gpu import need_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def X():
    need_gpu()
    from sparse_depth_token_gb300 import xmod
    xmod.load()
    return xmod


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,hq,hkv", [(32, 3, 1), (64, 6, 3), (128, 5, 5), (128, 1, 1), (128, 8, 4)])
@pytest.mark.parametrize("rot", [8, 32])
def test_gradient_without_epsilon(X, dtype, hd, hq, hkv, rot):
    """rms_eps of 0 with numbers of heads that no warp's lanes divide: lanes without a head have no
    norm to divide by."""
    M, g = 37, torch.Generator().manual_seed(hd + hq)
    dm = C.dims(X, hq, hkv, hd, dtype, 0.0)
    width = (hq + hkv) * hd
    qkv = torch.randn(M, width, generator=g).cuda().to(C.DT[dtype])
    dout = torch.randn(M, width, generator=g).cuda().to(C.DT[dtype])
    gains = {n: (1 + 0.2 * torch.randn(hd, generator=g)).cuda().to(C.DT[dtype]) for n in ("q_norm", "k_norm")}
    w, rope = X.layer_weights(gains), X.rope(hd, 1e4, rot_dim=rot)
    pos = torch.randint(0, 5000, (M,), generator=g).to(torch.int32).cuda()
    din, dq, dk = torch.zeros_like(dout), torch.zeros(hd, device="cuda"), torch.zeros(hd, device="cuda")
    ws = torch.zeros(X.qk_rope_bwd_workspace_bytes(dm, M), dtype=torch.uint8, device="cuda")
    X.qk_rope_bwd(dm, qkv, w, rope, dout, din, pos=pos, dq_norm=dq, dk_norm=dk, ws=ws)
    out = torch.zeros_like(qkv)
    X.qk_rope(dm, qkv, w, rope, out, pos=pos)
    # sums of hd terms in fp32 (halved by a root, doubled by a product), cosine and sine 1.02e-7, a
    # dozen roundings; of the gains' sums M rows of heads more
    rel = (2 * hd + 24) * 2.0 ** -24 + 1.02e-7
    for cols, gain, dgain in ((slice(0, hq * hd), "q_norm", dq), (slice(hq * hd, width), "k_norm", dk)):
        part = lambda t: t[:, cols].reshape(M, -1, hd)  # noqa: E731
        ref, size = R.rope_ref(part(qkv), gains[gain], 0.0, rope, pos)
        half = C.HALF[dtype]
        assert float(((part(out).double() - ref).abs() - size * rel - half * (ref.abs() + size * rel)).max()) <= 0
        dx, dg, err, terms = R.rope_grad_ref(part(qkv), gains[gain], 0.0, rope, pos, part(dout))
        assert float(((part(din).double() - dx).abs() - err * rel - half * (dx.abs() + err * rel)).max()) <= 0
        assert float(((dgain.double() - dg).abs() - terms * (rel + M * 2.0 ** -24)).max()) <= 0
