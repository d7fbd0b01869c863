"""The norm's sum and its gradient written where one of their inputs lies, few rows and many, aligned or not: the bits
of separate tensors."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import blockwise_scaled_fp8_gb300 as B  # noqa: E402

bf16, f32 = torch.bfloat16, torch.float32


def rows(T, K, off, values=None):
    """[T, K] inside a larger buffer, `off` elements from a 16-byte boundary (off 0: packed)."""
    ld = K + 3 * off
    t = torch.empty(T * ld + off + 8, device="cuda", dtype=bf16)[off:off + T * ld].view(T, ld)[:, :K]
    return t.copy_(torch.randn(T, K, device="cuda") if values is None else values)


def ld(t):
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


@pytest.mark.parametrize("T", [1, 100, 153, 700])
@pytest.mark.parametrize("K", [7, 513, 2001, 4096, 9001])
@pytest.mark.parametrize("off", [0, 1, 5])
def test_in_place(T, K, off):
    torch.manual_seed(T + K + off)
    x, r, w = rows(T, K, off), rows(T, K, 0), torch.randn(K, device="cuda")
    ref = B.rms_norm_quant(x, w, residual=r)
    h = rows(T, K, off, x)
    o = B.rms_norm_quant(h, w, residual=r, h=h)
    assert o.h is h and torch.equal(h, ref.h)
    dy, dh = rows(T, K, off), rows(T, K, off)
    dx, dw = B.rms_norm_bwd(dy, h, w, o.rstd, dh=dh)
    L = B.lib()
    n = max(L.bfp8_rms_norm_bwd_workspace_size(T, K), 16)
    for into in ("dy", "h", "dh"):
        t = {name: rows(T, K, off, v) for name, v in (("dy", dy), ("h", h), ("dh", dh))}
        ws, dw2 = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(K, device="cuda")
        st = L.bfp8_rms_norm_bwd(t["dy"].data_ptr(), T, K, ld(t["dy"]), t["h"].data_ptr(), ld(t["h"]), w.data_ptr(), 1,
                                 o.rstd.data_ptr(), t["dh"].data_ptr(), ld(t["dh"]), t[into].data_ptr(), ld(t[into]),
                                 dw2.data_ptr(), ws.data_ptr(), n, B._stream())
        assert st == B.BFP8_OK and torch.equal(t[into], dx) and torch.equal(dw2, dw), into
    B.check_device_errors()
