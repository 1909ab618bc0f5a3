"""Failure detection of the attention kernel without a GPU fault: in a test-only
build (~10 ms wait limit) every block leaves the first stage of its K and V ring
unfilled, so the bounded waits for it run out. The status has to say so, and
the next call on the same context has to be right."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TIMEOUT_STATUS = 4   # SWIGLU_ERR_DEVICE_TIMEOUT


@pytest.fixture(scope="module")
def fi_lib(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemm_swiglu_mlp_gb300 import build
    path = str(tmp_path_factory.mktemp("fi") / "libswiglu_faultinject.so")
    build.build_fault_injection_library(path)
    lib = ctypes.CDLL(path)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    lib.swiglu_test_set_fault_injection.argtypes = [ctypes.c_int]
    lib.swiglu_test_set_fault_injection.restype = None
    lib.swiglu_tree_attention_workspace_bytes.argtypes = [i64] * 4
    lib.swiglu_tree_attention_workspace_bytes.restype = sz
    lib.swiglu_tree_attention.argtypes = [vp, i64, i64, vp, vp, i64, i64, vp, i64, i64, vp, vp, vp,
                                          i64, ctypes.c_float, vp, i64, i64, i64, i64, vp, sz, vp]
    lib.swiglu_check_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
    return lib


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 30, 70])   # narrow; wide, one row tile and two
def test_wait_timeout_is_reported_and_context_survives(fi_lib, D, new):
    R, ctx, Hq, Hkv, P = 3, 400, 8, 2, 32
    gen = torch.Generator().manual_seed(D + new)
    per = (ctx + new + P - 1) // P
    k, v = (torch.randn(R * per, Hkv, P, D, generator=gen).bfloat16().cuda() for _ in range(2))
    q = torch.randn(R * new, Hq, D, generator=gen).bfloat16().cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(R * per, **i32).view(R, per)
    ctx_lens, start = torch.full((R,), ctx, **i32), torch.arange(R + 1, **i32) * new
    stream = torch.cuda.current_stream().cuda_stream
    nbytes = fi_lib.swiglu_tree_attention_workspace_bytes(R * new, Hq, Hkv, D)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")

    def call():
        out = torch.zeros_like(q)
        assert fi_lib.swiglu_tree_attention(
            q.data_ptr(), Hq * D, D, k.data_ptr(), v.data_ptr(), R * per, P, table.data_ptr(), R,
            per, ctx_lens.data_ptr(), start.data_ptr(), None, 0, D ** -0.5, out.data_ptr(), R * new,
            Hq, Hkv, D, ws.data_ptr(), nbytes, stream) == 0
        raw = ctypes.c_uint32(0)
        return out, fi_lib.swiglu_check_device_status(stream, ctypes.byref(raw)), raw.value

    fi_lib.swiglu_test_set_fault_injection(1)
    try:
        _, status, raw = call()
    finally:
        fi_lib.swiglu_test_set_fault_injection(0)
    assert status == TIMEOUT_STATUS and raw != 0

    out, status, raw = call()   # the word was cleared by the read
    assert status == 0 and raw == 0
    rows = torch.arange(ctx + new, device="cuda")
    for r in range(R):
        kr, vr = (c[table[r, rows // P].long(), :, rows % P].double() for c in (k, v))
        qr = q[r * new:(r + 1) * new].double().view(new, Hkv, Hq // Hkv, D)
        s = torch.einsum("nhgd,xhd->nhgx", qr, kr) * D ** -0.5
        hidden = rows[None, :] > ctx + torch.arange(new, device="cuda")[:, None]
        p = s.masked_fill(hidden[:, None, None], float("-inf")).softmax(-1)
        want = torch.einsum("nhgx,xhd->nhgd", p, vr).reshape(new, Hq, D)
        # weights and results are rounded to BF16: 2^-9 of the largest value each
        err = (out[r * new:(r + 1) * new].double() - want).abs().max() / vr.abs().max()
        assert err <= 2 ** -8
