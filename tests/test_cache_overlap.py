"""Refusals of attention outputs that lie on its inputs, made before any launch."""
import pytest


def addr(i):
    return 0x10000 + i * 0x10000000     # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from gemm_swiglu_mlp_gb300 import build
    build.build()
    import gemm_swiglu_mlp_gb300 as sg
    return sg.load_library()


def test_out_on_an_index_array(lib):
    table, ctx, start, mask = (addr(i) for i in range(3, 7))

    def refused(out):
        # only ever called with addresses that are refused: one that is not would be
        # launched with them where there is a GPU
        return lib.swiglu_tree_attention(addr(0), 256, 64, addr(1), addr(2), 4, 16, table, 2, 4, ctx,
                                         start, mask, 1, 0.125, out, 3, 4, 2, 64, None, 0, None) == 1

    # out has 1536 bytes; the table 32, the lengths 8, their sums 12, the masks 24
    for where, size in ((table, 32), (ctx, 8), (start, 12), (mask, 24)):
        assert refused(where)
        assert refused(where + 16 * ((size - 1) // 16))
        assert refused(where - 1536 + 16)


@pytest.mark.gpu
def test_workspace_on_an_input(lib):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_swiglu_mlp_gb300 as sg
    need = sg.swiglu_tree_attention_workspace_bytes(3, 4, 2, 64)
    ws = torch.zeros(need + 512, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    args = dict(block_table=torch.zeros(2, 4, **i32), ctx_lens=torch.full((2,), 5, **i32),
                query_start=torch.tensor([0, 1, 3], **i32),
                mask=torch.zeros(3, 1, dtype=torch.int64, device="cuda"))
    sg.swiglu_tree_attention(q, k, k.clone(), **args, workspace=ws)
    for name, t in args.items():
        n = t.numel() * t.element_size()
        for at in (0, need - 8 * (-(-n // 8))):     # at the workspace's start and end
            on = ws[at:at + n].view(t.dtype).view(t.shape)
            with pytest.raises(sg.SwigluError):
                sg.swiglu_tree_attention(q, k, k.clone(), **dict(args, **{name: on}), workspace=ws)
        off = ws[need:need + n].view(t.dtype).view(t.shape).copy_(t)
        sg.swiglu_tree_attention(q, k, k.clone(), **dict(args, **{name: off}), workspace=ws)
    sg.swiglu_check_device_status()
