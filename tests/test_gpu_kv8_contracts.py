"""What include/qsa.h promises of the 8-bit cache calls, seen from C (B200 only)."""
import pytest
import torch

from test_gpu_kv8_attention import SCALE, make

pytestmark = pytest.mark.gpu

qsa = pytest.importorskip("sparse_attention_block_qsa_b200")
DEV = torch.device("cuda")


def pointer(t):
    return None if t is None else t.data_ptr()


def attention(d, out, lse, weights=None, workspace=None, width=None):
    """qsa_sparse_attention_fp8 through the C ABI, contiguous tensors on the GPU."""
    T, Hq, _ = d["q"].shape
    pages, ps, H, _ = d["kc"].shape
    width = d["tok"].shape[1] if width is None else width
    blocks = d["ks"].shape[1]
    return qsa.lib().qsa_sparse_attention_fp8(
        pointer(d["q"]), Hq * 256, 256, Hq, pointer(d["kc"]), pointer(d["vc"]), pointer(d["ks"]), pointer(d["vs"]), pages,
        ps, ps // blocks, ps * H * 256, H * 256, 256, blocks * H, H, H, pointer(d["table"]), d["table"].shape[1],
        d["table"].shape[1], pointer(d["cu"]), pointer(d["sl"]), d["sl"].shape[0], pointer(d["tok"]), d["tok"].shape[1],
        width, T, None, SCALE, pointer(out), Hq * 256, pointer(lse), pointer(weights), width, pointer(workspace),
        0 if workspace is None else workspace.numel(), torch.cuda.current_stream().cuda_stream)


def test_empty_lists_need_no_workspace():
    """No entries: zeros and -infinity, without a workspace."""
    d = {k: v.to(DEV) for k, v in make([70, 40], [2, 300], 24, 2, 16, 16, 8, seed=17).items()}
    out = torch.full(d["q"].shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(out.shape[:2], 7.0, device=DEV)
    assert attention(d, out, lse, width=0) == 0
    torch.cuda.synchronize()
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
