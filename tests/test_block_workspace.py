"""The workspace query of the dense block product answers for the result type
it is asked about: on the CPU the flags it passes, on the GPU that a workspace
of that size is all the call needs for its K split."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from tests import _block as H
from tests import _gpu as U

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


class _Library:
    """Stands for the C query: 1000 bytes plus its flags."""
    def hq_block_gemm_workspace_size(self, flags, batch, m, n, k, out):
        self.asked = (batch, m, n, k)
        out._obj.value = 1000 + flags
        return 0


def test_query_passes_the_result_type(monkeypatch):
    lib = _Library()
    monkeypatch.setattr(hq, "load", lambda: lib)
    size = lambda t: hq.hq_block_gemm_workspace_size(5, 64, 128, 3, t)  # noqa: E731
    assert [size(t) - 1000 for t in (BF16, F16, F32)] == [0, hq.HQ_OUT_FP16, hq.HQ_OUT_FP32]
    assert lib.asked == (3, 5, 64, 128)
    assert size(None) == 1000 + hq.HQ_OUT_FP32           # the largest of them
    with pytest.raises(ValueError):
        size(torch.float64)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(512, 2048, 8192), (64, 4096, 4096), (128, 7168, 2048), (53, 1880, 14688)])
def test_queried_bytes_hold_the_split(m, n, k):
    """With exactly the bytes of the query a call gives the bits that it gives with
    the largest workspace: the same K slices, added in the same order."""
    U.banner(f"workspace {m}x{n}x{k}")
    r = H.rng("workspace", m, n, k)
    a, b = [H.dev(r.integers(0, 120, (rows, k)).astype(np.uint8)) for rows in (m, n)]
    sa, sb = [H.dev((1e-3 * r.random((rows, -(-k // 128)))).astype(np.float32)) for rows in (m, -(-n // 128))]
    sizes = {t: hq.hq_block_gemm_workspace_size(m, n, k, out_dtype=t) for t in (BF16, F16, F32)}
    assert sizes[F16] == sizes[F32] > 0
    assert hq.hq_block_gemm_workspace_size(m, n, k) == max(sizes.values())
    for dtype, accumulate in ((BF16, False), (F16, False), (F32, False), (F32, True)):
        outs = []
        for size in (sizes[dtype], hq.HQ_BLOCK_WORKSPACE_BYTES):
            ws = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda")
            out = torch.ones((m, n), dtype=dtype, device="cuda")
            hq.hq_block_gemm(a, sa, b, sb, out, accumulate=accumulate, workspace=ws[:size])
            torch.cuda.synchronize()
            assert torch.all(ws[size:] == 0xA5), "bytes past the workspace written"
            if size == sizes[dtype] > 0:
                assert torch.any(ws[:size] != 0xA5), f"{dtype}: K was not split"
            outs.append(out)
        assert torch.equal(outs[0], outs[1]), f"{dtype} accumulate={accumulate}"
