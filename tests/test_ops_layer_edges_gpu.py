"""The attention layer's operators on the GPU where they once went wrong: against the plain FP64
references of layer_ref.py, or against themselves."""
import numpy as np
import pytest
import torch

from test_ops_layer_gpu import BF16, F32, full, gdr, gen, heads, pack, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 64])
def test_documents_written_by_the_kernel_before(gdr, D):
    # no queries: dk and dv are zero in the rows that cu_keys names, which the kernel before writes
    # as it ends, though kernels behind it may begin early: the integers pass through layer norm's
    # dx = dh (dy = 0) as they are
    g, HK, rows, width = gen(D), 2, 20000, 512
    lens = [700, 0, 129, 300]
    (_, cuh), n = pack(lens), sum(lens)
    none, noneh = pack([0] * len(lens))
    dh = torch.zeros(rows, width, device="cuda")
    dh.view(torch.int32)[-1, :len(cuh)] = torch.tensor(cuh, dtype=torch.int32, device="cuda")
    x, dy = randn(g, rows, width), torch.zeros(rows, width, device="cuda")
    k, q = randn(g, n, HK, D, dtype=BF16), torch.empty(0, 4, D, dtype=BF16, device="cuda")
    lse = torch.empty(4, 0, device="cuda")
    for _ in range(5):
        dx = torch.zeros(rows, width, device="cuda")
        grads = {name: full((n, HK, D), BF16) for name in ("dk", "dv")}
        torch.cuda.synchronize()
        gdr.lnorm_bwd(x, dy=dy, dh=dh, grads={"dx": dx})
        cuk = dx.view(torch.int32)[-1, :len(cuh)]
        got = gdr.attn_bwd(q, k, k, q, lse, q, none, noneh, cu_keys=cuk, cu_keys_host=np.asarray(cuh, dtype=np.int32), grads=grads)
        assert (got["dk"] == 0).all() and (got["dv"] == 0).all()
        assert cuk.tolist() == cuh
