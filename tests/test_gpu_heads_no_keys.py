"""The heads' norm of keys with no heads: all outputs are what an empty sum gives."""
import ctypes

import pytest
import torch

from tests import attention_reference as ref
from tests.test_gpu_heads import both_types, close, put, wanted

pytestmark = pytest.mark.gpu


@both_types
@pytest.mark.parametrize("M", [0, 5])
@pytest.mark.parametrize("D", [64, 7])
def test_keys_without_heads(gdr, dtype, M, D):
    from chunked_gated_delta_08_gb300 import attention_ops as ops
    p = ref.head_inputs(max(M, 1), 2, 0, D, 0, dtype, seed=1)
    q = put({k: v if v is None or k == "wq" else v[:M] for k, v in p.items()})
    none = torch.zeros(M, 0, D, dtype=dtype, device="cuda")
    yq, yk = gdr.qk_norm_fwd(q["q"], none, q["wq"], q["wq"])
    assert yk.shape == none.shape
    dq, dk, dwq, dwk = gdr.qk_norm_bwd(q["dyq"], none, q["q"], none, q["wq"], q["wq"])
    assert dk.shape == none.shape and (dwk == 0).all()
    if M:
        want = wanted(p, False)
        close(yq, want["yq"])
        close(dwq, want["dwq"], 10)
    # the same through the C entry, on memory that holds something
    full = torch.full((D,), 7.0, device="cuda")
    desc = ops.GdrQkNormDesc(M, 2, 0, D, 0, 0, 2 * D, 0, 2 * D, 0, 1e-6, int(dtype == torch.bfloat16),
                             int(dtype == torch.bfloat16), 0, 0)
    a = lambda t: t.data_ptr()  # noqa: E731
    assert gdr.lib().gdr_qk_norm_bwd(ctypes.byref(desc), a(q["dyq"]), None, a(q["q"]), None, a(q["wq"]), None, None, None,
                                     None, a(dq), None, a(dwq), a(full), torch.cuda.current_stream().cuda_stream) == 0
    assert (full == 0).all()
    assert gdr.device_status() == 0
