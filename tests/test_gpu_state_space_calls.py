"""Calls at the edges of what the state-space layer's entry points take, on the GPU."""
import pytest
import torch

from sparse_memory_linear_amd import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g).to(DEV)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,d,K", [(2, 2, 8, 4), (3, 1, 5, 2), (1, 4, 12, 8)])
def test_convolution_backward_of_no_tokens(B, H, d, K, dtype):
    """No tokens, no strides given: the state's gradient is passed on, also in place, and the weights' are 0."""
    L, r, p = binding.lib(), gen(1), lambda t: t.data_ptr()  # noqa: E731
    w, S0, dS = r(H, d, K), r(B, H, K - 1, d).to(dtype), r(B, H, K - 1, d).to(dtype)
    want = dS.clone()
    ws = torch.empty(L.sdm_causal_conv_backward_workspace_bytes(B, H, 0, d, K), dtype=torch.uint8, device=DEV)
    for dS0 in (torch.full_like(dS, 7.0), dS):
        dw, db = torch.full_like(w, 7.0), torch.full((H, d), 7.0, device=DEV)
        rc = L.sdm_causal_conv_backward(None, None, int(dtype == BF), None, p(w), None, 1, p(S0), p(dS), None, None, None, None, p(dw), p(db),
                                        p(dS0), B, H, 0, d, K, p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0, L.sdm_last_error()
        assert torch.equal(dS0, want) and (dw == 0).all() and (db == 0).all()
