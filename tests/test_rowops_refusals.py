"""The binding refuses row operators' arguments that are missing or of another
kind by name, as ValueError or TypeError, before anything is launched."""
import pytest
import torch

from scaled_fp8_gemm_amd import fp8sg as F


def cases(dev):
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device=dev)
    f, i = torch.zeros(16, device=dev), torch.zeros(4, 2, dtype=torch.int32, device=dev)
    off, src = torch.zeros(9, dtype=torch.int32, device=dev), torch.zeros(8, dtype=torch.int32, device=dev)
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=dev)
    q, s = torch.zeros(4, 16, dtype=torch.uint8, device=dev), torch.zeros(4, 1, device=dev)
    held, out = F.operand(q, 0, 1, s), F.cast_out(q, 0, 1, s)
    return [
        ("gamma is required", lambda: F.fp8_layernorm_fwd(x, None, f, 1e-5, x, f, f)),
        ("beta is required", lambda: F.fp8_layernorm_fwd(x, f, None, 1e-5, x, f, f)),
        ("beta has dtype", lambda: F.fp8_layernorm_fwd(x, f, x[0], 1e-5, x, f, f)),
        ("yq must be a cast_out", lambda: F.fp8_layernorm_fwd(x, f, f, 1e-5, x, f, f, yq=held)),
        ("xhat must be a cast_out", lambda: F.fp8_layernorm_fwd(x, f, f, 1e-5, x, f, f, xhat=q)),
        ("dx is required",
         lambda: F.fp8_layernorm_bwd(x, x, f, f, f, None, f, f, workspace=ws)),
        ("gamma is required",
         lambda: F.fp8_layernorm_bwd(x, x, f, f, None, x, f, f, workspace=ws)),
        ("dx has dtype", lambda: F.fp8_layernorm_bwd(x, x, f, f, f, f, f, f, workspace=ws)),
        ("xhat must be an operand",
         lambda: F.fp8_layernorm_bwd(x, None, None, f, f, x, f, f, xhat=out, workspace=ws)),
        ("h is required", lambda: F.fp8_act_bwd(x, None, F.ACT_SILU, False, x)),
        ("ckpt must be a cast_out", lambda: F.fp8_act_fwd(x, F.ACT_SILU, False, x, ckpt=held)),
        ("ckpt must be a cast_out", lambda: F.fp8_checkpoint_save(x, held)),
        ("ckpt must be an operand", lambda: F.fp8_checkpoint_load(out, 4, 16, x)),
        ("src is required", lambda: F.fp8_moe_sort(i, 8, 1, off, f, i, None, workspace=ws)),
        ("src is required", lambda: F.fp8_moe_dispatch(x, i, None, off, x)),
        ("offsets is required", lambda: F.fp8_moe_dispatch(x, i, src, None, x)),
        ("offsets is required", lambda: F.fp8_moe_combine_bwd(x, x, f, i, src, None, x, f)),
    ]


NAMES = range(len(cases("cpu")))


@pytest.mark.parametrize("n", NAMES)
def test_refused_on_the_host(n):
    # that the tensors are not on a GPU may be found first
    with pytest.raises((ValueError, TypeError), match=cases("cpu")[n][0] + "|on the GPU"):
        cases("cpu")[n][1]()


@pytest.mark.gpu
@pytest.mark.parametrize("n", NAMES)
def test_refused_by_name(n):
    with pytest.raises((ValueError, TypeError), match=cases("cuda")[n][0]):
        cases("cuda")[n][1]()


@pytest.mark.gpu
def test_bf16_bits_and_bf16_are_one_type():
    """A BF16 tensor may come as int16 bits, next to one that does not."""
    x = torch.randn(4, 40, device="cuda").bfloat16()
    g, b = torch.randn(40, device="cuda").bfloat16(), torch.randn(40, device="cuda").bfloat16()
    out = []
    for gamma, beta in ((g, b), (g.view(torch.int16), b)):
        y, m, r = torch.empty_like(x), torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
        F.fp8_layernorm_fwd(x, gamma, beta, 1e-5, y, m, r)
        out.append(y)
    assert torch.equal(*out)
