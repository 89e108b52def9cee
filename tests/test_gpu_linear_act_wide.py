"""melded_linear_fwd_act with very many columns for a few tokens: more than a
launch of the few-token kernel holds.  Codes of +-1, so every sum is a small
integer, exact in float32 and bfloat16."""
import pytest
import torch

from tests.gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 16])
@pytest.mark.parametrize("d_out", [(1 << 26) - 16, 1 << 26])
def test_columns_past_a_grid_of_few_token_workgroups(gpu_lib, T, d_out):
    announce(f"melded_linear_fwd_act T={T} d_in=16 d_out={d_out}")
    g = torch.Generator(device="cuda")
    g.manual_seed(d_out + T)

    def signs(rows):
        t = torch.empty((rows, 16), dtype=torch.uint8, device="cuda")
        t.random_(0, 2, generator=g)
        return t.mul_(128).bitwise_or_(0x38)

    xq, wq, one = signs(T), signs(d_out), torch.ones(1, device="cuda")
    y = torch.full((T, d_out), float("nan"), dtype=torch.bfloat16, device="cuda")
    gpu_lib.melded_linear_fwd_act(xq, one, wq, one, y)
    x = xq.view(torch.float8_e4m3fn).float()
    for a in range(0, d_out, 1 << 23):
        w = wq[a:a + (1 << 23)].view(torch.float8_e4m3fn).float()
        assert torch.equal(y[:, a:a + (1 << 23)].float(), x @ w.T), a
    del wq, y
    torch.cuda.empty_cache()
