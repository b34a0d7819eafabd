"""GPU tests of checkpoints whose padding columns hold something: codes of another writer, or buffers used again."""
import pytest
import torch

from _helpers import nv, require_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu", "geglu"])
@pytest.mark.parametrize("m,n", [(3, 1), (5, 4), (130, 20), (40, 100), (7, 2072)])
def test_the_activation_does_not_see_padding_codes(m, n, act):
    k = 2 * n if act in ("swiglu", "geglu") else n
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(m, (k + 7) // 8 * 8, device="cuda", generator=g).to(torch.bfloat16)[:, :k]
    dout = torch.randn(m, (n + 7) // 8 * 8, device="cuda", generator=g).to(torch.bfloat16)[:, :n]
    _, q, sf = nv.act_checkpoint(x, act)
    want = nv.act_checkpoint_backward(dout, q, sf, act, recompute=True)
    for code in (0x7E, 0xFE, 0x7F):                          # the largest value, its negative, NaN
        q[:, k:] = code
        got = nv.act_checkpoint_backward(dout, q, sf, act, recompute=True)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert (got[1][:, n:] == 0).all()
