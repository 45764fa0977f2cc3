"""The products' forms, each against the definition in 64 bits, and calls that
follow each other at once."""
import pytest
import torch

from test_gpu_act8 import data, stored

pytestmark = pytest.mark.gpu


def _api():
    from bit_quantized_shampoo_b200 import api
    return api


@pytest.mark.parametrize("tokens,out,inner", [(1, 700, 900), (40, 500, 300), (2100, 2600, 400)])
def test_layers_back_to_back_take_their_own_scales(tokens, out, inner):
    """Calls whose scratch and scales lie where the call before them had its
    own, at other magnitudes; each product starts under the pass that writes
    them."""
    api = _api()
    w = stored(out, inner, 1)[0]
    xs = [data(tokens, inner, "bf16", 2 + k, scale=10.0 ** (3 * k - 6)) for k in range(5)]
    dys = [data(tokens, out, "bf16", 9 + k, scale=10.0 ** (6 - 3 * k)) for k in range(5)]
    ys, dxs = [], []
    for x, dy in zip(xs, dys):
        ys.append(api.act8_linear(x, *w))
        dxs.append(api.act8_input_grad(dy, *w))
        torch.cuda.synchronize()
    for _ in range(4):
        for k in (3, 0, 4, 1, 2):
            y, dx = api.act8_linear(xs[k], *w), api.act8_input_grad(dys[k], *w)
            assert torch.equal(y, ys[k]) and torch.equal(dx, dxs[k])
            y, dx = None, None
