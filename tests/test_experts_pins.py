"""The routed-experts oracle (oracle/moe_experts.py) against facts fixed outside it."""
import numpy as np
import torch

from oracle import moe_experts as X


def test_e4m3_rounding_matches_the_format():
    bits = torch.arange(0x7F, dtype=torch.uint8)
    assert np.array_equal(X.e4m3_grid(), bits.view(torch.float8_e4m3fn).double().numpy())
    g = torch.Generator().manual_seed(1)
    v = torch.cat([torch.randn(4000, generator=g) * torch.exp(3 * torch.randn(4000, generator=g)),
                   torch.tensor([0.0, 448.0, 432.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0])])
    v = v.clamp(-448, 448)
    assert np.array_equal(X.round_e4m3(v.double().numpy()), v.to(torch.float8_e4m3fn).double().numpy())


def test_sort_by_hand():
    idx = np.array([[3, 1], [1, 9], [-1, 3], [2, 2]], np.int32)
    s = X.sort(idx, 1, 3)
    assert s["expert_offsets"].tolist() == [0, 2, 4, 6]
    assert s["source_of"].tolist() == [1, 2, 6, 7, 0, 5, -1, -1]
    assert s["row_of"].tolist() == [[4, 0], [1, -1], [-1, 5], [2, 3]]


def test_weights_of_a_token_sum_to_the_scale():
    rng = np.random.default_rng(0)
    idx = rng.integers(0, 16, (9, 4)).astype(np.int32)
    w = X.routing_weights(idx, rng.random((9, 16)) + 0.1, True, 2.5)
    np.testing.assert_allclose(w.sum(1), 2.5, rtol=1e-12)
    assert not X.routing_weights(idx, np.zeros((9, 16)), True, 2.5).any()


def test_quantised_values_reach_448_and_come_back():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((5, 272))
    q, s = X.quantize(v)
    assert s.shape == (3, 5)
    for b in range(3):
        part = slice(128 * b, 128 * (b + 1))
        np.testing.assert_allclose(np.abs(q[:, part]).max(1), 448.0, rtol=1e-12)
        np.testing.assert_allclose(q[:, part] * s[b][:, None], v[:, part], rtol=1e-12)
    assert not X.quantize(np.zeros((1, 16)))[0].any()


def test_combine_and_gradient_against_autograd():
    rng = np.random.default_rng(2)
    idx = rng.integers(0, 6, (7, 3)).astype(np.int32)
    row_of = X.sort(idx, 1, 4)["row_of"]
    rows = torch.tensor(rng.standard_normal((21, 16)), requires_grad=True)
    w = torch.tensor(rng.random((7, 3)), requires_grad=True)
    out = sum(torch.where(torch.tensor(row_of[:, k] >= 0)[:, None],
                          w[:, k, None] * rows[torch.tensor(row_of[:, k]).clamp(min=0).long()], 0.0) for k in range(3))
    g = torch.tensor(rng.standard_normal((7, 16)))
    out.backward(g)
    np.testing.assert_allclose(X.combine(rows.detach().numpy(), row_of, w.detach().numpy()), out.detach().numpy(),
                               rtol=1e-12, atol=1e-12)
    gr, gw = X.combine_backward(g.numpy(), rows.detach().numpy(), row_of, w.detach().numpy())
    np.testing.assert_allclose(np.nan_to_num(gr), rows.grad.numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(gw, w.grad.numpy(), rtol=1e-12, atol=1e-12)


def test_product_is_the_dequantised_product():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((3, 272)), rng.standard_normal((144, 272))
    xs, ws = rng.random((3, 3)), rng.random((2, 3))
    xd = x * np.repeat(xs.T, 128, 1)[:, :272]
    wd = w * np.repeat(np.repeat(ws, 128, 0), 128, 1)[:144, :272]
    np.testing.assert_allclose(X.product(x, xs, w, ws)[0], xd @ wd.T, rtol=1e-10, atol=1e-10)
