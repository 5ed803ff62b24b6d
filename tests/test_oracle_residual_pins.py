"""Pins of the residual path's CPU oracle: published Philox vectors, torch's float64 layer norm
and autograd, central differences, a generator written a second way, masks by hand."""
import numpy as np
import pytest
import torch

from oracle import residual as orc


@pytest.mark.parametrize("ctr,key,out", [
    # the known answers published with the generator (10 rounds)
    ([0, 0, 0, 0], [0, 0], [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
    ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
    ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
     [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]),
])
def test_philox_known_answers(ctr, key, out):
    assert orc.philox4x32(ctr, key).tolist() == out


def test_kept_by_python_integers():
    """The mask of every element again, in Python integers."""
    seed, offset, p, n = 0x123456789abcdef0, (7 << 32) + 5, 0.3, 83

    def block(g):
        c = [g % 2 ** 32, g >> 32, offset % 2 ** 32, offset >> 32]
        k = [seed % 2 ** 32, seed >> 32]
        for _ in range(10):
            a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(b >> 32) ^ c[1] ^ k[0], b % 2 ** 32, (a >> 32) ^ c[3] ^ k[1], a % 2 ** 32]
            k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
        return c
    want = [((block(e // 8)[e % 8 // 2] >> (16 * (e % 2))) & 0xffff) >= round(p * 65536) for e in range(n)]
    assert orc.kept((n,), seed, offset, p).tolist() == want


def test_kept_share_and_independence():
    k = orc.kept((1 << 20,), 11, 3, 0.1)
    sd = np.sqrt(0.1 * 0.9 / k.size)
    assert abs((~k).mean() - round(6553.6) / 65536) < 5 * sd
    assert abs(np.mean(~k[:-1] & ~k[1:]) - 0.01) < 5 * np.sqrt(0.01 * 0.99 / k.size)
    other = orc.kept((1 << 20,), 11, 4, 0.1)
    assert abs(np.mean(~k & ~other) - 0.01) < 5 * np.sqrt(0.01 * 0.99 / k.size)
    assert orc.kept((100,), 1, 1, 0.0).all() and not orc.kept((100,), 1, 1, 1.0).any()


def case(B=3, T=5, C=11, seed=0):
    r = np.random.default_rng(seed)
    return (r.standard_normal((B, T, C)), r.standard_normal((B, T, C)), 1 + 0.1 * r.standard_normal(C),
            0.1 * r.standard_normal(C), np.array([5, 0, 3], np.int32)[:B])


def test_layernorm_matches_torch_and_its_autograd():
    x, dy, gamma, beta, lens = case()
    valid = np.arange(5)[None] < lens[:, None]
    xt = torch.tensor(x, requires_grad=True)
    gt, bt = torch.tensor(gamma, requires_grad=True), torch.tensor(beta, requires_grad=True)
    yt = torch.nn.functional.layer_norm(xt, (11,), gt, bt, 1e-5) * torch.tensor(valid)[..., None]
    yt.backward(torch.tensor(dy))
    y, mean, rstd = orc.layernorm_fwd(x, gamma, beta, lens, 1e-5)
    np.testing.assert_allclose(y, yt.detach().numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(mean, x.mean(-1) * valid, rtol=1e-12, atol=1e-14)
    dx, dgamma, dbeta = orc.layernorm_bwd(x, dy, gamma, mean, rstd, lens)
    np.testing.assert_allclose(dx, xt.grad.numpy(), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(dgamma, gt.grad.numpy(), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(dbeta, bt.grad.numpy(), rtol=1e-11, atol=1e-12)
    assert (y[~valid] == 0).all() and (dx[~valid] == 0).all() and (rstd[~valid] == 0).all()


def test_no_parameters_means_ones_and_zeros():
    x, dy, _, _, lens = case(seed=1)
    y, mean, rstd = orc.layernorm_fwd(x, None, None, lens, 1e-3)
    y1, _, _ = orc.layernorm_fwd(x, np.ones(11), np.zeros(11), lens, 1e-3)
    assert np.array_equal(y, y1)
    for a, b in zip(orc.layernorm_bwd(x, dy, None, mean, rstd, lens),
                    orc.layernorm_bwd(x, dy, np.ones(11), mean, rstd, lens)):
        assert np.array_equal(a, b)


def test_fused_gradients_against_central_differences():
    """d/d(input) of sum(dh . s) + sum(dy . y), every input of the fused forward."""
    x, dy, gamma, beta, lens = case(B=2, T=3, C=7, seed=2)
    lens = np.array([3, 1], np.int32)
    r = np.random.default_rng(9)
    res, dh = r.standard_normal(x.shape), r.standard_normal(x.shape)
    args = (5, 6, 0.4, 0.5)

    def loss(x, res, gamma, beta):
        s, y, _, _ = orc.dropout_add_layernorm_fwd(x, res, *args, gamma, beta, lens, 1e-5)
        return float((dh * s).sum() + (dy * y).sum())
    s, _, mean, rstd = orc.dropout_add_layernorm_fwd(x, res, *args, gamma, beta, lens, 1e-5)
    grads = orc.dropout_add_layernorm_bwd(dy, dh, s, gamma, mean, rstd, *args, lens)
    inputs = [x, res, gamma, beta]
    for i, g in enumerate(grads):
        num = np.zeros(inputs[i].size)
        for j in range(num.size):
            v = []
            for step in (1e-5, -1e-5):
                a = [u.copy() for u in inputs]
                a[i].reshape(-1)[j] += step
                v.append(loss(*a))
            num[j] = (v[0] - v[1]) / 2e-5
        # central differences: truncation h^2 f'''/6 and cancellation 2^-52 |loss| / h, both ~1e-9
        np.testing.assert_allclose(g.reshape(-1), num, rtol=1e-6, atol=1e-7)


def test_dropped_elements_ignore_what_they_hold():
    x, _, _, _, _ = case()
    keep = orc.kept(x.shape, 1, 2, 0.5)
    y = orc.dropout_add(np.where(keep, x, np.nan), None, 1, 2, 0.5, 1.0, None)
    assert np.isfinite(y).all() and np.allclose(y[keep], 2 * x[keep]) and (y[~keep] == 0).all()
