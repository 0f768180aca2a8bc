"""The 64-bit forms the GPU tests compare against, checked on their own: the
gradients against differences, a packed call against its sequences one by one,
and a scan cut in two against the whole."""
import torch

import layer_ref as R

torch.manual_seed(0)


def _r(*shape, std=1.0):
    return torch.randn(*shape, dtype=R.F64) * std


def test_norm_gradient_against_differences():
    assert torch.autograd.gradcheck(lambda x, w, r: R.norm(x, w, r), tuple(
        t.requires_grad_(True) for t in (_r(3, 5), _r(5), _r(3, 5))))


def test_conv_gradient_against_differences():
    args = [_r(6, 3), _r(3, 4), _r(3), _r(3, 3, 3)]
    assert torch.autograd.gradcheck(lambda x, w, b, s: R.conv(x, w, b, s, [2, 0, 4]),
                                    tuple(t.requires_grad_(True) for t in args))


def test_scan_gradient_against_differences():
    args = [_r(5, 4), _r(5, 4), -_r(4, 8).abs(), _r(5, 2, 8), _r(5, 2, 8), _r(4), _r(5, 4), _r(4), _r(2, 4, 8)]
    assert torch.autograd.gradcheck(lambda *a: R.scan(*a, [2, 3]), tuple(t.requires_grad_(True) for t in args))


def test_packed_equals_one_by_one_and_a_cut_scan_the_whole():
    lens = [3, 0, 5]
    x, w, st = _r(8, 3), _r(3, 4), _r(3, 3, 3)
    y, so = R.conv(x, w, None, st, lens)
    y2, s2 = R.conv(x[3:], w, None, st[2:], [5])
    assert torch.equal(y[3:], y2) and torch.equal(so[2:], s2) and torch.equal(so[1], st[1])
    a = [_r(8, 4), _r(8, 4), -_r(4, 8).abs(), _r(8, 1, 8), _r(8, 1, 8)]
    s0 = _r(1, 4, 8)
    y, h = R.scan(*a, None, None, None, s0, [8])
    cut = lambda i, j, s: R.scan(a[0][i:j], a[1][i:j], a[2], a[3][i:j], a[4][i:j], None, None, None, s, [j - i])
    y1, h1 = cut(0, 3, s0)
    y2, h2 = cut(3, 8, h1)
    assert torch.allclose(torch.cat([y1, y2]), y, rtol=1e-12) and torch.allclose(h, h2, rtol=1e-12)
