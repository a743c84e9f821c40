"""The 64-bit reference of the blocks of 128 and of routing (b128_reference.py) against what the formats and the
definition say, on the CPU."""
import pytest
import torch

import b128_reference as ref


@pytest.mark.parametrize("elem,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_codec_is_torchs(elem, dtype):
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    t, v = ref.decode_table(elem), codes.view(dtype).double()
    assert torch.equal(torch.nan_to_num(t, 7.5), torch.nan_to_num(v, 7.5))
    f = ref.FMAX[elem]
    x = torch.cat((torch.randn(20000, generator=torch.Generator().manual_seed(0)).double() * f / 3, t[torch.isfinite(t)]))
    grid = torch.unique(t[torch.isfinite(t)].abs())
    x = torch.cat((x, (grid[1:] + grid[:-1]) / 2, -(grid[1:] + grid[:-1]) / 2)).clamp(-f, f)
    assert torch.equal(ref.encode(x, elem), x.float().to(dtype).view(torch.uint8))


@pytest.mark.parametrize("elem", ["e4m3", "e5m2"])
def test_quantize(elem):
    x = torch.randn((5, 300), generator=torch.Generator().manual_seed(1))
    x[2, :128] = 0
    for rule in ("amax", "ceil"):
        c, s = ref.quantize(x, elem, rule)
        assert c.shape == (5, 384) and s.shape == (5, 3) and bool((c[:, 300:] == 0).all()) and float(s[2, 0]) == 1.0
        back = ref.values(c, s, elem)[:, :300]
        a = torch.nn.functional.pad(x.double(), (0, 84)).view(5, 3, 128).abs().amax(2).repeat_interleave(128, 1)[:, :300]
        # half a step of the value, or of the smallest normal number, and the rounding of the factor
        step = 2.0 ** -4 if elem == "e4m3" else 2.0 ** -3
        low = (2.0 ** -10 if elem == "e4m3" else 2.0 ** -17) / ref.FMAX[elem] * 2
        assert bool(((back - x).abs() <= step * x.abs().double() * (1 + 1e-6) + low * a + 1e-30).all())
        if rule == "ceil":
            m, _ = torch.frexp(s)
            assert bool((m == 0.5).all())
    c, s = ref.quantize(x, elem, tile=True)
    ct, st = ref.quantize(x.T, elem, tile=True)
    assert torch.equal(s.T, st) and torch.equal(c[:, :300].T, ct[:, :5])


def test_route_by_hand():
    z = torch.tensor([[0.0, 1.0, 1.0], [2.0, float("-inf"), float("-inf")], [float("-inf")] * 3, [5.0, 6.0, 7.0]])
    r = ref.route(z, 2, True, torch.tensor([True, True, True, False]))
    assert r["experts"].tolist() == [[1, 2], [0, -1], [-1, -1], [-1, -1]]
    assert r["shares"].tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0], [0.0, 0.0]]
    assert r["counts"].tolist() == [1, 1, 1] and r["order"].tolist() == [2, 0, 1, -1, -1, -1, -1, -1]
    assert abs(float(r["loss"]) - 3 * (1 / 6) * (2 / 3)) < 1e-12      # f = 1/6 each, P sums to 2/3


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_is_autograds(renorm):
    g = torch.Generator().manual_seed(2)
    z = torch.randn((7, 9), generator=g, dtype=torch.float64, requires_grad=True)
    c = torch.randn((7, 3), generator=g, dtype=torch.float64)
    up = torch.tensor(0.3)
    r = ref.route(z.detach(), 3, renorm, None, c, up)
    p = torch.softmax(z, 1)
    s = torch.gather(p, 1, r["experts"])
    s = s / s.sum(1, keepdim=True) if renorm else s
    ((s * c).sum() + float(up) * (r["slope"] * p.sum(0)).sum()).backward()
    assert torch.allclose(z.grad, r["d"], rtol=1e-10, atol=1e-12)
