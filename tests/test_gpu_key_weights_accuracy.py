"""How near lat_attn_key_weights comes to its definition: the size of its error beside the sums'.

Tolerance, as a part of the weights (Frobenius).  A pair's weight 2^(s' - lse') is off by ln 2 times what its
exponent is, which is at most
  * bf16: after each 16 channels the tensor pipe cuts its sum off, by 2^-22 of the largest number in
    it (the sums before and after, the products), times scale * log2(e);
    fp32: a sum's D roundings, without a common sign, 2^-24 sqrt(D) of |q.k| + |products|_2 together;
  * the roundings of the constant, the product, log2(e) lse and the difference: 2^-24 (2 |s'| + 2 |lse'|);
  * capped: bf16, four roundings of the score over the cap and its square, and the polynomial's 4e-8 of
    the score (5e-8 from 0.15 of the cap to 0.3); beyond, 3e-7 of the cap (1 - 2 / (1 + e^2y) has two
    fp32 operations on numbers up to it, and an exponential); fp32, tanh to 2^-22 of itself.
The exponential is off by 2^-22, and a key's sum of c columns, in chains of 32, by 2^-24 sqrt(min(c, 32))
and two more roundings.  The weights that the test adds onto are zero.
"""
import math

import pytest
import torch

from gpu_helpers import ensure_library
from test_gpu_key_weights import inputs, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    ensure_library()


# (D, Hq, Hkv, n_q, keys): a decode step, a window, a prompt's rows
SHAPES = [(D, 4, 2, 1, 20000) for D in (64, 80, 128, 256, 512)] + [
    (64, 8, 1, 1, 6000), (128, 4, 1, 40, 5000), (64, 4, 1, 300, 4000), (128, 2, 1, 300, 2000), (256, 2, 1, 200, 1500),
    (512, 2, 1, 140, 1000)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "D%dH%d-%dq%dL%d" % s)
@pytest.mark.parametrize("cap", [0.0, 50.0, 20.0, 6.0])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_the_size_of_the_error(shape, cap, dt):
    D, Hq, Hkv, n_q, n = shape
    G, scale, log2e = Hq // Hkv, D ** -0.5, math.log2(math.e)
    q, k = inputs(1, Hq, Hkv, D, n, n_q, dt, 77 + D)
    k = k.contiguous()
    pos = torch.arange(n - n_q, n, device="cuda")[:, None]
    seen = torch.arange(n, device="cuda")[None] <= pos
    lse = torch.empty(1, n_q, Hq, device="cuda")
    want, off = (torch.zeros(Hkv, n, dtype=torch.float64, device="cuda") for _ in range(2))
    for h in range(Hq):
        qh, kh = q[:, h * D:(h + 1) * D].double(), k[0, :, h // G].double()
        for i0 in range(0, n_q, 20):
            rows = slice(i0, min(n_q, i0 + 20))
            x = qh[rows, None] * kh[None]  # rows, keys, D
            s = x.sum(-1)
            if dt == "bf16":
                parts = x.unflatten(-1, (-1, 16))
                sums = parts.sum(-1).cumsum(-1).abs()
                before = torch.cat([torch.zeros_like(sums[..., :1]), sums[..., :-1]], -1)
                d = 2.0 ** -22 * torch.maximum(torch.maximum(sums, before), parts.abs().amax(-1)).sum(-1)
            else:
                d = 2.0 ** -24 * math.sqrt(D) * (s.abs() + x.square().sum(-1).sqrt())
            del x
            s, d = scale * s, scale * log2e * d
            if cap > 0:
                y = s.abs() / cap
                s = cap * torch.tanh(s / cap)
                if dt == "bf16":
                    d = d + torch.where(y < 0.3, log2e * s.abs() * (4 * 2.0 ** -24 + 5e-8), 3e-7 * log2e * cap)
                else:
                    d = d + 2.0 ** -22 * log2e * s.abs()
            l = torch.logsumexp(torch.where(seen[rows], s, -math.inf), -1).float()
            lse[0, rows, h] = l
            l = l.double()[:, None]
            d = d + 2.0 ** -24 * log2e * (2 * s.abs() + 2 * l.abs())
            w = torch.where(seen[rows], torch.exp(s - l), 0.0)
            want[h // G] += w.sum(0)
            off[h // G] += (w * d).sum(0) * math.log(2)
    got = torch.zeros(1, Hkv, n, device="cuda")
    st = run(q, k, [n], dt, Hq, Hkv, D, n_q, lse, got, cap=cap)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    error = ((got[0].double() - want).norm() / want.norm()).item()
    bound = (off.norm() / want.norm()).item() + 2.0 ** -22 + 2.0 ** -24 * (math.sqrt(min(n_q * G, 32)) + 2)
    assert error <= bound, "%.2e of %.2e" % (error, bound)
