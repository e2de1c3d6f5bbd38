"""The gradients of low-rank adapters from the calls for experts: rows sorted by adapter, grouped products, their weight
gradient, and the weighted copies back. For C = A B + scale[a] (A down_a) up_a, of C's gradient D:

    h = A down_a,  Ds = scale[a] D,  dh = Ds up_a,
    d up_a = sum over its rows of Ds h^T,  d down_a = sum of dh A^T,  d A (the adapters' part) = dh down_a

h, Ds and dh are rounded to BF16 (H = 2^-8 of each). Bounds: every rounding is H of its terms' magnitudes, and passes
through the sums after it; FP32 sums of n terms are n U.
"""
import numpy as np
import pytest
import torch

import dense_gemm_09_amd as g

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8


def gradients(a, d, ids, down, up, scale):
    """a: M x K, d: M x N, ids: INT32[M] (outside [0, G): none), down: G x R x K, up: G x N x R, scale: FP32[G]."""
    (M, K), N, (G, R, _) = a.shape, d.shape[1], down.shape
    new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, device=a.device, dtype=dtype)  # noqa: E731
    offsets, position = new(G + 1, dtype=torch.int32), new(M, dtype=torch.int32)
    g.route_order(M, G, ids, offsets, position)
    rows, ds, h, dh, back = new(M, K), new(M, N), new(M, R), new(M, R), new(M, K)
    g.dispatch_rows(M, 1, M, K, a, K, 2, position, rows, K)
    weight = scale[ids.clamp(0, G - 1).long()]
    g.combine_rows_grad(M, 1, M, N, d, N, g.OUT_BF16, None, N, g.OUT_BF16, position, weight, ds, N)
    g.gemm_grouped_bf16(G, M, R, K, 1.0, rows, K, offsets, down, K, g.COL, R * K, 0.0, h, R, g.OUT_BF16)
    g.gemm_grouped_bf16(G, M, R, N, 1.0, ds, N, offsets, up, R, g.ROW, N * R, 0.0, dh, R, g.OUT_BF16)
    dup, ddown = new(G, N, R, dtype=torch.float32), new(G, R, K, dtype=torch.float32)
    g.gemm_grouped_bf16_wgrad(G, M, N, R, 1.0, ds, N, h, R, offsets, 0.0, dup, R, N * R, g.OUT_F32)
    g.gemm_grouped_bf16_wgrad(G, M, R, K, 1.0, dh, R, rows, K, offsets, 0.0, ddown, K, R * K, g.OUT_F32)
    g.gemm_grouped_bf16(G, M, K, R, 1.0, dh, R, offsets, down, K, g.ROW, R * K, 0.0, back, K, g.OUT_BF16)
    da = new(M, K, dtype=torch.float32)
    g.combine_rows(M, 1, M, K, back, K, g.OUT_BF16, position, None, 0.0, da, K, g.OUT_F32)
    return dup, ddown, da


def problem(M, N, K, G, R):
    gen = torch.Generator().manual_seed(M)
    rand = lambda *s: torch.randn(*s, generator=gen).bfloat16()  # noqa: E731
    ids = torch.randint(-1, G + 1, (M,), generator=gen, dtype=torch.int32)
    ids[ids == 1] = 0  # an adapter without rows
    return rand(M, K), rand(M, N), ids, rand(G, R, K), rand(G, N, R), torch.rand(G, generator=gen) + 0.5


@pytest.mark.parametrize("M,N,K,G,R", [(1, 64, 64, 2, 8), (70, 96, 128, 5, 16), (513, 264, 520, 9, 24), (300, 512, 256, 40, 64)])
def test_gradients(M, N, K, G, R):
    args = problem(M, N, K, G, R)
    dup, ddown, da = (t.cpu().double().numpy() for t in gradients(*(t.cuda() for t in args)))
    a, d, ids, down, up, s = (t.double().numpy() for t in args)
    n = (M + N + K + R + 40) * U
    for i in range(G):
        r = ids == i
        h, dh = a[r] @ down[i].T, (s[i] * d[r]) @ up[i]
        hm, dhm = np.abs(a[r]) @ np.abs(down[i]).T, (s[i] * np.abs(d[r])) @ np.abs(up[i])
        want, mass = (s[i] * d[r]).T @ h, (s[i] * np.abs(d[r])).T @ hm
        assert (np.abs(dup[i] - want) <= ((1 + H) ** 2 - 1 + n) * mass + 1e-30).all(), i
        want, mass = dh.T @ a[r], dhm.T @ np.abs(a[r])
        assert (np.abs(ddown[i] - want) <= ((1 + H) ** 2 - 1 + n) * mass + 1e-30).all(), i
        want, mass = dh @ down[i], dhm @ np.abs(down[i])
        assert (np.abs(da[r] - want) <= ((1 + H) ** 3 - 1 + n) * mass + 1e-30).all(), i
    assert (da[(ids < 0) | (ids >= G)] == 0).all()


def test_against_differences():
    """Central differences of the definition in 64 bits along random directions: the loss sum(C * D) is linear in each
    of the arguments alone, so that they are exact; the gradients' bounds summed over the direction."""
    args = problem(40, 64, 96, 3, 16)
    dup, ddown, da = (t.cpu().double() for t in gradients(*(t.cuda() for t in args)))
    a, d, ids, down, up, s = (t.double() for t in args)
    n = 400 * U

    def loss(a, down, up):
        total = 0.0
        for m, i in enumerate(args[2].tolist()):
            if 0 <= i < 3:
                total = total + s[i] * ((up[i] @ (down[i] @ a[m])) * d[m]).sum()
        return total
    gen = torch.Generator().manual_seed(0)
    for name, grad, H_ in (("up", dup, 2), ("down", ddown, 2), ("a", da, 3)):
        v = {"a": a, "down": down, "up": up}
        direction = torch.randn(v[name].shape, generator=gen, dtype=torch.float64)
        hi, lo = dict(v), dict(v)
        hi[name], lo[name] = v[name] + direction, v[name] - direction
        diff = (loss(**hi) - loss(**lo)) / 2
        size = dict((k, t.abs()) for k, t in v.items())
        size[name] = direction.abs()
        mass = sum(s[i] * ((size["up"][i] @ (size["down"][i] @ size["a"][m])) * d[m].abs()).sum()
                   for m, i in enumerate(args[2].tolist()) if 0 <= i < 3)
        assert abs((grad * direction).sum() - diff) <= ((1 + H) ** H_ - 1 + n) * mass, name
