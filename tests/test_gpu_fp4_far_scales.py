"""NV products whose two tensor scales leave fp32's range together, where the results do not."""
import pytest

pytestmark = pytest.mark.gpu


def _matrix(rows, K, values, g):
    """Row r holds values[r % len(values)] = (code, scale byte) throughout: (Fp4, what an entry stands for without g, fp64)."""
    import torch
    from block_diffusion_speculative_hidden_gb300 import Fp4
    from fp4_ref import e4m3_values, pack, tile, GRID
    at = torch.arange(rows) % len(values)
    code = torch.tensor([v[0] for v in values])[at]
    byte = torch.tensor([v[1] for v in values])[at]
    t = Fp4(pack(code[:, None].expand(rows, K)).cuda(), tile(byte[:, None].expand(rows, K // 16), "nv").cuda(), "nv",
            torch.tensor([g], dtype=torch.float32, device="cuda"))
    one = torch.tensor(GRID, dtype=torch.float64)[code] * e4m3_values()[byte]
    return t, one.cuda()


# codes and scale bytes: 0, 1/2 under the smallest step, 1 under 1, 6 under the largest one
VALUES = [(0, 126), (1, 1), (2, 56), (7, 126)]


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
# (whole vectors and not; a long k of few tiles; several tiles under pairs)
@pytest.mark.parametrize("M,N,K", [(40, 640, 64), (40, 131, 64), (16, 128, 4096), (640, 4096, 256)])
@pytest.mark.parametrize("gw,gx", [(1.37 * 2.0 ** 70, 1.61 * 2.0 ** 70), (2.0 ** 100, 2.0 ** 100), (1.37 * 2.0 ** 100, 2.0 ** 28),
                                   (1.37 * 2.0 ** -75, 1.61 * 2.0 ** -75), (2.0 ** -80, 2.0 ** -80),
                                   (1.37 * 2.0 ** -100, 1.61 * 2.0 ** -30), (1.37 * 2.0 ** -30, 1.61 * 2.0 ** -100),
                                   (2.0 ** -100, 2.0 ** -100), (1.37 * 2.0 ** -100, 1.61 * 2.0 ** 100), (0.0, 1.0)])
def test_far_scales(gw, gx, M, N, K, dt):
    import torch
    from block_diffusion_speculative_hidden_gb300 import gemm_fp4
    t = getattr(torch, dt)
    W, w = _matrix(N, K, VALUES, gw)
    X, x = _matrix(M, K, VALUES[1:] + VALUES[:1], gx)
    out = gemm_fp4(W, X, dtype=t).double()
    # sums of K equal products of at most 8 bits are exact
    ref = x[:, None] * w * K * float(W.scale.double()) * float(X.scale.double())
    assert not torch.isnan(out).any()
    assert (out[ref == 0] == 0).all()
    # Two roundings in fp32 (the scales' product and that with the sum, or the sum with one scale after the other),
    # one to the type, each by at most half a step: (1 + 2^-24)^2 - 1 < 2.01 * 2^-24; below the normal range of
    # fp32 or the type by half its smallest number each.
    f = torch.finfo(t)
    rel = 2.01 * 2.0 ** -24
    tol = ref.abs() * (rel + f.eps / 2 * (1 + rel)) + 2.0 ** -149 + f.tiny * f.eps / 2
    sure = ref.abs() * (1 + rel) < f.max
    assert ((out - ref).abs()[sure] <= tol[sure]).all()
    past = ref.abs() * (1 - rel) >= f.max * (1 + f.eps)
    assert torch.isinf(out[past]).all() and (out[past] > 0).all()
