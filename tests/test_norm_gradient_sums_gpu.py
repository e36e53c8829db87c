"""The weight's gradient of the norm over many rows, within the roundings that its
sums make: those of a lane's rows, of the rows side by side in a wave, of the
workgroup's waves and of the workgroups' parts."""
import pytest
import torch

from mxfp4_weight_mixture_02_amd import rms_norm, rms_norm_backward

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _additions(T, H):
    """Of one element: as the launch splits T rows of H."""
    w = -(-H // 512)
    lanes = (16 if H <= 128 else 32 if H <= 256 else 64) if w <= 2 else 256 if w <= 8 else 512 if w <= 16 else 1024
    block = max(lanes, 256)
    groups = -(-T // (block // lanes))
    third = max(256, min(groups // 3, 4 * 65536 // block))
    parts = min(groups, third)
    rows = -(-groups // parts)
    waves = 3 if block > lanes else 0
    in_wave = {16: 2, 32: 1}.get(lanes, 0)
    return rows + in_wave + waves + (-(-parts // 16) + 15 if parts > 1 else 0)


def test_additions():
    assert _additions(1, 2880) == 1
    # 512 workgroups of 512 lanes: 2049 rows each, slices of 32 parts, 15 joins
    assert _additions(1048700, 4200) == 2049 + 32 + 15
    # 341 workgroups of 256 lanes: 4 rows, slices of 22
    assert _additions(1024, 2880) == 4 + 22 + 15


@pytest.mark.parametrize("T,H", [(1, 64), (17, 100), (700, 2880), (1024, 2880), (16384, 2880), (1 << 20, 64), (600001, 200),
                                 (400000, 1000), (262200, 4200), (60001, 9000), (30000, 20000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weight_gradient(T, H, dtype):
    print("sums", T, H, dtype, flush=True)
    g = torch.Generator(device=DEV).manual_seed(T + H)
    x = torch.empty(T, H, dtype=dtype, device=DEV).normal_(generator=g)
    dy = torch.empty(T, H, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    w = torch.rand(H, generator=g, device=DEV) + 0.5
    rstd = rms_norm(x, w).rstd
    _, dw = rms_norm_backward(dy, x, rstd, w)
    want, size = torch.zeros(2, H, dtype=torch.float64, device=DEV)
    for a in range(0, T, 1 << 15):
        b = a + (1 << 15)
        t = dy[a:b].double() * (x[a:b].double() * rstd[a:b, None].double())
        want += t.sum(0)
        size += t.abs().sum(0)
    # two roundings a term
    assert torch.all((dw.double() - want).abs() <= (2 + _additions(T, H)) * 2.0 ** -24 * size)
