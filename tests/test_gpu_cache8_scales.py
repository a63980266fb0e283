"""Single-token attention over 8 bits: scales of any size."""
import pytest

from gpu_helpers import host_f64, torch_dtype

pytestmark = pytest.mark.gpu


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 192, 256, 33])
def test_zeros_of_the_largest_scales(fk, D, dtype):
    """Rows of zero codes count as zeros whatever finite scale they have; the largest codes under the smallest
    scales as what they stand for."""
    import torch
    n, H, page = 90, 2, 16
    dt = torch_dtype(dtype)
    g = torch.Generator(device="cuda").manual_seed(D)
    pages = -(-n // page)
    k = torch.randn((pages, page, H, D), device="cuda", generator=g).to(torch.float8_e4m3fn)
    v = torch.randn((pages, page, H, D), device="cuda", generator=g).to(torch.float8_e4m3fn)
    ks, vs = (torch.full((pages, page, H), 1.0, device="cuda") for _ in range(2))
    for i, s in ((3, 2.0 ** 127), (40, 2.0 ** 120), (70, 2.0 ** 114)):
        v.view(torch.uint8)[i // page, i % page] = 0
        vs[i // page, i % page] = s
        k.view(torch.uint8)[(i + 1) // page, (i + 1) % page] = 0
        ks[(i + 1) // page, (i + 1) % page] = s
    v.view(torch.uint8)[0, 7], vs[0, 7] = 0x7E, 2.0 ** -126
    q = torch.randn((1, 4, D), device="cuda", generator=g).to(dt)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    k64, v64 = (c.double().cpu().numpy() * s.double().cpu().numpy()[..., None] for c, s in ((k, ks), (v, vs)))
    import oracle
    import test_gpu_cache8 as tc
    for scale in (D ** -0.5, 3.0):
        want = oracle.paged_attn(host_f64(q, dtype), k64, v64, table.cpu().numpy(), [n], scale)
        for hint in (0, n):
            got = fk.fk_paged_attn8(q, k, v, ks, vs, table, _i32([n]), scale, max_len=hint, return_lse=True)
            tc._check_attn(got, want, dtype, D, 0.0, f"scale {scale}, max_len {hint}")
