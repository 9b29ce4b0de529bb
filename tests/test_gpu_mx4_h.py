"""How the grouped FFN rounds h: by the format's own operations, as mx4.quantize rounds any other rows."""
import pytest
import torch

import mx4_reference as ref
from mixture_experts_layer_29_b200 import abi, mx4

pytestmark = pytest.mark.gpu


def borders(n, seed):
    """Multiples u of h's factor n, 512 of them: blocks of 16 whose scale is a multiple of four, 8 to 15
    times, or lies half way between two of them, and elements half way between two 4-bit numbers."""
    g = torch.Generator().manual_seed(seed)
    mid = torch.tensor([1, 3, 5, 7, 10, 14, 20])                       # in quarters
    rows = []
    for m in range(8, 16):
        ties = mid * m * n
        rows.append(torch.cat([torch.tensor([24 * m * n]), ties, ties + 1, torch.tensor([0])]))
        rows.append(torch.cat([torch.tensor([n * (24 * m + 12)]), torch.randint(0, 24 * m * n, (15,), generator=g)]))
    u = torch.stack(rows).flatten()
    return torch.cat([u, torch.randint(0, 24 * 15 * n, (512 - u.numel(),), generator=g)])


@pytest.mark.parametrize("fmt,n", [("mxfp4", 3), ("nvfp4", 3), ("nvfp4", 5), ("nvfp4", 9), ("nvfp4", 11)])
@pytest.mark.parametrize("rows", [40, 300])                     # one CTA per tile, and CTA pairs
def test_h_is_rounded_by_the_formats_operations(cuda_device, fmt, n, rows):
    """A row of x has a 4.0 at the start of each 32 elements; Wg turns it into G = 32, where silu(G) is G in
    fp32, and Wu into the numbers above, one binary digit per 32. So h = 32 x 4 u exactly, much of it on a
    border: rounded after other operations than the format's, some of it goes the other way. Wd is the
    identity: y is what h was rounded to."""
    K, inter, B = 512, 512, ref.BLOCK[fmt]
    u = borders(n, rows).cuda()
    sign = torch.where(torch.arange(inter, device="cuda") % 3 == 1, 8, 0)
    code = torch.zeros(1, 2 * inter, K, device="cuda", dtype=torch.uint8)
    e = torch.zeros(1, 2 * inter, K // B, device="cuda", dtype=torch.int64)
    code[0, :inter, 0] = 2                                             # 1.0
    e[0, :inter, 0] = 3
    assert int(u.max()) < 2 ** 13
    for b in range(13):                    # 2^b; e4m3 ends at 448, so from 2^8 on x brings 16 of it
        code[0, inter:, 32 * b] = (((u >> b) & 1) * (2 + sign)).to(torch.uint8)
        e[0, inter:, 32 * b // B] = b if b < 8 else b - 4

    def byte_of(e):
        return (e + 127 if fmt == "mxfp4" else (e + 7) << 3).to(torch.uint8)

    w = mx4.from_checkpoint(fmt, ref.pack(code), byte_of(e))
    eye = torch.eye(inter, device="cuda", dtype=torch.uint8)[None] * 2
    down = mx4.from_checkpoint(fmt, ref.pack(eye), byte_of(torch.zeros(1, inter, inter // B, device="cuda", dtype=torch.int64)))
    x = torch.zeros(rows, K, device="cuda", dtype=torch.uint8)
    x[:, ::32] = 6
    a = mx4.allocate(fmt, rows, K)
    a.codes.copy_(ref.pack(x))
    xe = torch.where(torch.arange(K // B) < 8 * 32 // B, 0, 4).expand(rows, -1)
    a.scales[ref.scale_index([0, rows], K, fmt, "cuda")] = byte_of(xe).cuda()
    t = torch.full((1,), 128.0 * n, device="cuda") if fmt == "nvfp4" else None
    ws = mx4.ffn_workspace(a, w)
    y = mx4.grouped_ffn(a, w, down, torch.empty(rows, K, device="cuda"), ws, t)
    assert abi.read_device_status(ws) == 0
    h = 128.0 * u.float() * torch.where(sign > 0, -1.0, 1.0)
    hcode, hbyte, want = ref.quantize(h, fmt, 1.0 if t is None else t)
    if fmt == "nvfp4":      # element times e4m3 scale, exact, then times the factor, one fp32 rounding
        v = ref.GRID.cuda()[(hcode & 7).long()] * torch.where(hcode > 7, -1.0, 1.0)
        want = ((v * hbyte.view(torch.float8_e4m3fn).double().repeat_interleave(B, -1)).float() * t).double()
    assert torch.equal(y.double(), want.expand(rows, -1))
