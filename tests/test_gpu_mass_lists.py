"""kev_attn_mass_paged with more questions times kv heads than a grid has CTAs."""
import pytest
import torch

import packed_question_isolated_gb300 as kev

pytestmark = pytest.mark.gpu


def test_more_lists_than_a_grid_holds():
    """4096 questions, one of them with a token, times 2^19 kv heads; keys of zeros, so every weight is 1 / 3 (off by the log
    sum's last place, the exponent's and the exponential's: less than 8 2^-24 relative, log2 3 being below 2)."""
    n, h, d = 4096, 1 << 19, 64
    lens = torch.zeros(n, dtype=torch.int32)
    lens[1000] = 1
    end = lens.cumsum(0).int()
    iv = torch.stack([end - lens, end], 1).int().cuda()
    prefix = torch.full((n,), 2, dtype=torch.int32, device="cuda")
    k = torch.zeros(1, h, 128, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scale = torch.zeros(1, h, 128, device="cuda")
    table = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    mass = torch.full((1, h, 128), 4.0, device="cuda")
    q = torch.ones(1, h, d, dtype=torch.bfloat16, device="cuda")
    shape = kev.make_shape(h, h, d, "bf16")
    cache = kev.make_paged_cache(k, k, table, 1, 1, "e4m3", scale, scale)
    size = kev.kev_attn_mass_workspace_size(n, 1, shape)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    kev.kev_attn_mass_paged(q, 1, iv, n, prefix, 1, cache, 0.5, mass, shape, ws, size, status)
    assert kev.kev_read_status(status) == 0
    third = 1 / 3
    assert (mass[0, :, :2] - (2 + third)).abs().max() < 3 * 2.0 ** -22
    assert (mass[0, :, 2] - third).abs().max() < 8 * 2.0 ** -24
    assert (mass[0, :, 3:] == 4).all()
