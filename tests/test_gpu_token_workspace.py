"""dl_decode_attn keeps to the workspace that dl_decode_workspace_size names,
and TokenStep without a budget runs on the smaller one."""
import pytest
import torch

import long_context_diffusion_b200 as dl
from tests.test_gpu_token_step import DT, _cache, _check_decode, _desc, _normal, _token_model

pytestmark = pytest.mark.gpu

GUARD = 1 << 16


@pytest.mark.parametrize("masses", [True, False])
@pytest.mark.parametrize("dtype,d,G,H_kv,L,lens", [
    ("bf16", 128, 20, 2, 5000, [5000, 77]), ("fp32", 64, 9, 2, 4100, [64, 4100]), ("bf16", 64, 2, 2, 300, [300, 0]),
    ("fp32", 128, 1, 3, 200, [200, 199]),
])
def test_nothing_behind_the_stated_size_is_written(dtype, d, G, H_kv, L, lens, masses, cuda_device):
    B, dt, dev = len(lens), DT[dtype], cuda_device
    K, V, table = _cache(95000 + L, B, H_kv, d, lens, L, dt)
    desc = _desc(B, G * H_kv, H_kv, d, L, dtype, n_slots=K.shape[0])
    Q = _normal(95990 + L, B, G * H_kv, d, dtype=dt)
    n = dl.dl_decode_workspace_size(desc, masses)
    buf = torch.full((n + GUARD,), 0xA5, dtype=torch.uint8, device=dev)
    O, lse = torch.empty(B, G * H_kv, d, dtype=dt, device=dev), torch.empty(B, G * H_kv, device=dev)
    mass0 = torch.full((B, H_kv, L), 0.5)
    mass = mass0.to(dev) if masses else None
    dl.dl_decode_attn(desc, Q.to(dev), K.to(dev), V.to(dev), table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                      O, lse, buf[:n], tok_mass=mass, decay=0.5)
    assert dl.dl_get_status() == dl.DL_OK and (buf[n:] == 0xA5).all()
    _check_decode(Q, K, V, table, lens, O, lse, mass0, mass, 0.5, dtype, H_kv, H_kv if masses else 0)
    with pytest.raises(dl.DLError) as e:
        dl.dl_decode_attn(desc, Q.to(dev), K.to(dev), V.to(dev), table.to(dev),
                          torch.tensor(lens, dtype=torch.int32, device=dev), O, lse, buf[:n - 1], tok_mass=mass)
    assert e.value.status == dl.DL_ERR_WORKSPACE


def test_token_step_without_a_budget(cuda_device):
    B, H, H_kv, d = 3, 6, 2, 64
    desc, step, table, pools, w = _token_model(cuda_device, layers=1, budget=0)
    n0, width = 70, (H + 2 * H_kv) * d
    x = _normal(96000, B, n0, width, dtype=torch.bfloat16).to(cuda_device)
    pos = torch.arange(n0, dtype=torch.int32, device=cuda_device).expand(B, n0).contiguous()
    step.append(0, x, pos, *w[0], *pools[0], table, torch.empty(B, H, n0, d, dtype=torch.bfloat16, device=cuda_device))
    step.advance()
    for i in range(3):
        step.attend(0, x[:, i:i + 1].contiguous(), pos[:, :1] + (n0 + i), *w[0], *pools[0], table)
        step.advance()
    assert dl.dl_get_status() == dl.DL_OK and step.start.tolist() == [n0 + 3] * B
    _check_decode(step.Q[:, :, 0].cpu(), pools[0][0].cpu(), pools[0][1].cpu(), table.cpu(), [n0 + 3] * B, step.O[0],
                  step.lse[0], None, None, 1.0, "bf16", H_kv, 0)
