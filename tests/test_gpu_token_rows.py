"""Masses that more than 64 query heads share (the join kernel takes 64 at a
time), on clusters and on runs.  Tolerances: those of test_gpu_token_step.py."""
import pytest
import torch

import long_context_diffusion_b200 as dl
import synth
from long_context_diffusion_b200 import pipeline
from tests.test_gpu_token_step import DT, SEED, _cache, _check_decode, _desc, _normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("decay", [0.0, 0.5])
@pytest.mark.parametrize("L,lens", [(200, [200, 1]), (5000, [4999, 0, 66])])
@pytest.mark.parametrize("H,H_kv", [(65, 5), (65, 65), (128, 8), (224, 32)])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 64)])
def test_masses_of_many_shared_heads(dtype, d, H, H_kv, L, lens, decay, cuda_device):
    B, dt, sid = len(lens), DT[dtype], 90000 + H
    K, V, table = _cache(sid, B, H_kv, d, lens, L, dt)
    desc = _desc(B, H, H_kv, d, L, dtype, n_slots=K.shape[0])
    Q = _normal(sid + 990, B, H, d, dtype=dt)
    mass0 = synth.uniforms(SEED, sid + 991, 0, B * L).reshape(B, 1, L).float()
    if decay == 0:
        mass0[:] = float("nan")  # not read
    for b, n in enumerate(lens):
        mass0[b, :, n:] = -4.0
    dev = lambda t: t.to(cuda_device)  # noqa: E731
    mass = dev(mass0)
    O, lse = torch.empty(B, H, d, dtype=dt, device=cuda_device), torch.empty(B, H, device=cuda_device)
    dl.dl_decode_attn(desc, dev(Q), dev(K), dev(V), dev(table), dev(torch.tensor(lens, dtype=torch.int32)), O, lse,
                      pipeline.workspace(desc, cuda_device), tok_mass=mass, decay=decay)
    assert dl.dl_get_status() == dl.DL_OK
    _check_decode(Q, K, V, table, lens, O, lse, mass0, mass, decay, dtype, H_kv, 1)
