"""fp32 dl_decode_attn within the bounds of its own arithmetic
(tests/fp32_bounds.py): ordinary rows, a sink's logit near 35, and logits of 8000
that differ by a few, where fp32 dot products would be off by 1e-3."""
import numpy as np
import pytest
import torch

import long_context_diffusion_b200 as dl
from long_context_diffusion_b200 import pipeline
from tests.fp32_bounds import U, decode_bounds, far_rows
from tests.helpers import np_
from tests.test_gpu_token_step import _desc, _table

pytestmark = pytest.mark.gpu


# query heads per KV head (blocks of two, four, eight rows; several), d, capacity, lengths
@pytest.mark.parametrize("level", [0, 35, 8000])
@pytest.mark.parametrize("per_head", [True, False])
@pytest.mark.parametrize("G,d,L,lens", [
    (1, 128, 200, [200, 33, 64]), (4, 64, 130, [130, 65]), (3, 128, 257, [257, 100]), (8, 128, 100, [97, 31]),
    (7, 64, 200, [200, 129]), (11, 64, 90, [90, 40]),
    (1, 64, 3000, [2900, 70]), (4, 128, 2500, [2500, 200]), (6, 128, 2100, [2049, 64]), (2, 64, 5000, [1000, 320]),
])
def test_fp32_attention_keeps_to_its_arithmetic(G, d, L, lens, per_head, level, cuda_device):
    H_kv, B, dev = 2, len(lens), cuda_device
    n_mass = H_kv if per_head else 1
    desc = _desc(B, G * H_kv, H_kv, d, L, "fp32")
    table = _table(99000 + L + d, B, desc.n_pages, desc.n_slots)
    rng = np.random.default_rng([G, d, L, level])
    Q = np.zeros((B, G * H_kv, d), np.float32)
    K, V = (np.full((desc.n_slots, H_kv, 64, d), np.nan, np.float32) for _ in range(2))
    rows = {}
    for b, n in enumerate(lens):
        t = np.arange(n)
        slot = np_(table)[b].astype(int)[t // 64]
        for g in range(H_kv):
            if level == 8000:
                q, k, v = far_rows(rng, G, n, d, level)
            else:
                q, k, v = (rng.normal(size=s).astype(np.float32) for s in ((G, d), (n, d), (n, d)))
                if level:  # one key near the first query's direction
                    k[n // 2] = q[0] * np.float32(level * np.sqrt(d) / (q[0] @ q[0]))
            Q[b, g * G:(g + 1) * G] = q
            K[slot, g, t % 64], V[slot, g, t % 64] = k, v
            rows[b, g] = decode_bounds(*(x.astype(np.float64) for x in (q, k, v)))
    mass0 = rng.random((B, n_mass, L)).astype(np.float32)
    put = lambda x: torch.from_numpy(x).to(dev)  # noqa: E731
    O, lse = torch.empty(B, G * H_kv, d, device=dev), torch.empty(B, G * H_kv, device=dev)
    mass = put(mass0)
    dl.dl_decode_attn(desc, put(Q), put(K), put(V), table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), O, lse,
                      pipeline.workspace(desc, dev), tok_mass=mass, decay=0.5)
    assert dl.dl_get_status() == dl.DL_OK
    worst = {}
    for b, n in enumerate(lens):
        add, tol = np.zeros((n_mass, n)), np.zeros((n_mass, n))
        for g in range(H_kv):
            h = slice(g * G, (g + 1) * G)
            (o, s, w), (to, ts, tw) = rows[b, g]
            for name, got, ref, t in (("O", O[b, h], o, to), ("lse", lse[b, h], s, ts)):
                worst[name] = max(worst.get(name, 0), float((np.abs(np_(got) - ref) / t).max()))
            add[g if per_head else 0] += w.sum(0)
            tol[g if per_head else 0] += tw.sum(0)
        ref = 0.5 * mass0[b, :, :n].astype(np.float64) + add
        t = tol + (G * H_kv // n_mass + 3) * U * ref
        worst["mass"] = max(worst.get("mass", 0), float((np.abs(np_(mass)[b, :, :n] - ref) / t).max()))
        assert np.array_equal(np_(mass)[b, :, n:], mass0[b, :, n:])
    assert max(worst.values()) <= 1.0, worst
