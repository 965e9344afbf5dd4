"""dl_decode_attn at the ends of its ranges: hundreds of sequences, a cache of
millions of tokens, the largest capacity, and a first call that is captured."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import long_context_diffusion_b200 as dl
import synth
from long_context_diffusion_b200 import pipeline
from tests.helpers import np_
from tests.test_gpu_token_step import DT, SEED, U, _cache, _check_decode, _desc, _near, _normal, _table

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype,d,H,H_kv,n_mass,B", [
    ("bf16", 64, 2, 1, 1, 700), ("fp32", 64, 2, 2, 2, 450), ("bf16", 128, 6, 2, 1, 333), ("fp32", 128, 3, 1, 1, 90),
])
def test_hundreds_of_sequences(dtype, d, H, H_kv, n_mass, B, cuda_device):
    """More sequences than lanes that look them up, most of them short."""
    L, dt, sid = 150, DT[dtype], 100000 + B
    u = np_(synth.uniforms(SEED, sid + 995, 0, B))
    lens = [0 if x < 0.1 else 1 if x < 0.2 else int(x ** 3 * (L + 1)) for x in u]
    K, V, table = _cache(sid, B, H_kv, d, lens, L, dt)
    desc = _desc(B, H, H_kv, d, L, dtype, n_slots=K.shape[0])
    Q = _normal(sid + 990, B, H, d, dtype=dt)
    mass0 = synth.uniforms(SEED, sid + 991, 0, B * n_mass * L).reshape(B, n_mass, L).float()
    put = lambda t: t.to(cuda_device)  # noqa: E731
    mass = put(mass0)
    O, lse = torch.empty(B, H, d, dtype=dt, device=cuda_device), torch.empty(B, H, device=cuda_device)
    dl.dl_decode_attn(desc, put(Q), put(K), put(V), put(table), put(torch.tensor(lens, dtype=torch.int32)), O, lse,
                      pipeline.workspace(desc, cuda_device), tok_mass=mass, decay=0.5)
    assert dl.dl_get_status() == dl.DL_OK
    _check_decode(Q, K, V, table, lens, O, lse, mass0, mass, 0.5, dtype, H_kv, n_mass)


def test_a_cache_of_millions_of_tokens(cuda_device):
    """Nine million tokens, masses of two heads shared: more chunks of masses than
    CTAs take them.  Reference in fp64 on the device; values positive, so that O
    keeps its size.  Sums: 475 tiles a run, 16 terms each to O (a whole step a
    term, as in test_gpu_token_step.py), then runs, warps and lanes: 300."""
    dev, d, H, n, L = cuda_device, 64, 2, 9_000_001, 9_000_200
    desc = _desc(1, H, 1, d, L, "bf16")
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    K, V = (torch.empty(desc.n_slots, 1, 64, d, dtype=torch.bfloat16, device=dev).normal_(generator=g) for _ in range(2))
    V.abs_()
    Q = torch.empty(1, H, d, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    table = torch.randperm(desc.n_slots, generator=g, device=dev).to(torch.int32)[None]
    mass0 = torch.rand(1, 1, L, generator=g, device=dev)
    mass, O, lse = mass0.clone(), torch.empty(1, H, d, dtype=torch.bfloat16, device=dev), torch.empty(1, H, device=dev)
    dl.dl_decode_attn(desc, Q, K, V, table, torch.tensor([n], dtype=torch.int32, device=dev), O, lse,
                      pipeline.workspace(desc, dev), tok_mass=mass, decay=0.5)
    assert dl.dl_get_status() == dl.DL_OK
    k, v = (P[table[0].long()].reshape(-1, d)[:n].double() for P in (K, V))
    a = Q[0].double() @ k.T / d ** 0.5
    ref_lse = torch.logsumexp(a, 1)
    w = torch.exp(a - ref_lse[:, None])
    ref = w @ v
    delta = (2 * d + 8) * U * float(Q.double().norm(dim=-1).max() * k.norm(dim=1).max()) / d ** 0.5
    eps_w = 2 * delta + (475 * 2 + 300 + 64) * U + 2.0 ** -16
    tol = ref * (2 * eps_w + 475 * 32 * U)
    _near(np_(O[0]), np_(ref), np_(tol + 2.0 ** -8 * (ref + tol)), "O")
    _near(np_(lse[0]), np_(ref_lse), delta + 1314 * U + 4 * U * np_(ref_lse), "lse")
    add = w.sum(0)
    want = 0.5 * mass0[0, 0, :n].double() + add
    assert ((mass[0, 0, :n] - want).abs() <= 2 * eps_w * add + 4 * U * want).all()
    assert torch.equal(mass[0, 0, n:], mass0[0, 0, n:])


def test_the_largest_capacity(cuda_device):
    """Room for 2^30 tokens a sequence, of which a few are there."""
    B, H, H_kv, d, L, lens = 2, 4, 2, 64, 1 << 30, [130, 1]
    K, V, table = _cache(102000, B, H_kv, d, lens, 130, torch.bfloat16)
    desc = dl.make_desc(B, H, H_kv, d, L, 1, 64, L // 64, K.shape[0], torch.bfloat16)
    wide = torch.full((B, desc.n_pages), -1, dtype=torch.int32, device=cuda_device)
    wide[:, :table.shape[1]] = table.to(cuda_device)
    Q = _normal(102990, B, H, d, dtype=torch.bfloat16)
    O, lse = torch.empty(B, H, d, dtype=torch.bfloat16, device=cuda_device), torch.empty(B, H, device=cuda_device)
    ws = torch.empty(dl.dl_decode_workspace_size(desc, False), dtype=torch.uint8, device=cuda_device)
    dl.dl_decode_attn(desc, Q.to(cuda_device), K.to(cuda_device), V.to(cuda_device), wide,
                      torch.tensor(lens, dtype=torch.int32, device=cuda_device), O, lse, ws)
    assert dl.dl_get_status() == dl.DL_OK
    _check_decode(Q, K, V, table, lens, O, lse, None, None, 1.0, "bf16", H_kv, 0)


FIRST = """
import torch
import long_context_diffusion_b200 as dl
from long_context_diffusion_b200 import pipeline
dev = torch.device("cuda:0")
B, H, H_kv, d, L = 2, 4, 2, 64, 300
desc = dl.make_desc(B, H, H_kv, d, L, 1, 64, 5, 10, torch.bfloat16)
step = pipeline.TokenStep(desc, 1, torch.bfloat16, dev, budget=100)
pools = [torch.zeros(10, H_kv, 64, d, dtype=torch.bfloat16, device=dev) for _ in range(2)]
table = torch.arange(10, dtype=torch.int32, device=dev).reshape(B, 5)
x = torch.ones(B, 1, (H + 2 * H_kv) * d, dtype=torch.bfloat16, device=dev)
pos = torch.zeros(B, 1, dtype=torch.int32, device=dev)
step.start.fill_(200)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    O = step.attend(0, x, pos, None, None, *pools, table)
    step.evict(pools[:1], pools[1:], table)
g.replay()
assert dl.dl_get_status() == 0 and step.start.tolist() == [100, 100]
assert torch.allclose(step.lse[0].exp(), torch.full_like(step.lse[0], 200.0) + torch.tensor(8.0).exp().item(), rtol=1e-3)
"""


def test_the_first_calls_of_a_process_may_be_captured(cuda_device):
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("L,lens", [(100, [100]), (3300, [3201])])
def test_thousands_of_heads_of_one_group(dtype, L, lens, cuda_device):
    H, d, dt = 2500, 64, DT[dtype]
    K, V, table = _cache(103000 + L, 1, 1, d, lens, L, dt)
    desc = _desc(1, H, 1, d, L, dtype, n_slots=K.shape[0])
    Q = _normal(103990 + L, 1, H, d, dtype=dt)
    mass0 = torch.full((1, 1, L), 0.5)
    put = lambda t: t.to(cuda_device)  # noqa: E731
    mass = put(mass0)
    O, lse = torch.empty(1, H, d, dtype=dt, device=cuda_device), torch.empty(1, H, device=cuda_device)
    dl.dl_decode_attn(desc, put(Q), put(K), put(V), put(table), put(torch.tensor(lens, dtype=torch.int32)), O, lse,
                      pipeline.workspace(desc, cuda_device), tok_mass=mass, decay=0.5)
    assert dl.dl_get_status() == dl.DL_OK
    # a mass adds 2500 weights in turn: one rounding each of the sum so far, beside the weights' own
    n = lens[0]
    m = mass[0, 0, :n].double().cpu() - 0.25
    _check_decode(Q, K, V, table, lens, O, lse, None, None, 0.5, dtype, 1, 0)
    k = K[table[0].long()].reshape(-1, d)[:n].double()
    w = torch.softmax(Q[0].double() @ k.T / d ** 0.5, 1).sum(0)
    delta = (2 * d + 8) * U * float(Q.double().norm(dim=-1).max() * k.norm(dim=1).max()) / d ** 0.5
    eps_w = 2 * delta + (n + 64) * U + (2.0 ** -16 if dtype == "bf16" else 0.0)
    assert ((m - w).abs() <= 2 * eps_w * w + (H + 4) * U * (w + 0.25)).all()
    assert (mass[0, 0, n:] == 0.5).all()
