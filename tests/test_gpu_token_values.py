"""Attention of one token with NaN and infinite entries among its live tokens:
what the formulas give where they define a value, and the documented rest.

  - a NaN dot product: the row's sum is NaN, so O, lse and every weight are;
  - one of +infinity: lse is +infinity, O and the weights are NaN;
  - one of -infinity: weight 0; if every one is, O is 0 and lse -infinity;
  - an infinite or NaN value reaches its column of O alone.
Whatever is not named so stays within the bounds of test_gpu_token_step.py."""
import numpy as np
import pytest
import torch

import long_context_diffusion_b200 as dl
from long_context_diffusion_b200 import pipeline
from tests.helpers import np_
from tests.test_gpu_token_step import DT, _cache, _check_decode, _desc, _normal

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
B, H_KV = 2, 2

# dtype, d, query heads per KV head, capacity, lengths: row blocks of every size, on
# clusters and on runs; 17 tokens leave one alone with its warp
SHAPES = [
    ("bf16", 128, 4, 200, [17, 200]),
    ("bf16", 64, 12, 200, [17, 131]),
    ("fp32", 128, 2, 200, [9, 200]),
    ("fp32", 64, 7, 200, [17, 131]),
    ("bf16", 64, 8, 9000, [9000, 17]),
    ("bf16", 128, 16, 9000, [8001, 17]),
    ("fp32", 64, 3, 9000, [5000, 17]),
    ("fp32", 128, 8, 9000, [4097, 9]),
]
IDS = ["-".join(map(str, s[:4])) for s in SHAPES]


class Case:
    def __init__(self, shape, sid):
        self.dtype, self.d, self.G, self.L, self.lens = shape
        self.dt, self.H = DT[self.dtype], self.G * H_KV
        self.K, self.V, self.table = _cache(sid, B, H_KV, self.d, self.lens, self.L, self.dt)
        self.Q = _normal(sid + 990, B, self.H, self.d, dtype=self.dt)

    def at(self, b, t):
        return int(self.table[b, t // 64]), t % 64

    def run(self, dev, per_head):
        n_mass = H_KV if per_head else 1
        desc = _desc(B, self.H, H_KV, self.d, self.L, self.dtype, n_slots=self.K.shape[0])
        self.O = torch.full((B, self.H, self.d), 5.0, dtype=self.dt, device=dev)
        self.lse = torch.full((B, self.H), 5.0, device=dev)
        self.mass0 = torch.full((B, n_mass, self.L), 0.25)
        self.mass = self.mass0.to(dev)
        dl.dl_decode_attn(desc, self.Q.to(dev), self.K.to(dev), self.V.to(dev), self.table.to(dev),
                          torch.tensor(self.lens, dtype=torch.int32, device=dev), self.O, self.lse,
                          pipeline.workspace(desc, dev), tok_mass=self.mass, decay=0.5)
        assert dl.dl_get_status() == dl.DL_OK

    def heads(self, g):
        return slice(g * self.G, (g + 1) * self.G)

    def check_kv_head(self, b, g):
        """KV head g of sequence b alone, by the oracle."""
        h = self.heads(g)
        per_head = self.mass.shape[1] > 1
        _check_decode(self.Q[b:b + 1, h], self.K[:, g:g + 1], self.V[:, g:g + 1], self.table[b:b + 1], [self.lens[b]],
                      self.O[b:b + 1, h], self.lse[b:b + 1, h], self.mass0[b:b + 1, g:g + 1] if per_head else None,
                      self.mass[b:b + 1, g:g + 1] if per_head else None, 0.5, self.dtype, 1, 1 if per_head else 0)

    def check_others(self, bad):
        for b in range(B):
            for g in range(H_KV):
                if (b, g) != bad:
                    self.check_kv_head(b, g)
            assert (self.mass[b, :, self.lens[b]:] == 0.25).all()


def _places(c):
    return [(b, t) for b in range(B) for t in (0, c.lens[b] - 1)]


@pytest.mark.parametrize("per_head", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_a_nan_key_makes_its_rows_nan(shape, per_head, cuda_device):
    for i, (b, t) in enumerate(_places(Case(shape, 80000))):
        c = Case(shape, 80000)
        slot, row = c.at(b, t)
        c.K[slot, 1, row, 3] = NAN
        c.run(cuda_device, per_head)
        n, h = c.lens[b], c.heads(1)
        assert torch.isnan(c.O[b, h]).all() and torch.isnan(c.lse[b, h]).all(), (b, t)
        assert torch.isnan(c.mass[b, 1 if per_head else 0, :n]).all(), (b, t)
        c.check_others((b, 1))


@pytest.mark.parametrize("per_head", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_a_nan_query_makes_its_row_nan(shape, per_head, cuda_device):
    c = Case(shape, 81000)
    b, head = 0, c.G  # the first head of KV head 1
    c.Q[b, head, 7] = NAN
    c.run(cuda_device, per_head)
    assert torch.isnan(c.O[b, head]).all() and torch.isnan(c.lse[b, head]).all()
    assert torch.isnan(c.mass[b, 1 if per_head else 0, :c.lens[b]]).all()
    for other in range(c.G, 2 * c.G):
        if other != head:
            assert torch.isfinite(c.O[b, other]).all() and torch.isfinite(c.lse[b, other])
    c.check_others((b, 1))


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_infinite_dot_products(shape, cuda_device):
    # -infinity at the first and last tokens: as if they were not cached
    c = Case(shape, 82000)
    c.Q[..., 5] = c.Q[..., 5].abs() + 0.5
    for b, t in _places(c):
        slot, row = c.at(b, t)
        c.K[slot, :, row, 5] = -INF
        c.K[slot, :, row, :5] = 1.0  # no tripled sink among them
    c.run(cuda_device, True)
    ref = Case(shape, 82000)
    ref.Q = c.Q
    for b in range(B):
        for g in range(H_KV):
            K, V = (torch.zeros_like(P[:, g:g + 1]) for P in (c.K, c.V))
            n = c.lens[b]
            src, to = np.arange(1, n - 1), np.arange(n - 2)
            t = c.table[b].long()
            for new, old in ((K, c.K), (V, c.V)):
                new[t[to // 64], 0, to % 64] = old[t[src // 64], g, src % 64]
            h = c.heads(g)
            m0, m1 = (m[b:b + 1, g:g + 1, 1:n - 1].contiguous() for m in (c.mass0, c.mass))
            _check_decode(c.Q[b:b + 1, h], K, V, c.table[b:b + 1], [n - 2], c.O[b:b + 1, h], c.lse[b:b + 1, h], m0, m1, 0.5,
                          c.dtype, 1, 1)
            assert (c.mass[b, g, [0, n - 1]] == 0.125).all()
    # every token: no weight is left
    for b in range(B):
        t = np.arange(c.lens[b])
        c.K[c.table[b].long()[t // 64], 1, t % 64, 5] = -INF
    c.run(cuda_device, True)
    for b in range(B):
        assert (c.O[b, c.heads(1)] == 0).all() and torch.isneginf(c.lse[b, c.heads(1)]).all()
        assert (c.mass[b, 1, :c.lens[b]] == 0.125).all()
    # +infinity
    for b, t in _places(c):
        slot, row = c.at(b, t)
        c.K[slot, 0, row, 5] = INF
    c.run(cuda_device, True)
    for b in range(B):
        assert torch.isnan(c.O[b, c.heads(0)]).all() and torch.isposinf(c.lse[b, c.heads(0)]).all()
        assert torch.isnan(c.mass[b, 0, :c.lens[b]]).all()


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_infinite_and_nan_values_reach_their_columns(shape, cuda_device):
    c = Case(shape, 83000)
    clean = c.V.clone()
    for b, t in _places(c):
        slot, row = c.at(b, t)
        c.V[slot, 1, row, 2], c.V[slot, 1, row, 9] = INF, -INF
        c.V[slot, 1, row, c.d - 1] = NAN
    for b in range(B):  # infinities of both signs in one column
        for t, v in ((0, INF), (c.lens[b] - 1, -INF)):
            slot, row = c.at(b, t)
            c.V[slot, 1, row, 17] = v
    c.run(cuda_device, True)
    h = c.heads(1)
    assert torch.isposinf(c.O[:, h, 2]).all() and torch.isneginf(c.O[:, h, 9]).all()
    assert torch.isnan(c.O[:, h, c.d - 1]).all() and torch.isnan(c.O[:, h, 17]).all()
    # the other columns, and everything else, as with the clean values
    c.V = clean
    keep = [i for i in range(c.d) if i not in (2, 9, 17, c.d - 1)]
    got = c.O.clone()
    c.run(cuda_device, True)
    assert torch.equal(c.O[:, :, keep], got[:, :, keep])
    for b in range(B):
        for g in range(H_KV):
            c.check_kv_head(b, g)
    assert np.isfinite(np_(got[:, c.heads(0)])).all()
