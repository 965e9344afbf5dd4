"""The long-prompt kernel of dl_qk_norm_rope: cache only (a prompt), K_out and
V_out only (a decode block of a long batch), and both, against the formula.

run_rope takes it for tokens of at least 1280 values of heads, rotations that are
multiples of 16, and 2 x 148 groups of eight tokens (fp32: 3 x 148).
Tolerances: those of test_gpu_token_step.py."""
import numpy as np
import pytest
import torch

import long_context_diffusion_b200 as dl
import synth
from tests.helpers import np_
from tests.test_gpu_token_step import DT, HALF, SEED, U, _desc, _near, _normal, _rope_ref, _table

pytestmark = pytest.mark.gpu

CASES = [
    # dtype, d, H, H_kv, n_tok, batch, rot, norm, inter
    ("bf16", 64, 16, 2, 1203, 2, 64, True, True),
    ("bf16", 64, 15, 3, 801, 3, 32, False, True),
    ("bf16", 64, 21, 1, 2401, 1, 64, True, False),
    ("bf16", 128, 8, 1, 1205, 2, 128, True, True),
    ("bf16", 128, 6, 2, 2402, 1, 64, True, True),
    ("bf16", 128, 9, 3, 803, 3, 16, True, False),
    ("bf16", 128, 4, 4, 1207, 2, 0, True, False),
    ("fp32", 64, 16, 2, 1203, 3, 64, True, True),
    ("fp32", 64, 18, 1, 1801, 2, 48, True, False),
    ("fp32", 128, 8, 1, 3601, 1, 128, False, True),
    ("fp32", 128, 8, 2, 1202, 3, 96, True, False),
]


@pytest.mark.parametrize("mode", ["cache", "out", "both"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_long_prompts_match_the_formula(case, mode, cuda_device):
    dtype, d, H, H_kv, n, B, rot, norm, inter = case
    dt, R, eps, dev = DT[dtype], H + 2 * H_kv, 1e-5, cuda_device
    tiles = B * -(-n // 8)
    assert R * d >= 1280 and rot % 16 == 0 and tiles >= (2 if dtype == "bf16" else 3) * 148  # the kernel meant
    sid = 97000 + 10 * CASES.index(case)
    qkv = _normal(sid, B, n, R * d, dtype=dt)
    pos = (synth.uniforms(SEED, sid + 1, 0, B * n) * (1 << 20)).to(torch.int32).reshape(B, n)
    f = None if rot == 0 else (10000.0 ** (-torch.arange(0, rot, 2).double() / rot)).float()
    qw, kw = ((1 + 0.2 * _normal(sid + 2 + j, d)).to(dt) if norm else None for j in range(2))
    L = n + 70
    desc = _desc(B, H, H_kv, d, L, dtype, n_slots=B * (-(-L // 64)) + 2)
    table = _table(sid + 4, B, desc.n_pages, desc.n_slots)
    start = torch.tensor([(37 * b) % 71 for b in range(B)], dtype=torch.int32)
    fits = np.ones(B, bool)
    if B > 1:  # the last sequence does not fit: nothing of it is appended
        start[B - 1], fits[B - 1] = 71, False
    put = lambda t: None if t is None else t.to(dev)  # noqa: E731
    Q = torch.full((B, H, n, d), 9.0, dtype=dt, device=dev)
    outs = [torch.full((B, H_kv, n, d), 9.0, dtype=dt, device=dev) for _ in range(2)] if mode != "cache" else [None] * 2
    cache = {}
    if mode != "out":
        pools = [torch.full((desc.n_slots, H_kv, 64, d), 7.0, dtype=dt, device=dev) for _ in range(2)]
        end = torch.full((B,), -9, dtype=torch.int32, device=dev)
        book = torch.full((B, H_kv, L), -5, dtype=torch.int32, device=dev), torch.full((B, H_kv, L), 3.0, device=dev)
        cache = dict(start=put(start), page_table=put(table), K_pool=pools[0], V_pool=pools[1], end=end, tok_pos=book[0],
                     tok_mass=book[1])
    dl.dl_qk_norm_rope(desc, put(qkv), put(pos), put(qw), put(kw), eps, put(f), Q, *outs, interleaved=inter, **cache)
    assert dl.dl_get_status() == (dl.DL_ERR_BAD_INDEX if cache and not fits.all() else dl.DL_OK)
    x, p, fn = np_(qkv).reshape(B, n, R, d), np_(pos), None if f is None else np_(f)
    ref, tol = x.astype(np.float64), np.zeros(x.shape)
    for lo, hi, w in ((0, H, qw), (H, H + H_kv, kw)):
        y, mag = _rope_ref(x[:, :, lo:hi], p[:, :, None].repeat(hi - lo, 2), None if w is None else np_(w), eps, fn, inter)
        ref[:, :, lo:hi], tol[:, :, lo:hi] = y, 16 * U * mag + HALF[dtype] * (np.abs(y) + 16 * U * mag)
    heads = (slice(0, H), slice(H, H + H_kv), slice(H + H_kv, R))
    _near(np_(Q).transpose(0, 2, 1, 3), ref[:, :, heads[0]], tol[:, :, heads[0]], "Q")
    for o, h, name in zip(outs, heads[1:], "KV"):
        if o is not None:
            _near(np_(o).transpose(0, 2, 1, 3), ref[:, :, h], tol[:, :, h], name)  # values: a bound of zero
    if not cache:
        return
    seen = np.zeros((desc.n_slots, 64), bool)
    tp, ms = np_(book[0]), np_(book[1])
    for b in range(B):
        rest = np.ones(L, bool)
        if fits[b]:
            t = int(start[b]) + np.arange(n)
            slot = np_(table)[b, t // 64]
            for pool, h, name in zip(pools, heads[1:], "KV"):
                _near(np_(pool)[slot, :, t % 64], ref[b][:, h], tol[b][:, h], name + " pool")
            seen[slot, t % 64] = True
            assert (tp[b][:, t] == p[b]).all() and (ms[b][:, t] == 0).all()
            rest[t] = False
        assert (tp[b][:, rest] == -5).all() and (ms[b][:, rest] == 3).all()
    for pool in pools:
        assert (np_(pool).transpose(0, 2, 1, 3)[~seen] == 7).all()
    assert np_(end).tolist() == [int(start[b]) + (n if fits[b] else 0) for b in range(B)]


@pytest.mark.parametrize("extra", [4, 1, 200])
def test_a_single_token_may_have_anything_behind_its_heads(extra, cuda_device):
    """One token has no neighbour, so the width of its tensor is no step."""
    H, H_kv, d = 4, 2, 64
    desc = _desc(1, H, H_kv, d, 10, "bf16")
    x = _normal(98000, 1, 1, (H + 2 * H_kv) * d + extra, dtype=torch.bfloat16)
    pos = torch.full((1, 1), 77, dtype=torch.int32, device=cuda_device)
    f = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float().to(cuda_device)
    got = []
    for t in (x, x[..., :(H + 2 * H_kv) * d].contiguous()):
        o = [torch.full((1, h, 1, d), 9.0, dtype=torch.bfloat16, device=cuda_device) for h in (H, H_kv, H_kv)]
        dl.dl_qk_norm_rope(desc, t.to(cuda_device), pos, None, None, 0.0, f, *o)
        got.append(o)
    assert dl.dl_get_status() == dl.DL_OK
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_a_denoising_block_is_committed_with_its_pooled_keys(cuda_device):
    """K_out and V_out as a decode block, then dl_cache_write: the rows that an
    append of the same block writes, with the pooled keys kept."""
    dev, B, H, H_kv, d, n, L = cuda_device, 2, 8, 4, 128, 32, 192
    desc = _desc(B, H, H_kv, d, L, "bf16")
    table = _table(98500, B, desc.n_pages, desc.n_slots).to(dev)
    x = _normal(98501, B, n, (H + 2 * H_kv) * d, dtype=torch.bfloat16).to(dev)
    pos = (torch.arange(n, dtype=torch.int32, device=dev) + 100).expand(B, n).contiguous()
    f = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float().to(dev)
    w = torch.ones(d, dtype=torch.bfloat16, device=dev)
    start = torch.tensor([100, 7], dtype=torch.int32, device=dev)
    pools = [[_normal(98502 + j, desc.n_slots, H_kv, 64, d, dtype=torch.bfloat16).to(dev) for j in range(2)] for _ in range(2)]
    Q = torch.empty(B, H, n, d, dtype=torch.bfloat16, device=dev)
    dl.dl_qk_norm_rope(desc, x, pos, w, w, 1e-6, f, Q, start=start, page_table=table, K_pool=pools[0][0], V_pool=pools[0][1])
    K, V = (torch.empty(B, H_kv, n, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    kbar, want = (torch.empty(B, H_kv, desc.n_pages, d, device=dev) for _ in range(2))
    dl.dl_pool_keys(desc, pools[1][0], table, desc.n_pages, 64, 0, 64, kbar)
    dl.dl_qk_norm_rope(desc, x, pos, w, w, 1e-6, f, Q, K, V)
    dl.dl_cache_write(desc, K, V, start, table, *pools[1], kbar)
    dl.dl_pool_keys(desc, pools[0][0], table, desc.n_pages, 64, 0, 64, want)
    assert dl.dl_get_status() == dl.DL_OK
    for a, b in zip(pools[0], pools[1]):
        assert torch.equal(a, b)
    assert torch.equal(kbar, want)
