"""GPU parity of the token-by-token operators (dl_qk_norm_rope,
dl_decode_attn, dl_evict_select, dl_cache_compact) against the fp64 oracle.

Tolerances, derived from the arithmetic (u = 2^-24, half an fp32 step; r =
half a step of the output dtype: 2^-8 for bf16, u for fp32):
 - rotated row: a pair (x, y) of normed values has at most 7 u (mean square,
   halved by the square root) + 3 u (inverse root and two products) relative
   error; cosine and sine carry 2 u (sincospi) + 1.6 u (the angle in turns
   rounded to fp32, times 2 pi); product and sum 2 u: together 16 u (|x| + |y|),
   then the rounding to the dtype.
 - logits: a dot product of d terms, each product and each of at most d + 3
   sums rounded: delta = (2 d + 8) u scale |q| |k|, largest over the keys (the
   tensor cores' sums are allowed a whole step a term).
 - weights: relative 2 delta + 8 u (exponential and its argument, |a| < 30:
   30 u more); sums over n tokens: n u more; bf16 weights of the P V product
   are held to 16 bits (2^-16): eps_w = 2 delta + (n + 64) u + [bf16] 2^-16.
   O is off by at most eps_w sum_t w_t |v_t| twice (numerator and
   normaliser), then the rounding; lse by delta + (n + 64) u + 2 u |lse|; a mass
   by 2 eps_w of the weights added and 4 u of the result.
Moves, positions, lists and lengths are exact."""
import numpy as np
import pytest
import torch

import long_context_diffusion_b200 as dl
import oracle
import synth
from long_context_diffusion_b200 import pipeline
from tests.helpers import np_

pytestmark = pytest.mark.gpu

SEED = 20261208
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": U}


def _normal(sid, *shape, dtype=torch.float32):
    return synth.normals(SEED, sid, 0, int(np.prod(shape))).reshape(shape).to(dtype)


def _table(sid, batch, n_pages, n_slots):
    perm = torch.argsort(synth.uniforms(SEED, sid, 0, n_slots))[:batch * n_pages]
    return perm.to(torch.int32).reshape(batch, n_pages)


def _desc(batch, H, H_kv, d, L_ctx, dtype, n_slots=None, L_q=1):
    n_pages = -(-L_ctx // 64)
    return dl.make_desc(batch, H, H_kv, d, L_ctx, L_q, 64, n_pages,
                        n_slots or max(1, batch * n_pages), DT[dtype])


def _near(got, ref, tol, what):
    got, ref, tol = np.asarray(got), np.asarray(ref), np.broadcast_to(tol, np.shape(ref))
    same = got == ref                                   # infinities
    bad = ~same & ~(np.abs(np.where(same, 0, got) - np.where(same, 0, ref)) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - ref) / tol):.3g} of the bound"


# --------------------------------------------------------------- c1
def _rope_ref(x, pos, w, eps, f, inter):
    """Rows x [..., d] at pos [...]: value and the pair's magnitude |x| + |y|."""
    x = x.astype(np.float64)
    d, n = x.shape[-1], 0 if f is None else len(f)
    if w is not None:
        x = x * w / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y, mag = x.copy(), np.abs(x)
    if n:
        i = np.arange(n)
        u, v = (2 * i, 2 * i + 1) if inter else (i, i + n)
        a = pos[..., None].astype(np.float64) * f
        y[..., u] = x[..., u] * np.cos(a) - x[..., v] * np.sin(a)
        y[..., v] = x[..., v] * np.cos(a) + x[..., u] * np.sin(a)
        mag[..., u] = mag[..., v] = np.abs(x[..., u]) + np.abs(x[..., v])
    return y, mag


ROPE_CASES = [
    # dtype, d, H, H_kv, n_tok, batch, rot, norm, inter, extra columns
    ("bf16", 128, 28, 4, 1, 3, 128, True, False, 0),
    ("bf16", 128, 32, 32, 5, 1, 128, True, True, 0),
    ("bf16", 64, 4, 4, 33, 2, 64, False, False, 0),
    ("fp32", 64, 4, 1, 7, 2, 64, True, False, 24),
    ("fp32", 128, 7, 1, 70, 1, 32, True, False, 0),
    ("fp32", 128, 2, 2, 9, 3, 24, True, True, 8),
    ("bf16", 64, 1, 1, 2, 1, 24, False, False, 40),
    ("bf16", 128, 3, 1, 4, 2, 0, True, False, 0),
    ("fp32", 64, 5, 5, 130, 2, 48, True, False, 0),
    ("bf16", 128, 16, 8, 300, 4, 128, True, False, 128),
    # enough tokens for the long-prompt kernel (at least 2 x 148 groups of eight)
    # -- but of fewer than 1280 values each, which go row by row; with rows enough
    # for that kernel: the last cases here, and test_gpu_token_prompt.py
    ("bf16", 128, 5, 1, 2373, 1, 128, True, False, 0),
    ("bf16", 64, 4, 2, 1203, 2, 32, True, False, 8),
    ("bf16", 128, 2, 2, 803, 3, 96, False, True, 0),
    ("bf16", 64, 1, 1, 2401, 1, 0, True, False, 0),
    ("bf16", 128, 2, 1, 2404, 1, 40, True, False, 0),    # 40: by fours
    ("fp32", 128, 3, 1, 1201, 2, 128, True, True, 4),
    ("fp32", 64, 4, 2, 2369, 1, 64, False, False, 0),
    # many tokens of few rows
    ("bf16", 64, 1, 1, 6400, 3, 64, True, False, 0),
    ("bf16", 128, 4, 2, 9500, 2, 24, False, True, 0),
    ("bf16", 128, 20, 2, 1200, 2, 128, True, False, 0),
    # enough tokens and rows for the long-prompt kernel; rows that its groups of
    # two (128 columns) or four (64) do not divide, kinds shorter than a group
    ("bf16", 128, 10, 1, 1203, 2, 128, True, False, 0),
    ("bf16", 64, 20, 1, 803, 3, 32, True, False, 8),
    ("bf16", 128, 9, 3, 2373, 1, 96, False, True, 0),
    ("bf16", 64, 22, 1, 2401, 1, 0, True, False, 0),
    ("bf16", 128, 11, 1, 2404, 1, 40, True, False, 0),   # 40: by fours
    ("fp32", 128, 9, 3, 1803, 2, 128, True, True, 4),
    ("fp32", 64, 18, 2, 1203, 3, 64, False, False, 0),
]


@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "-".join(map(str, c)))
def test_qk_norm_rope_matches_the_formula(case, cuda_device):
    dtype, d, H, H_kv, n, B, rot, norm, inter, extra = case
    dt, R, eps = DT[dtype], H + 2 * H_kv, 1e-5
    sid = 21000 + 10 * ROPE_CASES.index(case)
    wide = _normal(sid, B, n, R * d + extra, dtype=dt)
    qkv = wide.to(cuda_device)[..., :R * d]           # a view when extra > 0
    pos = (synth.uniforms(SEED, sid + 1, 0, B * n) * (1 << 20)).to(torch.int32).reshape(B, n)
    pos[0, 0] = 0
    f = None if rot == 0 else (10000.0 ** (-torch.arange(0, rot, 2).double() / rot)).float()
    qw, kw = ((1 + 0.2 * _normal(sid + 2 + j, d)).to(dt) if norm else None for j in range(2))
    L = n + 70
    desc = _desc(B, H, H_kv, d, L, dtype, n_slots=B * (-(-L // 64)) + 2)
    table = _table(sid + 4, B, desc.n_pages, desc.n_slots)
    start = torch.tensor([(37 * b) % 71 for b in range(B)], dtype=torch.int32)
    dev = lambda t: None if t is None else t.to(cuda_device)  # noqa: E731
    outs = [torch.full((B, h, n, d), 9.0, dtype=dt, device=cuda_device) for h in (H, H_kv, H_kv)]
    pools = [torch.full((desc.n_slots, H_kv, 64, d), 7.0, dtype=dt, device=cuda_device) for _ in range(2)]
    end = torch.full((B,), -9, dtype=torch.int32, device=cuda_device)
    tok_pos = torch.full((B, H_kv, L), -5, dtype=torch.int32, device=cuda_device)
    mass = torch.full((B, H_kv, L), 3.0, device=cuda_device)
    dl.dl_qk_norm_rope(desc, qkv, dev(pos), dev(qw), dev(kw), eps, dev(f), *outs, dev(start), dev(table),
                       *pools, end, tok_pos, mass, interleaved=inter)
    assert dl.dl_get_status() == dl.DL_OK
    x = np_(wide[..., :R * d]).reshape(B, n, R, d)
    p, fn = np_(pos), None if f is None else np_(f)
    ref, tol = np.empty_like(x), np.empty_like(x)
    for lo, hi, w in ((0, H, qw), (H, H + H_kv, kw)):
        y, mag = _rope_ref(x[:, :, lo:hi], p[:, :, None].repeat(hi - lo, 2), None if w is None else np_(w), eps,
                           fn, inter)
        ref[:, :, lo:hi], tol[:, :, lo:hi] = y, 16 * U * mag + HALF[dtype] * (np.abs(y) + 16 * U * mag)
    # one row against the oracle's own, slow form
    one = oracle.norm_rotate(x[B - 1, n - 1, 0], int(p[B - 1, n - 1]), None if qw is None else np_(qw), eps, fn, inter)
    np.testing.assert_allclose(ref[B - 1, n - 1, 0], one, rtol=1e-12, atol=1e-14)
    got = [np_(o).transpose(0, 2, 1, 3) for o in outs]
    _near(got[0], ref[:, :, :H], tol[:, :, :H], "Q")
    _near(got[1], ref[:, :, H:H + H_kv], tol[:, :, H:H + H_kv], "K")
    assert np.array_equal(got[2], x[:, :, H + H_kv:])
    # the cache: the same rows at start.. through the page table, nothing else written
    kp, vp = np_(pools[0]), np_(pools[1])
    seen = np.zeros(kp.shape[:1] + kp.shape[2:3], bool)
    tp, ms = np_(tok_pos), np_(mass)
    for b in range(B):
        t = int(start[b]) + np.arange(n)
        slot = np_(table)[b, t // 64]
        assert np.array_equal(kp[slot, :, t % 64], got[1][b]) and np.array_equal(vp[slot, :, t % 64], got[2][b])
        seen[slot, t % 64] = True
        assert (tp[b][:, t] == p[b]).all() and (ms[b][:, t] == 0).all()
        rest = np.ones(L, bool)
        rest[t] = False
        assert (tp[b][:, rest] == -5).all() and (ms[b][:, rest] == 3).all()
    assert (kp.transpose(0, 2, 1, 3)[~seen] == 7).all() and (vp.transpose(0, 2, 1, 3)[~seen] == 7).all()
    assert np.array_equal(np_(end), np_(start) + n)


def test_qk_norm_rope_far_positions_keep_their_phase(cuda_device):
    d, n = 64, 6
    x = _normal(21900, 1, n, 3 * d)
    pos = torch.tensor([[2**24 + 1, 2**31 - 1, -1, -2**31, 10**8 + 7, 0]], dtype=torch.int32)
    f = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float()
    desc = _desc(1, 1, 1, d, n, "fp32")
    out = [torch.empty(1, 1, n, d, device=cuda_device) for _ in range(3)]
    dl.dl_qk_norm_rope(desc, x.to(cuda_device), pos.to(cuda_device), None, None, 0.0, f.to(cuda_device), *out)
    y, mag = _rope_ref(np_(x)[0][:, :d], np_(pos)[0], None, 0.0, np_(f), False)
    # angle: pos f / 2pi held in fp64, below 2^29 turns: 2^-24 turns twice, 6.3 rad a turn
    far = np.abs(np_(pos)[0])[:, None] * 2.0 ** -53 * 2 * 3
    _near(np_(out[0])[0, 0], y, (16 * U + far) * mag, "far")


@pytest.mark.parametrize("n_mass", [1, 2])
def test_qk_norm_rope_reports_and_skips_what_does_not_fit(n_mass, cuda_device):
    B, H, H_kv, d, n, L = 4, 2, 2, 64, 3, 130
    desc = _desc(B, H, H_kv, d, L, "bf16")
    x = _normal(21950, B, n, (H + 2 * H_kv) * d, dtype=torch.bfloat16).to(cuda_device)
    pos = torch.arange(B * n, dtype=torch.int32, device=cuda_device).reshape(B, n)
    table = torch.arange(B * 3, dtype=torch.int32).reshape(B, 3)
    table[3, 0] = desc.n_slots                         # sequence 3: bad first page
    start = torch.tensor([128, -1, 2**31 - 2, 62], dtype=torch.int32, device=cuda_device)
    pools = [torch.zeros(desc.n_slots, H_kv, 64, d, dtype=torch.bfloat16, device=cuda_device) for _ in range(2)]
    end = torch.zeros(B, dtype=torch.int32, device=cuda_device)
    tp = torch.full((B, n_mass, L), -7, dtype=torch.int32, device=cuda_device)
    Q = torch.full((B, H, n, d), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    dl.dl_qk_norm_rope(desc, x, pos, None, None, 1e-6, None, Q, start=start, page_table=table.to(cuda_device),
                       K_pool=pools[0], V_pool=pools[1], end=end, tok_pos=tp)
    assert dl.dl_get_status() == dl.DL_ERR_BAD_INDEX
    assert torch.isfinite(Q).all()                     # the queries are all there
    assert end.tolist() == [128, -1, 2**31 - 2, 65]
    k = np_(pools[0])
    assert (k[:9] == 0).all() and (k[9] == 0).all()    # 0: 128 + 3 > 130; 3: page 0 skipped
    assert np.array_equal(k[10][:, 0], np_(x)[3, 2].reshape(-1, d)[H:H + H_kv])
    assert (k[10][:, 1:] == 0).all() and (k[11:] == 0).all()
    assert (np_(tp)[:3] == -7).all() and (np_(tp)[3][:, 64] == 11).all() and (np_(tp)[3][:, :64] == -7).all()


# --------------------------------------------------------------- c2
def _cache(sid, B, H_kv, d, lens, L, dt, spare=2):
    """Pools whose rows behind every sequence's length, and spare slots, are NaN."""
    n_pages = -(-L // 64)
    n_slots = max(1, B * n_pages) + spare
    table = _table(sid, B, n_pages, n_slots)
    K = torch.full((n_slots, H_kv, 64, d), float("nan"), dtype=dt)
    V = K.clone()
    for b, n in enumerate(lens):
        t = torch.arange(n)
        slot = table[b].long()[t // 64]
        K[slot, :, t % 64] = _normal(sid + 1 + b, n, H_kv, d, dtype=dt)
        V[slot, :, t % 64] = _normal(sid + 500 + b, n, H_kv, d, dtype=dt)
        if n:
            K[slot[0], :, 0] *= 3
    return K, V, table


def _check_decode(Q, K, V, table, lens, O, lse, mass0, mass, decay, dtype, H_kv, n_mass, what=""):
    """Against the oracle, sequence by sequence and KV head by KV head."""
    B, H, d = Q.shape
    G = H // H_kv
    On, ln = np_(O), None if lse is None else np_(lse)
    scale = d ** -0.5
    for b, n in enumerate(lens):
        add = np.zeros((n_mass, n))
        err = np.zeros((n_mass, n))
        for g in range(H_kv):
            Kb, Vb = (oracle.cached_rows(P, np_(table)[b], g, n, 64) for P in (K, V))
            q = np_(Q[b, g * G:(g + 1) * G])
            o, s, w = oracle.decode_attention(q, Kb, Vb)
            delta = 0.0 if n == 0 else (2 * d + 8) * U * scale * np.linalg.norm(q, axis=1).max() * \
                np.linalg.norm(Kb, axis=1).max()
            eps_w = 2 * delta + (n + 64) * U + (2.0 ** -16 if dtype == "bf16" else 0.0)
            ab = w @ np.abs(Vb) if n else np.zeros_like(o)
            tol = 2 * eps_w * ab
            _near(On[b, g * G:(g + 1) * G], o, tol + HALF[dtype] * (np.abs(o) + tol), f"{what} O {b},{g}")
            if ln is not None:
                _near(ln[b, g * G:(g + 1) * G], s, delta + (n + 64) * U + 2 * U * np.abs(s), f"{what} lse {b},{g}")
            m = g if n_mass > 1 or H_kv == 1 else 0
            if n_mass:
                add[m] += w.sum(0)
                err[m] += 2 * eps_w * w.sum(0)
        if mass is not None:
            m0, m1 = np_(mass0)[b], np_(mass)[b]
            old = 0.0 if decay == 0 else np.float64(np.float32(decay)) * m0[:, :n]
            ref = old + add
            _near(m1[:, :n], ref, err + 4 * U * np.abs(ref) + 1e-38, f"{what} mass {b}")
            assert np.array_equal(m1[:, n:], m0[:, n:], equal_nan=True)   # rows behind the length


DECODE_CASES = [
    # dtype, d, G, H_kv, L_ctx, lens, n_mass (0: no masses), decay
    ("bf16", 128, 1, 4, 1000, [1000, 1, 0, 64], 4, 1.0),
    ("bf16", 128, 7, 4, 700, [65, 700], 1, 0.5),
    ("bf16", 128, 4, 2, 333, [333, 63, 129], 2, 0.0),
    ("bf16", 64, 8, 1, 500, [499, 500, 2], 1, 0.9),
    ("bf16", 64, 3, 3, 130, [130, 17], 0, 1.0),
    ("bf16", 128, 16, 2, 257, [257, 0, 200], 2, 1.0),
    ("bf16", 128, 40, 1, 190, [190, 100], 1, 1.0),       # more query heads than one row block
    ("bf16", 64, 17, 2, 90, [64, 90], 1, 1.0),
    ("fp32", 128, 1, 3, 600, [600, 5, 0], 3, 1.0),
    ("fp32", 64, 4, 4, 1024, [1023, 1, 640], 1, 0.25),
    ("fp32", 128, 7, 2, 200, [128, 200], 2, 0.0),
    ("fp32", 64, 20, 1, 129, [129, 127], 1, 1.0),
    ("bf16", 128, 2, 8, 64, [64] * 5 + [0] * 3 + [1] * 4, 8, 1.0),
    ("bf16", 128, 1, 1, 4000, [4000], 1, 1.0),           # one long row over the whole grid
    ("fp32", 64, 1, 1, 3001, [3001], 1, 1.0),
    ("bf16", 64, 2, 2, 1, [1, 0], 2, 1.0),               # capacity of one token
    ("bf16", 128, 2, 2, 9000, [9000, 0, 70], 2, 0.5),    # too long for clusters
    ("bf16", 64, 3, 4, 8100, [5000, 8100], 1, 1.0),
    ("bf16", 128, 12, 1, 6000, [6000, 5999], 1, 0.3),
    ("fp32", 128, 2, 2, 5000, [4990, 33], 2, 0.0),
    ("fp32", 64, 9, 1, 2100, [2100, 64], 1, 1.0),
    ("fp32", 128, 2, 3, 3000, [2999], 3, 1.0),
    ("bf16", 64, 1, 5, 150, [150, 20, 0] * 12, 5, 1.0),  # clusters of one CTA
    ("bf16", 64, 16, 8, 130, [130, 1, 0, 64] * 10, 8, 1.0),  # more query rows than the join takes at once
    ("fp32", 64, 4, 16, 3, [3, 0, 1] * 9, 1, 0.5),
    # fp32 blocks of two, four and eight rows: lengths that end in each warp's keys
    ("fp32", 64, 3, 2, 70, [15, 16, 17, 48, 49, 63, 64, 65, 70, 1], 2, 1.0),
    ("fp32", 128, 3, 1, 100, [7, 8, 9, 24, 25, 32, 33, 96, 97], 1, 1.0),
    ("fp32", 128, 8, 1, 300, [300, 8, 9], 1, 1.0),
    ("fp32", 64, 4, 3, 7000, [7000, 4097], 1, 0.7),
    ("fp32", 128, 4, 2, 5100, [5100, 31, 33], 2, 1.0),
    ("fp32", 64, 2, 2, 6000, [6000, 17], 2, 1.0),
    # more items than clusters of eight (of four) that are resident at once
    ("bf16", 128, 8, 4, 520, [520, 100, 0] * 3, 4, 1.0),
    ("bf16", 64, 5, 4, 900, [900, 450] * 9, 1, 1.0),
]


@pytest.mark.parametrize("case", DECODE_CASES, ids=lambda c: "-".join(str(x) for x in c[:5]) + f"-b{len(c[5])}-m{c[6]}")
def test_decode_attn_matches_oracle(case, cuda_device):
    dtype, d, G, H_kv, L, lens, n_mass, decay = case
    dt, B = DT[dtype], len(lens)
    sid = 22000 + 1000 * DECODE_CASES.index(case)
    K, V, table = _cache(sid, B, H_kv, d, lens, L, dt)
    desc = _desc(B, G * H_kv, H_kv, d, L, dtype, n_slots=K.shape[0])
    Q = _normal(sid + 990, B, G * H_kv, d, dtype=dt)
    dev = lambda t: t.to(cuda_device)  # noqa: E731
    O = torch.full((B, G * H_kv, d), float("nan"), dtype=dt, device=cuda_device)
    lse = torch.full((B, G * H_kv), float("nan"), device=cuda_device)
    mass0 = mass = None
    if n_mass:
        mass0 = synth.uniforms(SEED, sid + 991, 0, B * n_mass * L).reshape(B, n_mass, L).float()
        if decay == 0:
            mass0[:] = float("nan")                     # not read
        for b, n in enumerate(lens):
            mass0[b, :, n:] = -4.0
        mass = dev(mass0)
    ws = torch.full((max(dl.dl_workspace_size(desc), 256),), 255, dtype=torch.uint8, device=cuda_device)
    ctx_len = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    dl.dl_decode_attn(desc, dev(Q), dev(K), dev(V), dev(table), ctx_len, O, lse, ws, tok_mass=mass, decay=decay)
    assert dl.dl_get_status() == dl.DL_OK
    _check_decode(Q, K, V, table, lens, O, lse, mass0, mass, decay, dtype, H_kv, n_mass)
    # without lse and masses: the same output, bit for bit, from a used workspace
    O2 = torch.empty_like(O)
    dl.dl_decode_attn(desc, dev(Q), dev(K), dev(V), dev(table), ctx_len, O2, None, ws)
    assert dl.dl_get_status() == dl.DL_OK and torch.equal(O, O2)


def test_decode_attn_equals_dense_attention_of_the_framework(cuda_device):
    """All lengths full: the framework's own attention with the last token as
    its decode block gives the same row (dl_sparse_attn, L_q 1)."""
    B, H, H_kv, d, L = 2, 8, 2, 128, 330
    K, V, table = _cache(40000, B, H_kv, d, [L, L], L, torch.bfloat16)
    Q = _normal(40990, B, H, d, dtype=torch.bfloat16).to(cuda_device)
    last = [torch.stack([P[table[b].long()[(L - 1) // 64], :, (L - 1) % 64] for b in range(B)])[:, :, None] for P in (K, V)]
    K, V, table = K.to(cuda_device), V.to(cuda_device), table.to(cuda_device)
    full, cut = (_desc(B, H, H_kv, d, n, "bf16", n_slots=K.shape[0]) for n in (L, L - 1))
    assert full.n_pages == cut.n_pages
    O1, O2 = (torch.empty(B, 1, H, d, dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    l1, l2 = (torch.empty(B, H, 1, device=cuda_device) for _ in range(2))
    ws = pipeline.workspace(full, cuda_device)
    dl.dl_sparse_attn(cut, Q.view(B, H, 1, d), K, V, table, None, None, last[0].contiguous().to(cuda_device),
                      last[1].contiguous().to(cuda_device), O1, l1, ws)
    lens = torch.full((B,), L, dtype=torch.int32, device=cuda_device)
    dl.dl_decode_attn(full, Q, K, V, table, lens, O2, l2, ws)
    assert dl.dl_get_status() == dl.DL_OK
    # both within one bf16 step of the exact row (P in bf16 in the one: 2^-8 of weights |v| < 5)
    assert (O1.float() - O2.float()).abs().max() <= 2.0 ** -8 * (O1.float().abs().max() + 5)
    assert (l1 - l2).abs().max() <= 1e-3


def test_decode_attn_bad_lengths_and_pages_are_reported(cuda_device):
    B, H, H_kv, d, L = 5, 4, 2, 128, 200
    lens = [200, 100, 200, 64, 10]
    K, V, table = _cache(41000, B, H_kv, d, lens, L, torch.bfloat16)
    desc = _desc(B, H, H_kv, d, L, "bf16", n_slots=K.shape[0])
    Q = _normal(41990, B, H, d, dtype=torch.bfloat16)
    bad = torch.tensor([201, 100, -1, 64, 2**31 - 1], dtype=torch.int32)
    t2 = table.clone()
    t2[3, 0] = -1
    t2[1, 2:] = desc.n_slots + 5                        # behind the length: never read
    O = torch.full((B, H, d), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    lse = torch.empty(B, H, device=cuda_device)
    mass = torch.full((B, 2, L), 0.5, device=cuda_device)
    ws = pipeline.workspace(desc, cuda_device)
    dev = lambda t: t.to(cuda_device)  # noqa: E731
    dl.dl_decode_attn(desc, dev(Q), dev(K), dev(V), dev(t2), dev(bad), O, lse, ws, tok_mass=mass)
    assert dl.dl_get_status() == dl.DL_ERR_BAD_INDEX
    for b in (0, 2, 4):                                 # count as empty
        assert (O[b] == 0).all() and torch.isneginf(lse[b]).all() and (mass[b] == 0.5).all()
    keep = [1]
    _check_decode(Q[keep], K, V, table[keep], [100], O[keep], lse[keep], torch.full((1, 2, L), 0.5), mass[keep], 1.0,
                  "bf16", H_kv, 2)
    dl.dl_decode_attn(desc, dev(Q), dev(K), dev(V), dev(table), dev(torch.tensor(lens, dtype=torch.int32)), O, lse, ws)
    assert dl.dl_get_status() == dl.DL_OK


def test_decode_attn_of_an_empty_cache(cuda_device):
    desc = _desc(2, 4, 2, 64, 0, "fp32")
    O = torch.full((2, 4, 64), 5.0, device=cuda_device)
    lse = torch.zeros(2, 4, device=cuda_device)
    pool = torch.zeros(desc.n_slots, 2, 64, 64, device=cuda_device)
    z = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    dl.dl_decode_attn(desc, torch.ones(2, 4, 64, device=cuda_device), pool, pool,
                      torch.zeros(2, 0, dtype=torch.int32, device=cuda_device), z, O, lse,
                      pipeline.workspace(desc, cuda_device),
                      tok_mass=torch.zeros(2, 1, 0, device=cuda_device))
    assert dl.dl_get_status() == dl.DL_OK and (O == 0).all() and torch.isneginf(lse).all()


# --------------------------------------------------------------- c3
def _plan(desc, mass, pos, lens, budget, n_first, n_recent, dev, extra=0):
    n_mass = mass.shape[1]
    hole, fill, cnt = pipeline.eviction_buffers(desc, n_mass, budget, dev)
    if extra:
        hole, fill = (torch.empty(*t.shape[:2], t.shape[2] + extra, dtype=torch.int32, device=dev) for t in (hole, fill))
    hole.fill_(-77), fill.fill_(-77), cnt.fill_(-77)
    new = torch.full((desc.batch,), -77, dtype=torch.int32, device=dev)
    dl.dl_evict_select(desc, mass.to(dev), None if pos is None else pos.to(dev),
                       torch.tensor(lens, dtype=torch.int32, device=dev), budget, n_first, n_recent, hole, fill, cnt, new)
    return hole, fill, cnt, new


def _check_plan(mass, pos, lens, budget, n_first, n_recent, L, plan):
    hole, fill, cnt, new = (np_(t) for t in plan)
    for b, n in enumerate(lens):
        for m in range(mass.shape[1]):
            p = None if pos is None else np_(pos)[b, m, :n]
            h, f = oracle.evict_plan(np_(mass)[b, m, :n], p, budget, n_first, n_recent)
            assert cnt[b, m] == len(h), (b, m)
            assert hole[b, m, :len(h)].tolist() == h and fill[b, m, :len(f)].tolist() == f, (b, m)
            assert (hole[b, m, len(h):] == -1).all() and (fill[b, m, len(f):] == -1).all()
        assert new[b] == min(n, budget)


EVICT_CASES = [
    # L, lens, n_mass, budget, n_first, n_recent, positions, masses
    (1000, [1000, 300, 301, 0], 2, 300, 4, 64, True, "random"),
    (1000, [999], 1, 998, 0, 0, False, "random"),
    (65, [65, 64, 1], 3, 64, 0, 1, False, "random"),
    (2112, [2112, 2100], 4, 2048, 4, 128, True, "random"),
    (5000, [5000, 4097, 4096], 1, 1, 0, 0, False, "ties"),
    (5000, [5000, 2048], 2, 1700, 1, 1, True, "ties"),
    (700, [700], 2, 100, 60, 40, True, "zero"),          # nothing but the held and ties of zero
    (3000, [3000, 2999], 1, 1500, 0, 500, False, "odd"),  # infinities, NaN, -0, negative masses
    (2, [2], 1, 1, 1, 0, False, "random"),
    (100, [100, 50], 2, 100, 10, 10, False, "random"),   # budget = capacity: no moves at all
    (40000, [40000, 12345], 1, 5000, 4, 300, True, "random"),
    (130001, [130001], 1, 65000, 0, 0, False, "ties"),
    (420001, [420001, 400000], 1, 100000, 4, 1000, True, "random"),   # keys not kept on chip
    (400000, [400000], 1, 90000, 0, 0, False, "ties"),
    (300001, [300001], 1, 150000, 0, 9, True, "ties"),                  # 37 iterations a warp
    (1500, [1500] * 90 + [900, 1200], 2, 800, 2, 16, False, "random"),  # more rows than SMs
    (9001, [9001, 8999] * 40, 2, 3000, 1, 8, False, "ties"),
    (17000, [17000, 16000] * 40, 2, 1000, 0, 50, True, "random"),
    # more rows than clusters of eight (of four) that are resident at once
    (17001, [17001, 17000], 8, 900, 4, 100, True, "random"),
    (18000, [18000, 17000], 17, 9000, 0, 0, False, "ties"),
]


@pytest.mark.parametrize("case", EVICT_CASES, ids=lambda c: f"{c[0]}-b{len(c[1])}-{'-'.join(map(str, c[2:]))}")
def test_evict_select_is_the_oracles_plan(case, cuda_device):
    L, lens, n_mass, budget, n_first, n_recent, moved, kind = case
    B, sid = len(lens), 50000 + 10 * EVICT_CASES.index(case)
    u = synth.uniforms(SEED, sid, 0, B * n_mass * L).reshape(B, n_mass, L)
    mass = u.float() ** 3
    if kind == "ties":
        mass = torch.floor(u * 5).float()
    elif kind == "zero":
        mass = torch.zeros_like(mass)
    elif kind == "odd":
        mass = torch.floor(u * 7).float() - 3
        mass[mass == 3], mass[mass == -3], mass[mass == 2] = float("inf"), float("-inf"), float("nan")
        mass[mass == 0] *= torch.where(u[mass == 0] * 7 % 1 < 0.5, -1.0, 1.0).float()
    pos = None
    if moved:
        pos = torch.argsort(u, dim=-1, stable=True).to(torch.int32) * 3 - 5
    desc = _desc(B, n_mass, n_mass, 64, L, "bf16")
    plan = _plan(desc, mass, pos, lens, budget, n_first, n_recent, cuda_device, extra=case[2] % 2)
    assert dl.dl_get_status() == dl.DL_OK
    _check_plan(mass, pos, lens, budget, n_first, n_recent, L, plan)


def test_evict_select_bad_length_is_reported(cuda_device):
    L, budget = 500, 100
    mass = synth.uniforms(SEED, 51000, 0, 3 * 2 * L).reshape(3, 2, L).float()
    desc = _desc(3, 4, 2, 64, L, "bf16")
    plan = _plan(desc, mass, None, [501, 500, -3], budget, 0, 0, cuda_device)
    assert dl.dl_get_status() == dl.DL_ERR_BAD_INDEX
    assert plan[3].tolist() == [501, 100, -3]
    assert (plan[2][[0, 2]] == 0).all() and (plan[0][[0, 2]] == -1).all()
    _check_plan(mass[1:2], None, [500], budget, 0, 0, L, [t[1:2] for t in plan])


# --------------------------------------------------------------- c4
@pytest.mark.parametrize("dtype,d,H_kv,n_mass,L,budget,lens", [
    ("bf16", 128, 2, 2, 500, 130, [500, 131, 100]),
    ("bf16", 64, 3, 1, 300, 64, [300, 65]),
    ("fp32", 128, 1, 1, 257, 200, [257, 256]),
    ("fp32", 64, 4, 4, 90, 7, [90, 8, 7, 0]),
    ("bf16", 128, 4, 4, 2112, 2048, [2112, 2049]),
])
@pytest.mark.parametrize("book", [True, False])
def test_evict_then_compact(dtype, d, H_kv, n_mass, L, budget, lens, book, cuda_device):
    B, dt, sid = len(lens), DT[dtype], 52000 + L
    K, V, table = _cache(sid, B, H_kv, d, lens, L, dt)
    desc = _desc(B, H_kv, H_kv, d, L, dtype, n_slots=K.shape[0])
    mass = synth.uniforms(SEED, sid + 990, 0, B * n_mass * L).reshape(B, n_mass, L).float()
    pos = torch.argsort(mass, dim=-1).to(torch.int32)
    dev = lambda t: t.to(cuda_device)  # noqa: E731
    Kd, Vd, md, pd = dev(K), dev(V), dev(mass), dev(pos)
    plan = pipeline.eviction_buffers(desc, n_mass, budget, cuda_device)
    new = torch.empty(B, dtype=torch.int32, device=cuda_device)
    if book:
        pipeline.evict(desc, Kd, Vd, dev(table), dev(torch.tensor(lens, dtype=torch.int32)), new, md, budget=budget,
                       n_first=3, n_recent=min(4, budget - 3), plan=plan, tok_pos=pd)
    else:
        dl.dl_evict_select(desc, md, pd, dev(torch.tensor(lens, dtype=torch.int32)), budget, 3, min(4, budget - 3), *plan,
                           new)
        dl.dl_cache_compact(desc, *plan, dev(table), Kd, Vd)
    assert dl.dl_get_status() == dl.DL_OK
    Kr, Vr, mr, pr = np_(K), np_(V), np_(mass), np_(pos)
    for b, n in enumerate(lens):
        for m in range(n_mass):
            h, f = oracle.evict_plan(mr[b, m, :n], pr[b, m, :n], budget, 3, min(4, budget - 3))
            for g in range(H_kv) if n_mass == 1 else [m]:
                oracle.compact_rows(Kr, np_(table)[b], g, h, f, 64)
                oracle.compact_rows(Vr, np_(table)[b], g, h, f, 64)
            if book:
                mr[b, m, h], pr[b, m, h] = mr[b, m, f], pr[b, m, f]
    assert np.array_equal(np_(Kd), Kr, equal_nan=True) and np.array_equal(np_(Vd), Vr, equal_nan=True)
    assert np.array_equal(np_(md), mr) and np.array_equal(np_(pd), pr)
    assert new.tolist() == [min(n, budget) for n in lens]


def test_compact_bad_moves_are_reported_and_skipped(cuda_device):
    B, H_kv, d, L = 2, 2, 64, 200
    K, V, table = _cache(53000, B, H_kv, d, [200, 200], L, torch.bfloat16)
    desc = _desc(B, H_kv, H_kv, d, L, "bf16", n_slots=K.shape[0])
    dev = lambda t: t.to(cuda_device)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    good = ([[[0, 1], [5, 6]], [[2, 3], [4, 7]]], [[[100, 101], [150, 199]], [[120, 121], [130, 131]]])

    def run(hole, fill, cnt, tab):
        Kd, Vd = dev(K), dev(V)
        dl.dl_cache_compact(desc, i32(hole), i32(fill), i32(cnt), dev(tab), Kd, Vd)
        st, Kr = dl.dl_get_status(), np_(K)
        for b in range(B):
            for m in range(H_kv):
                for i in range(max(0, min(2, cnt[b][m]))):
                    to, fr = hole[b][m][i], fill[b][m][i]
                    if not (0 <= to < L and 0 <= fr < L):
                        continue
                    st_, sf = int(tab[b, to // 64]), int(tab[b, fr // 64])
                    if 0 <= st_ < desc.n_slots and 0 <= sf < desc.n_slots:
                        Kr[st_, m, to % 64] = np_(K)[sf, m, fr % 64]
        assert np.array_equal(np_(Kd), Kr, equal_nan=True)
        return st

    assert run(*good, [[2, 1], [0, 2]], table) == dl.DL_OK
    assert run(*good, [[2, 5], [-1, 2]], table) == dl.DL_ERR_BAD_INDEX        # counts
    assert run([[[0, -1], [5, 200]], [[2, 3], [4, 7]]], good[1], [[2, 2], [2, 2]], table) == dl.DL_ERR_BAD_INDEX
    assert run(good[0], [[[100, 2**31 - 1], [150, -5]], good[1][1]], [[2, 2], [2, 2]], table) == dl.DL_ERR_BAD_INDEX
    t2 = table.clone()
    t2[0, 1], t2[1, 0] = desc.n_slots, -1
    assert run(*good, [[2, 2], [2, 2]], t2) == dl.DL_ERR_BAD_INDEX


# --------------------------------------------------------------- far offsets
def test_rows_past_32_bit_offsets(cuda_device):
    """A pool of more than 2^32 elements: append, attention and moves in its
    last pages."""
    H_kv, d, L = 4, 128, 200
    n_slots = (1 << 32) // (H_kv * 64 * d) + 8
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * n_slots * H_kv * 64 * d * 2:
        pytest.skip("needs two pools of 8.6 GB")
    desc = _desc(1, 4, H_kv, d, L, "bf16", n_slots=n_slots)
    K, V = (torch.empty(n_slots, H_kv, 64, d, dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    table = torch.tensor([[n_slots - 1, 0, n_slots - 3, n_slots - 2]], dtype=torch.int32)
    td = table.to(cuda_device)
    x = _normal(54000, 1, L, 12 * d, dtype=torch.bfloat16).to(cuda_device)
    pos = torch.arange(L, dtype=torch.int32, device=cuda_device)[None]
    Q = torch.empty(1, 4, L, d, dtype=torch.bfloat16, device=cuda_device)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=cuda_device)  # noqa: E731
    dl.dl_qk_norm_rope(desc, x, pos, None, None, 0.0, None, Q, start=i32(0), page_table=td, K_pool=K, V_pool=V)
    small = [P[td[0].long()].cpu() for P in (K, V)]
    xs = np_(x)[0].reshape(L, 12, d)
    order = np.arange(L)
    assert np.array_equal(np_(small[0])[order // 64, :, order % 64], xs[:, 4:8])
    assert np.array_equal(np_(small[1])[order // 64, :, order % 64], xs[:, 8:])
    O, lse = torch.empty(1, 4, d, dtype=torch.bfloat16, device=cuda_device), torch.empty(1, 4, device=cuda_device)
    ws = pipeline.workspace(desc, cuda_device)
    q = Q[:, :, 7].contiguous()
    dl.dl_decode_attn(desc, q, K, V, td, i32(L), O, lse, ws)
    local = torch.arange(4, dtype=torch.int32)[None]
    _check_decode(q.cpu(), *small, local, [L], O, lse, None, None, 1.0, "bf16", H_kv, 0)
    dl.dl_cache_compact(desc, i32(0, 130).view(1, 1, 2), i32(70, 199).view(1, 1, 2), i32(2).view(1, 1), td, K, V)
    assert dl.dl_get_status() == dl.DL_OK
    after = np_(K[td[0].long()])
    assert np.array_equal(after[0, :, 0], np_(small[0])[1, :, 6]) and np.array_equal(after[2, :, 2], np_(small[0])[3, :, 7])


# --------------------------------------------------------------- together
def _token_model(dev, dtype="bf16", B=3, H=6, H_kv=2, d=64, L=140, layers=2, budget=96, per_head=True, decay=1.0):
    dt = DT[dtype]
    desc = _desc(B, H, H_kv, d, L, dtype, n_slots=B * 3 + 1)
    f = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float().to(dev)
    step = pipeline.TokenStep(desc, layers, dt, dev, inv_freq=f, budget=budget, n_first=2, n_recent=8, per_head=per_head,
                              decay=decay)
    table = _table(60000, B, desc.n_pages, desc.n_slots).to(dev)
    pools = [[torch.full((desc.n_slots, H_kv, 64, d), float("nan"), dtype=dt, device=dev) for _ in range(2)]
             for _ in range(layers)]
    w = [[(1 + 0.1 * _normal(60010 + 2 * l + j, d)).to(dt).to(dev) for j in range(2)] for l in range(layers)]
    return desc, step, table, pools, w


@pytest.mark.parametrize("per_head", [True, False])
def test_prompt_tokens_eviction_run_together(per_head, cuda_device):
    """A prompt, tokens until past the budget, an eviction, more tokens: after
    every step the cache, positions, masses and outputs follow the oracle run
    on the device's own cached rows (the rows are compared when written)."""
    B, H, H_kv, d, layers, budget, n0 = 3, 6, 2, 64, 2, 96, 90
    desc, step, table, pools, w = _token_model(cuda_device, per_head=per_head, decay=0.5)
    G, n_mass = H // H_kv, H_kv if per_head else 1
    f = np_(step.inv_freq)
    width = (H + 2 * H_kv) * d
    for l in range(layers):
        x = _normal(61000 + l, B, n0, width, dtype=torch.bfloat16).to(cuda_device)
        pos = torch.arange(n0, dtype=torch.int32, device=cuda_device).expand(B, n0).contiguous()
        q = torch.empty(B, H, n0, d, dtype=torch.bfloat16, device=cuda_device)
        step.append(l, x, pos, *w[l], *pools[l], table, q)
    step.advance()
    # a ragged batch: sequence 1 counts only 40 tokens of its prompt
    step.start.copy_(torch.tensor([n0, 40, n0], dtype=torch.int32))
    at = [n0, 40, n0]
    for i in range(12):
        lens0 = step.start.tolist()
        for l in range(layers):
            x = _normal(62000 + 10 * i + l, B, 1, width, dtype=torch.bfloat16)
            pos = torch.tensor([[at[b] + i] for b in range(B)], dtype=torch.int32)
            mass0 = step.tok_mass[l].clone()
            O = step.attend(l, x.to(cuda_device), pos.to(cuda_device), *w[l], *pools[l], table)
            assert dl.dl_get_status() == dl.DL_OK
            K, V = (P.cpu() for P in pools[l])
            lens = [n + 1 for n in lens0]
            xs = np_(x)[:, 0].reshape(B, -1, d)
            for b in range(B):
                for g in range(H_kv):
                    key = np_(K)[int(table[b, lens0[b] // 64]), g, lens0[b] % 64]
                    ref = oracle.norm_rotate(xs[b, H + g], int(pos[b]), np_(w[l][1]), 1e-6, f, False)
                    assert np.abs(key - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-5
                mass0[b, :, lens0[b]] = 0
            _check_decode(step.Q[:, :, 0].cpu(), K, V, table.cpu(), lens, O, step.lse[l], mass0, step.tok_mass[l], 0.5,
                          "bf16", H_kv, n_mass, f"token {i} layer {l}")
            assert [int(step.tok_pos[l][b, 0, lens0[b]]) for b in range(B)] == pos[:, 0].tolist()
        if i in (5, 9):
            before = [([P.cpu().clone() for P in pools[l]], np_(step.tok_mass[l]), np_(step.tok_pos[l])) for l in range(layers)]
            ends = step.end.tolist()
            step.evict([p[0] for p in pools], [p[1] for p in pools], table)
            assert dl.dl_get_status() == dl.DL_OK
            assert step.start.tolist() == [min(n, budget) for n in ends]
            for l in range(layers):
                (K, V), m, p = before[l]
                Kr, Vr = np_(K), np_(V)
                for b in range(B):
                    for a in range(n_mass):
                        n = ends[b]
                        h, fl = oracle.evict_plan(m[b, a, :n], p[b, a, :n], budget, 2, 8)
                        for g in range(H_kv) if n_mass == 1 else [a]:
                            oracle.compact_rows(Kr, np_(table)[b], g, h, fl, 64)
                            oracle.compact_rows(Vr, np_(table)[b], g, h, fl, 64)
                        m[b, a, h], p[b, a, h] = m[b, a, fl], p[b, a, fl]
                assert np.array_equal(np_(pools[l][0]), Kr, equal_nan=True)
                assert np.array_equal(np_(pools[l][1]), Vr, equal_nan=True)
                assert np.array_equal(np_(step.tok_mass[l]), m) and np.array_equal(np_(step.tok_pos[l]), p)
        else:
            step.advance()


def test_captured_step_replays_with_new_inputs(cuda_device):
    """A whole step (two layers, then the cut) captured once and replayed on
    new tokens gives what eager calls give, bit for bit."""
    B, H, H_kv, d, layers = 3, 6, 2, 64, 2
    width = (H + 2 * H_kv) * d
    got = {}
    for how in ("eager", "graph"):
        desc, step, table, pools, w = _token_model(cuda_device, budget=70)
        x = [torch.zeros(B, 1, width, dtype=torch.bfloat16, device=cuda_device) for _ in range(layers)]
        pos = torch.zeros(B, 1, dtype=torch.int32, device=cuda_device)
        for l in range(layers):
            p = _normal(63000 + l, B, 69, width, dtype=torch.bfloat16).to(cuda_device)
            pp = torch.arange(69, dtype=torch.int32, device=cuda_device).expand(B, 69).contiguous()
            step.append(l, p, pp, *w[l], *pools[l], table, torch.empty(B, H, 69, d, dtype=torch.bfloat16, device=cuda_device))
        step.advance()

        def body():
            for l in range(layers):
                step.attend(l, x[l], pos, *w[l], *pools[l], table)
            step.evict([q[0] for q in pools], [q[1] for q in pools], table)

        if how == "graph":
            saved = [t.clone() for t in [step.start, *step.tok_pos, *step.tok_mass, *(t for q in pools for t in q)]]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                body()
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                body()
            for t, s in zip([step.start, *step.tok_pos, *step.tok_mass, *(t for q in pools for t in q)], saved):
                t.copy_(s)
        seen = []
        for i in range(6):
            for l in range(layers):
                x[l].copy_(_normal(64000 + 10 * i + l, B, 1, width, dtype=torch.bfloat16))
            pos.fill_(69 + i)
            graph.replay() if how == "graph" else body()
            seen += [step.O[l].clone() for l in range(layers)] + [step.start.clone()] + [t.clone() for t in step.tok_mass]
        assert dl.dl_get_status() == dl.DL_OK
        got[how] = seen + [t for q in pools for t in q]
    for a, b in zip(got["eager"], got["graph"]):
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


def test_two_streams_at_once(cuda_device):
    """Two decodings with workspaces of their own on two streams."""
    args = []
    for k in range(2):
        lens = [700, 130, 3]
        K, V, table = _cache(65000 + 1000 * k, 3, 4, 128, lens, 700, torch.bfloat16)
        desc = _desc(3, 8, 4, 128, 700, "bf16", n_slots=K.shape[0])
        Q = _normal(65990 + k, 3, 8, 128, dtype=torch.bfloat16)
        dev = [t.to(cuda_device) for t in (Q, K, V, table, torch.tensor(lens, dtype=torch.int32))]
        out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device=cuda_device), torch.empty(3, 8, device=cuda_device)
        args.append((desc, dev, out, pipeline.workspace(desc, cuda_device), torch.cuda.Stream(),
                     torch.zeros(3, 4, 700, device=cuda_device), (Q, K, V, table, lens)))
    torch.cuda.synchronize()
    for _ in range(20):
        for desc, dev, out, ws, st, mass, _ in args:
            mass_arg = mass
            dl.dl_decode_attn(desc, *dev, *out, ws, tok_mass=mass_arg, decay=0.0, stream=st)
    torch.cuda.synchronize()
    for desc, dev, out, ws, st, mass, (Q, K, V, table, lens) in args:
        _check_decode(Q, K, V, table, lens, *out, torch.zeros(3, 4, 700), mass, 0.0, "bf16", 4, 4)


def _busy_run(dev, sync, body_streams=None):
    """Steps that leave no gap between the calls and the framework's and
    torch's own work on the same buffers; `sync` waits after every one."""
    B, H, H_kv, d, L, layers = 3, 6, 2, 64, 140, 2
    desc, step, table, pools, w = _token_model(dev, budget=64, decay=0.5)
    width = (H + 2 * H_kv) * d
    x = [_normal(66000 + l, B, 40, width, dtype=torch.bfloat16).to(dev) for l in range(layers)]
    base = torch.arange(40, dtype=torch.int32, device=dev).expand(B, 40).contiguous()
    q = torch.empty(B, H, 40, d, dtype=torch.bfloat16, device=dev)
    wait = torch.cuda.synchronize if sync else (lambda: None)
    n_blk = desc.n_pages
    kbar = torch.zeros(B, H_kv, n_blk, d, device=dev)
    seen = []
    for l in range(layers):
        step.append(l, x[l], base, *w[l], *pools[l], table, q)
        wait()
    step.advance()
    tok = torch.empty(B, 1, width, dtype=torch.bfloat16, device=dev)
    pos = torch.full((B, 1), 39, dtype=torch.int32, device=dev)
    for i in range(30):
        pos.add_(1)
        for l in range(layers):
            torch.add(x[l][:, i:i + 1], 0.25 * l, out=tok)
            wait()
            O = step.attend(l, tok, pos, *w[l], *pools[l], table)
            wait()
            seen += [O.clone(), step.lse[l].clone()]
            O.zero_()
            tok.zero_()
            # a kernel of the framework between two of the calls
            new = x[l][:, :2, :H_kv * d].reshape(B, 2, H_kv, d).transpose(1, 2).contiguous()
            dl.dl_cache_write(desc, new, new, torch.full((B,), i % 20, dtype=torch.int32, device=dev), table, *pools[l], kbar)
            wait()
        if i % 3 == 2:
            step.evict([p[0] for p in pools], [p[1] for p in pools], table)
        else:
            step.advance()
        wait()
        seen += [step.start.clone(), *(t.clone() for t in step.tok_mass), *(t.clone() for t in step.tok_pos)]
    assert dl.dl_get_status() == dl.DL_OK
    return seen + [t for p in pools for t in p]


def test_calls_without_gaps_see_each_others_results(cuda_device):
    """The calls are launched programmatically (their start overlaps the end of
    what comes before): with nothing waiting between them, torch's kernels and
    the framework's on the same buffers, they give what they give when every
    call is waited for."""
    for a, b in zip(_busy_run(cuda_device, False), _busy_run(cuda_device, True)):
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


def test_captured_on_forked_streams(cuda_device):
    """A capture that forks: two sequences' decodings on two streams between an
    append and an eviction on the first; replayed twice on new inputs."""
    dev, H_kv, d, L = cuda_device, 2, 64, 200
    desc = _desc(1, 4, H_kv, d, L, "bf16", n_slots=4)
    table = torch.arange(4, dtype=torch.int32, device=dev)[None]
    K, V = (_normal(67000 + j, 4, H_kv, 64, d, dtype=torch.bfloat16).to(dev) for j in range(2))
    x = torch.zeros(1, 1, 8 * d, dtype=torch.bfloat16, device=dev)
    pos, start, end, new = (torch.zeros(1, dtype=torch.int32, device=dev) for _ in range(4))
    Q = torch.empty(1, 4, 1, d, dtype=torch.bfloat16, device=dev)
    mass = torch.zeros(1, H_kv, L, device=dev)
    out = [torch.empty(1, 4, d, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    ws = [pipeline.workspace(desc, dev) for _ in range(2)]
    plan = pipeline.eviction_buffers(desc, H_kv, 120, dev)
    side = torch.cuda.Stream()

    def body():
        dl.dl_qk_norm_rope(desc, x, pos[None], None, None, 1e-6, None, Q, start=start, page_table=table, K_pool=K,
                           V_pool=V, end=end, tok_mass=mass)
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        dl.dl_decode_attn(desc, Q, K, V, table, end, out[0], None, ws[0], tok_mass=mass, decay=0.5)
        dl.dl_decode_attn(desc, Q, K, V, table, start, out[1], None, ws[1], stream=side)
        main.wait_stream(side)
        pipeline.evict(desc, K, V, table, end, new, mass, budget=120, n_first=1, n_recent=4, plan=plan)

    state = [K.clone(), V.clone(), mass.clone()]

    def reset(i):
        for t, s in zip((K, V, mass), state):
            t.copy_(s)
        x.copy_(_normal(67010 + i, 1, 1, 8 * d, dtype=torch.bfloat16))
        pos.fill_(150 + i), start.fill_(150 + i)

    want = []
    for i in range(2):
        reset(i)
        body()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (*out, K, V, mass, new, end, *plan)])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for i in range(2):
        reset(i)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*out, K, V, mass, new, end, *plan), want[i]):
            assert torch.equal(a, b)
    assert dl.dl_get_status() == dl.DL_OK


@pytest.mark.parametrize("what", ["dtype", "size", "strided", "host", "rows"])
def test_buffers_that_do_not_fit_are_refused(what, cuda_device):
    """Wrong tensors never reach the library: ValueError, nothing written."""
    dev, B, H, H_kv, d, L = cuda_device, 2, 4, 2, 64, 100
    desc = _desc(B, H, H_kv, d, L, "bf16")
    good = dict(Q=torch.zeros(B, H, d, dtype=torch.bfloat16, device=dev),
                K_pool=torch.zeros(desc.n_slots, H_kv, 64, d, dtype=torch.bfloat16, device=dev),
                V_pool=torch.zeros(desc.n_slots, H_kv, 64, d, dtype=torch.bfloat16, device=dev),
                page_table=torch.zeros(B, 2, dtype=torch.int32, device=dev),
                ctx_len=torch.zeros(B, dtype=torch.int32, device=dev),
                O=torch.full((B, H, d), 7.0, dtype=torch.bfloat16, device=dev), lse=torch.zeros(B, H, device=dev),
                ws=pipeline.workspace(desc, dev), tok_mass=torch.zeros(B, H_kv, L, device=dev))
    for name in good:
        bad = dict(good)
        t = bad[name]
        if what == "dtype":
            if name == "ws":
                continue
            bad[name] = t.double()
        elif what == "size":
            if name == "ws":
                continue
            bad[name] = torch.zeros(t.numel() + 1, dtype=t.dtype, device=dev)[1:-1].clone() if name != "tok_mass" \
                else torch.zeros(B, H_kv, L + 1, device=dev)
        elif what == "strided":
            wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device=dev)
            bad[name] = wide[..., ::2]
        elif what == "host":
            bad[name] = t.cpu()
        elif name != "tok_mass":
            continue
        else:
            bad[name] = torch.zeros(B, L, H_kv, device=dev)   # rows and tokens swapped
        with pytest.raises((ValueError, dl.DLError)):
            dl.dl_decode_attn(desc, **bad)
    torch.cuda.synchronize()
    assert (good["O"] == 7).all()
    dl.dl_decode_attn(desc, **good)
    assert dl.dl_get_status() == dl.DL_OK and (good["O"] == 0).all()


def test_streams_by_object_and_by_handle(cuda_device):
    desc = _desc(1, 2, 2, 64, 64, "fp32")
    x = _normal(68000, 1, 3, 6 * 64).to(cuda_device)
    pos = torch.arange(3, dtype=torch.int32, device=cuda_device)[None]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    outs = []
    for stream in (None, st, st.cuda_stream):
        o = [torch.empty(1, 2, 3, 64, device=cuda_device) for _ in range(3)]
        torch.cuda.synchronize()
        dl.dl_qk_norm_rope(desc, x, pos, None, None, 0.0, None, *o, stream=stream)
        torch.cuda.synchronize()
        outs.append(o)
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_sink_masses_cut_a_denoising_context(cuda_device):
    """The diffusion path: column masses of a denoising step (dl_sink_mass)
    decide which context stays; the cut cache serves dl_pool_keys and the
    dense attention of the next step, which then equals the oracle's over the
    kept tokens."""
    wl = synth.workload("llada8k", L_ctx=640, H=4, H_kv=4)
    inp = synth.make_step_inputs(wl, device=cuda_device)
    B, L, budget = wl.batch, wl.L_ctx, 320
    desc = dl.make_desc(B, wl.H, wl.H_kv, wl.d, L, wl.L_q, 64, wl.n_pages, wl.n_slots, dl.DL_BF16)
    ws = pipeline.workspace(desc, cuda_device)
    q_idx = torch.arange(wl.L_q, dtype=torch.int32, device=cuda_device).expand(B, wl.L_q).contiguous()
    q_cnt = torch.full((B,), wl.L_q, dtype=torch.int32, device=cuda_device)
    mass = torch.empty(B, 1, L, device=cuda_device)
    dl.dl_sink_mass(desc, inp.q_dec, q_idx, q_cnt, inp.k_pool, inp.page_table, inp.k_dec, mass, ws)
    K0, V0 = inp.k_pool.cpu().clone(), inp.v_pool.cpu().clone()
    lens = torch.full((B,), L, dtype=torch.int32, device=cuda_device)
    new = torch.empty_like(lens)
    m = np_(mass)
    pipeline.evict(desc, inp.k_pool, inp.v_pool, inp.page_table, lens, new, mass, budget=budget, n_first=1, n_recent=64,
                   plan=pipeline.eviction_buffers(desc, 1, budget, cuda_device))
    assert dl.dl_get_status() == dl.DL_OK and new.tolist() == [budget] * B
    cut = dl.make_desc(B, wl.H, wl.H_kv, wl.d, budget, wl.L_q, 64, wl.n_pages, wl.n_slots, dl.DL_BF16)
    O = torch.empty(B, wl.L_q, wl.H, wl.d, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.empty(B, wl.H, wl.L_q, device=cuda_device)
    dl.dl_sparse_attn(cut, inp.q_dec, inp.k_pool, inp.v_pool, inp.page_table, None, None, inp.k_dec, inp.v_dec, O, lse, ws)
    assert dl.dl_get_status() == dl.DL_OK
    for b in range(B):
        holes, fills = oracle.evict_plan(m[b, 0], None, budget, 1, 64)
        stay = np.array(sorted((set(range(budget)) - set(holes)) | set(fills)))
        for g in range(wl.H_kv):
            k = oracle.steps.gather_context(K0, np_(inp.page_table)[b], g, stay, 64)
            v = oracle.steps.gather_context(V0, np_(inp.page_table)[b], g, stay, 64)
            k = np.concatenate([k, np_(inp.k_dec)[b, g]])
            v = np.concatenate([v, np_(inp.v_dec)[b, g]])
            ref, _ = oracle.attention_rows(np_(inp.q_dec)[b, g], k, v, oracle.scale_for(wl.d))
            err = np.abs(np_(O)[b, :, g] - ref)
            assert err.max() <= 2e-2 and err.mean() <= 2e-3  # the framework's bar for this kernel
