"""Refusals of the token-by-token entry points on a host without a GPU: every
bad argument is rejected before anything is launched, with nothing changed."""
import ctypes

import pytest
import torch

import long_context_diffusion_b200 as dl
from long_context_diffusion_b200 import _abi, pipeline

FAKE = 0x10000
ODD = 0x10008


def _desc(**kw):
    base = dict(batch=2, H=28, H_kv=4, d=128, L_ctx=1000, L_q=1, page=64, n_pages=16, n_slots=32,
                dtype=dl.DL_BF16)
    base.update(kw)
    return dl.make_desc(**base)


def _call(name, desc, args, **over):
    a = dict(args)
    assert set(over) <= set(a), over
    a.update(over)
    st = getattr(_abi.lib, name)(ctypes.byref(desc) if desc else None, *a.values())
    return st, _abi.lib.dl_last_error_message().decode()


ROPE = dict(qkv=FAKE, qkv_stride=36 * 128, n_tok=1, pos=FAKE, q_weight=FAKE, k_weight=FAKE,
            eps=1e-6, inv_freq=FAKE, rot_dim=128, interleaved=0, Q_out=FAKE, K_out=FAKE, V_out=FAKE,
            start=FAKE, page_table=FAKE, K_pool=FAKE, V_pool=FAKE, end=FAKE * 2, tok_pos=FAKE,
            tok_mass=FAKE, n_mass=4, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(qkv=None), 1), (dict(pos=None), 1), (dict(Q_out=None), 1), (dict(inv_freq=None), 1),
    (dict(K_out=None), 1), (dict(V_out=None), 1),                   # together
    (dict(start=None), 1), (dict(page_table=None), 1), (dict(K_pool=None), 1), (dict(V_pool=None), 1),
    (dict(start=None, page_table=None, K_pool=None, V_pool=None), 1),  # end without the cache
    (dict(start=None, page_table=None, K_pool=None, V_pool=None, end=None, tok_pos=None,
          tok_mass=None, K_out=None, V_out=None), 1),               # nowhere to put the keys
    (dict(end=FAKE), 1),                                            # the buffer of start
    (dict(n_mass=2), 1), (dict(n_mass=0), 1),
    (dict(n_tok=0), 1), (dict(n_tok=1 << 30), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(rot_dim=-8), 1), (dict(rot_dim=136), 1), (dict(rot_dim=12), 2),
    (dict(qkv_stride=36 * 128 - 8), 1), (dict(qkv_stride=36 * 128 + 4), 1),
    (dict(qkv=ODD), 1), (dict(q_weight=ODD), 1), (dict(k_weight=ODD), 1), (dict(Q_out=ODD), 1),
    (dict(K_out=ODD), 1), (dict(V_out=ODD), 1), (dict(K_pool=ODD), 1), (dict(V_pool=ODD), 1),
])
def test_qk_norm_rope_refusals(over, status):
    st, msg = _call("dl_qk_norm_rope", _desc(), ROPE, **over)
    assert st == status and msg, over


DECODE = dict(Q=FAKE, K_pool=FAKE, V_pool=FAKE, page_table=FAKE, ctx_len=FAKE, O=FAKE, lse=FAKE,
              tok_mass=FAKE, n_mass=4, decay=1.0, ws=FAKE, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(Q=None), 1), (dict(K_pool=None), 1), (dict(V_pool=None), 1), (dict(page_table=None), 1),
    (dict(ctx_len=None), 1), (dict(O=None), 1), (dict(Q=ODD), 1), (dict(K_pool=ODD), 1),
    (dict(V_pool=ODD), 1), (dict(O=ODD), 1), (dict(n_mass=3), 1), (dict(decay=-0.1), 1),
    (dict(decay=1.5), 1), (dict(decay=float("nan")), 1), (dict(ws=None), 3), (dict(ws_bytes=256), 3),
    (dict(ws=FAKE + 16), 3),
])
def test_decode_attn_refusals(over, status):
    st, msg = _call("dl_decode_attn", _desc(), DECODE, **over)
    assert st == status and msg, over


def test_decode_attn_takes_one_token_only():
    st, msg = _call("dl_decode_attn", _desc(L_q=2), DECODE)
    assert st == dl.DL_ERR_UNSUPPORTED and "L_q" in msg


EVICT = dict(tok_mass=FAKE, tok_pos=FAKE, n_mass=4, ctx_len=FAKE, budget=400, n_first=4,
             n_recent=100, hole_idx=FAKE, fill_idx=FAKE, max_move=400, move_cnt=FAKE,
             new_len=FAKE * 2, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(tok_mass=None), 1), (dict(ctx_len=None), 1), (dict(move_cnt=None), 1),
    (dict(new_len=None), 1), (dict(hole_idx=None), 1), (dict(fill_idx=None), 1),
    (dict(new_len=FAKE), 1),                                        # the buffer of ctx_len
    (dict(n_mass=2), 1), (dict(budget=0), 1), (dict(n_first=-1), 1), (dict(n_recent=-1), 1),
    (dict(n_first=301), 1), (dict(n_first=2**31 - 1, n_recent=2**31 - 1), 1),
    (dict(max_move=399), 1), (dict(budget=700, max_move=299), 1), (dict(max_move=-1), 1),
])
def test_evict_select_refusals(over, status):
    st, msg = _call("dl_evict_select", _desc(), EVICT, **over)
    assert st == status and msg, over


COMPACT = dict(hole_idx=FAKE, fill_idx=FAKE, move_cnt=FAKE, max_move=400, n_mass=4,
               page_table=FAKE, K_pool=FAKE, V_pool=FAKE, tok_pos=FAKE, tok_mass=FAKE, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(hole_idx=None), 1), (dict(fill_idx=None), 1), (dict(move_cnt=None), 1),
    (dict(page_table=None), 1), (dict(K_pool=None), 1), (dict(V_pool=None), 1),
    (dict(K_pool=ODD), 1), (dict(V_pool=ODD), 1), (dict(n_mass=0), 1), (dict(max_move=-1), 1),
])
def test_cache_compact_refusals(over, status):
    st, msg = _call("dl_cache_compact", _desc(), COMPACT, **over)
    assert st == status and msg, over


@pytest.mark.parametrize("name,args", [("dl_qk_norm_rope", ROPE), ("dl_decode_attn", DECODE),
                                       ("dl_evict_select", EVICT), ("dl_cache_compact", COMPACT)])
def test_descriptor_is_checked(name, args):
    assert _call(name, None, args)[0] == dl.DL_ERR_INVALID_ARG
    for kw in (dict(d=96), dict(page=32), dict(H=30), dict(batch=0), dict(n_pages=3), dict(dtype=7)):
        assert _call(name, _desc(**kw), args)[0] in (dl.DL_ERR_INVALID_ARG, dl.DL_ERR_UNSUPPORTED), kw


def test_decode_attn_capacity_limit():
    big = _desc(L_ctx=(1 << 30) + 1, n_pages=(1 << 24) + 1)
    st, msg = _call("dl_decode_attn", big, DECODE)
    assert st == dl.DL_ERR_UNSUPPORTED and "L_ctx" in msg


@pytest.mark.parametrize("name,args", [("dl_decode_attn", DECODE), ("dl_cache_compact", COMPACT)])
def test_pools_of_2_31_rows_are_refused(name, args):
    st, msg = _call(name, _desc(n_slots=1 << 23), args)
    assert st == dl.DL_ERR_UNSUPPORTED and "rows" in msg


def test_workspace_holds_the_dot_products_of_single_token_descriptors():
    one = dl.dl_workspace_size(_desc())
    assert one % 256 == 0 and one >= 2 * 28 * 1024 * 4      # batch, H, L_ctx padded to tiles
    # DECODE's call is refused with one byte less than it needs
    with_mass = DECODE | dict(ws_bytes=2 * 28 * 1024 * 4)
    assert _call("dl_decode_attn", _desc(), with_mass)[0] == dl.DL_ERR_WORKSPACE


def test_token_step_without_a_budget_has_nothing_to_evict():
    step = object.__new__(pipeline.TokenStep)
    step.budget = 0
    with pytest.raises(ValueError, match="budget"):
        step.evict([], [], None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="a host without a GPU")
def test_host_tensors_are_refused():
    desc = _desc(batch=1, H=1, H_kv=1, d=64)
    x = torch.zeros(1, 1, 192, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="current CUDA device"):
        dl.dl_qk_norm_rope(desc, x, i, None, None, 1e-6, None, x, x, x)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dl.dl_decode_attn(desc, q, q, q, i, i, q, None, q)
    m = torch.zeros(1, 1, 1000)
    with pytest.raises(ValueError):
        dl.dl_evict_select(desc, m, None, i, 100, 0, 0, None, None, i, i)
    with pytest.raises(ValueError):
        dl.dl_cache_compact(desc, m, m, i, i, q, q)


def test_wrong_objects_are_refused():
    desc = _desc(batch=1, H=1, H_kv=1, d=64)
    with pytest.raises(TypeError, match="torch.Tensor"):
        dl.dl_qk_norm_rope(desc, 3, None, None, None, 1e-6, None, None)
    with pytest.raises(TypeError):
        dl.dl_decode_attn("desc", None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError):
        dl.dl_evict_select(desc, torch.zeros(1, 1, 1000), None, None, 1 << 40, 0, 0, None, None, None, None)
    with pytest.raises(ValueError, match="current CUDA device"):  # nothing but None: no device
        dl.dl_cache_compact(desc, None, None, None, None, None, None)


def test_the_extension_checks_its_argument_count():
    with pytest.raises(TypeError, match="number of arguments"):
        _abi._calls.decode_attn(_desc())
