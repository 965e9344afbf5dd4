"""The workspace of dl_decode_attn: with masses, without, and what TokenStep
takes (CPU)."""
import ctypes

import pytest
import torch

import long_context_diffusion_b200 as dl
from long_context_diffusion_b200 import _abi, pipeline
from tests.test_token_host import DECODE, _call, _desc


@pytest.mark.parametrize("dtype,size", [(dl.DL_BF16, 4), (dl.DL_FP32, 8)])
def test_dot_products_are_counted_with_masses_alone(dtype, size):
    desc = _desc(dtype=dtype)
    without, with_, every = dl.dl_decode_workspace_size(desc, False), dl.dl_decode_workspace_size(desc), \
        dl.dl_workspace_size(desc)
    assert with_ - without == 2 * 28 * 1024 * size  # batch, H, L_ctx in whole tiles
    assert every >= with_ and without % 256 == 0
    long = _desc(dtype=dtype, L_ctx=131072, n_pages=2048, n_slots=4096)
    assert dl.dl_decode_workspace_size(long, False) == without  # no part of it grows with the capacity


@pytest.mark.parametrize("masses", [True, False])
def test_the_call_refuses_a_byte_less(masses):
    n = dl.dl_decode_workspace_size(_desc(), masses)
    over = {} if masses else dict(tok_mass=None)
    assert _call("dl_decode_attn", _desc(), DECODE, ws_bytes=n - 1, **over)[0] == dl.DL_ERR_WORKSPACE


def test_descriptors_that_the_call_refuses_have_no_size():
    for kw, st in ((dict(L_q=2), 2), (dict(L_ctx=(1 << 30) + 1, n_pages=(1 << 24) + 1), 2), (dict(batch=0), 1)):
        with pytest.raises(dl.DLError) as e:
            dl.dl_decode_workspace_size(_desc(**kw))
        assert e.value.status == st, kw
    assert _abi.lib.dl_decode_workspace_size(ctypes.byref(_desc()), 1, None) == dl.DL_ERR_INVALID_ARG


@pytest.mark.parametrize("budget", [0, 300])
def test_token_step_takes_what_its_calls_need(budget):
    desc = _desc()
    step = pipeline.TokenStep(desc, 1, torch.bfloat16, "cpu", budget=budget)
    assert step.ws.numel() == dl.dl_decode_workspace_size(desc, budget > 0)
