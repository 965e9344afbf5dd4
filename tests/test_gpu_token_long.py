"""The attention of long caches in a running step: the kernel of equal runs and
the join kernel behind an append that has just written the lengths, captured,
replayed with growing lengths and run without gaps; masses that all heads of a
sequence share, on clusters and on runs.

Tolerances: those of test_gpu_token_step.py."""
import pytest
import torch

import long_context_diffusion_b200 as dl
from long_context_diffusion_b200 import pipeline
from tests.test_gpu_token_step import DT, _busy_run, _check_decode, _desc, _normal, _table

pytestmark = pytest.mark.gpu

# dtype, B, H, H_kv, d, L_ctx, per_head, prompt: which kernels a step's attention takes
STEPS = [
    ("bf16", 3, 6, 2, 64, 6000, True, 5200),      # runs + join
    ("bf16", 2, 96, 8, 128, 17000, False, 16300),  # runs + join, masses of 96 heads in two turns
    ("fp32", 2, 6, 2, 128, 5000, False, 700),     # runs + join, few tiles of the capacity
    ("bf16", 3, 6, 2, 64, 700, False, 500),       # clusters, then the join kernel for the masses
    ("fp32", 2, 96, 8, 64, 300, False, 200),
]


def _made(case, dev, budget):
    dtype, B, H, H_kv, d, L, per_head, n0 = case
    dt, layers = DT[dtype], 2
    desc = _desc(B, H, H_kv, d, L, dtype)
    f = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float().to(dev)
    step = pipeline.TokenStep(desc, layers, dt, dev, inv_freq=f, budget=budget, n_first=2, n_recent=8, per_head=per_head,
                              decay=0.5)
    table = _table(70000, B, desc.n_pages, desc.n_slots).to(dev)
    pools = [[_normal(70001 + 2 * l + j, desc.n_slots, H_kv, 64, d, dtype=dt).to(dev) for j in range(2)]
             for l in range(layers)]
    w = [[(1 + 0.1 * _normal(70010 + 2 * l + j, d)).to(dt).to(dev) for j in range(2)] for l in range(layers)]
    for l in range(layers):  # a cache as a prompt leaves it
        at = torch.arange(n0, dtype=torch.int32, device=dev)
        step.tok_pos[l][:, :, :n0] = at
    step.start.copy_(torch.tensor([n0 - 37 * b for b in range(B)], dtype=torch.int32))
    return desc, step, table, pools, w


def _inputs(case, n_steps, dev):
    dtype, B, H, H_kv, d = case[:5]
    width = (H + 2 * H_kv) * d
    return [[_normal(71000 + 2 * i + l, B, 1, width, dtype=DT[dtype]).to(dev) for l in range(2)] for i in range(n_steps)]


@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c)))
def test_step_without_gaps_sees_the_lengths_just_written(case, cuda_device):
    """Appends, attention and evictions with nothing waiting between them give
    what waited-for calls give, bit for bit; the newest token has its mass."""
    dtype, B, H, H_kv, d, L, per_head, n0 = case
    xs, got = _inputs(case, 9, cuda_device), []
    for wait in (lambda: None, torch.cuda.synchronize):
        desc, step, table, pools, w = _made(case, cuda_device, n0 + 3)
        pos = torch.zeros(B, 1, dtype=torch.int32, device=cuda_device)
        seen, new = [], []
        for i, x in enumerate(xs):
            pos.fill_(n0 + i)
            for l in range(2):
                O = step.attend(l, x[l], pos, *w[l], *pools[l], table)
                wait()
                seen += [O.clone(), step.lse[l].clone()]
                at = (step.end.long() - 1)[:, None, None].expand(-1, step.tok_mass[l].shape[1], 1)
                new.append(torch.gather(step.tok_mass[l], 2, at))
                O.zero_()
            if i % 4 == 3:
                step.evict([p[0] for p in pools], [p[1] for p in pools], table)
            else:
                step.advance()
            wait()
            seen += [step.start.clone(), *(t.clone() for t in step.tok_mass), *(t.clone() for t in step.tok_pos)]
        assert dl.dl_get_status() == dl.DL_OK
        assert all((t > 0).all() for t in new)
        got.append(seen + [t for p in pools for t in p])
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c)))
def test_captured_long_step_replays_with_growing_lengths(case, cuda_device):
    """A captured step of two layers, replayed while the lengths grow, against
    waited-for eager calls, bit for bit; the last step against the oracle."""
    dtype, B, H, H_kv, d, L, per_head, n0 = case
    xs, got = _inputs(case, 6, cuda_device), {}
    for how in ("eager", "graph"):
        desc, step, table, pools, w = _made(case, cuda_device, L)
        x = [t.clone() for t in xs[0]]
        pos = torch.zeros(B, 1, dtype=torch.int32, device=cuda_device)

        def body(wait=lambda: None):
            for l in range(2):
                step.attend(l, x[l], pos, *w[l], *pools[l], table)
                wait()
            step.advance()
            wait()

        if how == "graph":
            state = [step.start, *step.tok_pos, *step.tok_mass, *(t for q in pools for t in q)]
            saved = [t.clone() for t in state]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                body()
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                body()
            for t, s in zip(state, saved):
                t.copy_(s)
        seen = []
        for i in range(6):
            for l in range(2):
                x[l].copy_(xs[i][l])
            pos.fill_(n0 + i)
            mass0 = [t.cpu() for t in step.tok_mass] if i == 5 and how == "graph" else None
            graph.replay() if how == "graph" else body(torch.cuda.synchronize)
            seen += [t.clone() for l in range(2) for t in (step.O[l], step.lse[l], step.tok_mass[l])] + [step.start.clone()]
        assert dl.dl_get_status() == dl.DL_OK
        assert step.start.tolist() == [n0 - 37 * b + 6 for b in range(B)]
        got[how] = seen + [t for q in pools for t in q]
    for a, b in zip(got["eager"], got["graph"]):
        assert torch.equal(a, b)
    lens = step.start.tolist()
    for b in range(B):
        mass0[1][b, :, lens[b] - 1] = 0  # what the append leaves
    _check_decode(step.Q[:, :, 0].cpu(), pools[1][0].cpu(), pools[1][1].cpu(), table.cpu(), lens, step.O[1], step.lse[1],
                  mass0[1], step.tok_mass[1], 0.5, dtype, H_kv, step.tok_mass[1].shape[1])


def test_calls_without_gaps_behind_programmatic_launches_of_the_framework(kernel_flags, cuda_device):
    """The same with the framework's other kernels launched programmatically too."""
    want = _busy_run(cuda_device, True)
    kernel_flags(dl.DL_FLAG_PDL)
    for a, b in zip(_busy_run(cuda_device, False), want):
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))
