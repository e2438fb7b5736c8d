"""Scored kernels with several rounds of work units per SM, every kind of score: units handed out by the GPU, the
hand-over of Q, O and row sums between them, and the backward's second and later units.  192 heads of three query tiles
(the last ragged) are 576 units in the forward and 288 or more in each backward kernel, on 152 SMs."""

import pytest
import torch

from test_scored_gpu import run_case
from test_scored_paged_gpu import run_case as paged_case

pytestmark = pytest.mark.gpu
KINDS = [(0.0, False), (20.0, False), (0.0, True), (20.0, True)]


@pytest.mark.parametrize("cap,bias", KINDS)
@pytest.mark.parametrize("D,mask", [(256, m) for m in ("causal", "window", "docs", "prefix", "ranges")]
                         + [(d, m) for d in (64, 128) for m in ("causal", "docs", "ranges")])
def test_rounds_of_units(D, mask, cap, bias):
    run_case(4, 48, 24, 300, 300, D, mask, cap, bias, torch.float16 if bias else torch.bfloat16, 91,
             wide=3.0 if cap else 1.0)


@pytest.mark.parametrize("cap,bias", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("Nq", [1, 140])
def test_rounds_of_paged_units(Nq, splits, D, cap, bias):
    g = torch.Generator().manual_seed(9)
    B, H, Hkv = (48, 8, 8) if Nq == 1 else (24, 8, 4)
    lens = [int(x) for x in torch.randint(Nq, 600, (B,), generator=g)]
    q_lens = [int(x) for x in torch.randint(0, Nq + 1, (B,), generator=g)]
    paged_case(B, H, Hkv, Nq, lens, D, 32, 92, q_lens=q_lens, cap=cap, bias=bias, splits=splits,
               dtype=torch.bfloat16 if cap else torch.float16, window=200 if bias else 0)
