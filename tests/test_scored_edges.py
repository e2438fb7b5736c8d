"""Scaled rotary frequencies, arguments and imports of the scored entry points at their edges (all on the CPU)."""

import math

import pytest
import torch

import attention_sm_flashattention_gb300 as fa


@pytest.mark.parametrize("rot,base", [(64, 10000.0), (128, 10000.0), (128, 500000.0), (16, 100.0)])
@pytest.mark.parametrize("original_len", [4, 7, 200, 4096, 65536, 131072, 1 << 20, 1 << 30])
def test_yarn_ramp(rot, base, original_len):
    """Pairs that turn less than beta_slow times within original_len are divided by the whole factor, pairs that turn
    more than beta_fast times are kept, and in between the share of the division grows evenly from pair to pair."""
    factor, fast, slow = 4.0, 32.0, 1.0
    plain, _ = fa.rotary_freqs(rot, base, device="cpu")
    yarn, _ = fa.rotary_freqs(rot, base, "yarn", factor, original_len, fast, slow, device="cpu")
    turns = plain * original_len / (2 * math.pi)
    share = (1 - yarn / plain) / (1 - 1 / factor)  # 0: kept, 1: divided
    # the ramp starts at the last pair that turns more than beta_fast times (the first pair, where none does) and
    # ends at the first that turns less than beta_slow times, as if there were pairs past the last
    first = max(0, math.floor(math.log(original_len / (fast * 2 * math.pi), base) * rot / 2))
    last = math.ceil(math.log(original_len / (slow * 2 * math.pi), base) * rot / 2)
    for j in range(rot // 2):
        if j >= last:
            want = 1.0
        elif j <= first:
            want = 0.0
        else:
            want = (j - first) / (last - first)
        assert abs(float(share[j]) - want) < 1e-12, j
    assert (share[turns < slow] > 1 - 1e-12).all() and (share[turns > fast].abs() < 1e-12).all()
    assert (yarn[1:] < yarn[:-1]).all()


def test_yarn_last_pair_of_a_long_context():
    # 64 values, 131072 positions: the last pair turns 2.8 times, so it is on the ramp (22 .. 35), not behind it
    plain, _ = fa.rotary_freqs(64, device="cpu")
    yarn, _ = fa.rotary_freqs(64, scaling="yarn", factor=4.0, original_len=131072, device="cpu")
    assert abs(float(yarn[-1] / plain[-1]) - (1 - 9 / 13 * 0.75)) < 1e-12


def test_package_imports_without_torchs_cuda_bindings():
    """A CPU build of torch has no CUDA names in torch._C: the parts that need no GPU still work there."""
    import subprocess
    import sys
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda')]:\n"
            "    delattr(torch._C, n)\n"
            "import attention_sm_flashattention_gb300 as fa\n"
            "assert fa.rotary_freqs(8, device='cpu')[0].numel() == 4\n"
            "try:\n"
            "    fa.fwd_scored(*[torch.zeros((1, 1, 8, 64), dtype=torch.float16)] * 3)\n"
            "except ValueError:\n"
            "    print('refused')\n")
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                         cwd=__file__.rsplit("/", 2)[0])
    assert run.returncode == 0 and run.stdout.strip() == "refused", run.stderr[-2000:]


def test_arguments_past_the_c_types():
    from attention_sm_flashattention_gb300 import scored
    top = 2 ** 31 - 1
    for n in (0, 1, -1, top, 1 - 2 ** 31):
        assert scored._c_int(n) == n
    for n in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 70):
        assert scored._c_int(n) == top and scored._c_int(-n) == -top
    for x in (0.0, 1e-38, 30.0, -1.0, math.inf, -math.inf, 2.0 ** -149):
        assert scored._c_cap(x) == x
    for x in (1e-46, 1e-300, 2.0 ** -150):
        assert scored._c_cap(x) == 2.0 ** -149 and scored._c_cap(-x) == -2.0 ** -149
    assert math.isnan(scored._c_cap(math.nan))


def test_workspaces_have_the_memory_they_name():
    """A view with strides names more bytes than are its own; kernels would write past them."""
    from attention_sm_flashattention_gb300 import api
    for t in (torch.empty(1, dtype=torch.uint8).expand(4096), torch.empty(64, dtype=torch.uint8)[::2],
              torch.empty((8, 8), dtype=torch.float32).t()):
        with pytest.raises(ValueError, match="contiguous"):
            api._workspace(t)
    with pytest.raises(ValueError, match="CUDA"):
        api._workspace(torch.empty(64, dtype=torch.uint8))
    with pytest.raises(TypeError):
        api._workspace(4096)


def test_oracle_rows_before_position_zero():
    import numpy as np
    from oracle import scored as orc
    g = torch.Generator().manual_seed(1)
    q, kc, vc = (torch.randn(s, generator=g) for s in ((1, 1, 5, 8), (2, 4, 1, 8), (2, 4, 1, 8)))
    for causal in (False, True):
        o, lse, _, _ = orc.paged_scored_fwd(q, kc, vc, [[1, 0]], [3], [5], causal, 0.3)
        want, rl, _, _ = orc.paged_scored_fwd(q[:, :, 2:], kc, vc, [[1, 0]], [3], None, causal, 0.3)
        assert not o[0, 0, :2].any() and np.isneginf(lse[0, 0, :2]).all()
        assert np.array_equal(o[:, :, 2:], want) and np.array_equal(lse[:, :, 2:], rl)


def test_outputs_that_overlap_themselves_are_refused():
    """Two values of an output in one place of memory: threads would race for it."""
    from attention_sm_flashattention_gb300 import scored
    buf = torch.empty(1 << 16, dtype=torch.float16)
    qkv = buf[:2 * 5 * 8 * 64].view(2, 5, 8, 64)  # [Z, N, heads, D]
    for t in (qkv, qkv.transpose(1, 2), qkv[:, :, 2:5].transpose(1, 2), qkv[:, ::2, :, :16].transpose(1, 2),
              buf.as_strided((1, 4, 1, 64), (7, 64, 3, 1)), buf.as_strided((2, 0, 3, 64), (1, 1, 1, 1))):
        scored._written("out", t)
    for size, stride in (((2, 3, 4, 64), (0, 256, 64, 1)), ((1, 3, 4, 64), (0, 64, 32, 1)), ((1, 2, 3, 64), (9, 64, 64, 1)),
                         ((2, 3, 4, 64), (700, 256, 64, 1)), ((1, 1, 2, 64), (1, 1, 63, 1))):
        with pytest.raises(ValueError):
            scored._written("out", buf.as_strided(size, stride))
