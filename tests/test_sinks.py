"""Windows with sinks on the CPU: the oracle's mask, the kernels' work units
(compiled for the host from the kernels' own header) and the refusals."""

import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import attention_sm_flashattention_gb300 as fa
from attention_sm_flashattention_gb300 import _native
from oracle import scored as orc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "attention_sm_flashattention_gb300", "csrc")
FAKE = 1 << 20  # an aligned non-null address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_native.LIB_PATH):
        from attention_sm_flashattention_gb300 import build
        build.build()
    return _native.lib()


def test_work_units(tmp_path):
    """Every tile with a visible pair once, partial results apart from each other (tests/sink_units.cu)."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = str(tmp_path / "sink_units")
    run = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O1", "-std=c++17",
                          "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                          os.path.join(ROOT, "tests", "sink_units.cu"), "-o", exe], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout


@pytest.mark.parametrize("Nq,Nk,window,sinks", [(1, 1, 1, 1), (7, 7, 2, 3), (3, 9, 4, 2), (9, 9, 1, 20), (5, 12, 30, 2)])
def test_oracle_mask(Nq, Nk, window, sinks):
    seen = orc.visible(Nq, Nk, causal=True, window=window, sinks=sinks)
    for i in range(Nq):
        p = i + Nk - Nq
        for j in range(Nk):
            assert seen[i, j] == (j <= p and (p - j < window or j < sinks))


def test_oracle_paged_equals_dense():
    g = torch.Generator().manual_seed(0)
    B, H, Hkv, Nq, n, D, page = 1, 2, 1, 3, 11, 8, 4
    q = torch.randn((B, H, Nq, D), generator=g)
    k, v = torch.randn((2, 12, Hkv, D), generator=g).unbind(0)
    kc, vc = (t.reshape(3, page, Hkv, D)[torch.tensor([1, 2, 0])] for t in (k, v))
    o, lse, _, _ = orc.paged_scored_fwd(q, kc, vc, np.array([[2, 0, 1]]), [n], None, True, 0.3, window=4, sinks=2)
    ro, rl, _, _ = orc.scored_fwd(q, *(t[:n].transpose(0, 1)[None] for t in (k, v)), 0.3,
                                  seen=lambda z: orc.visible(Nq, n, causal=True, window=4, sinks=2))
    assert np.abs(o - ro).max() < 1e-12 and np.abs(lse - rl).max() < 1e-12


def fwd(lib, Z=1, H=2, Hkv=1, Nq=300, Nk=300, D=64, scale=0.125, cap=0.0, window=100, sinks=4, dtype=0, q=FAKE, lse=FAKE):
    return lib.fa_fwd_sinks(q, FAKE, FAKE, FAKE, lse, Z, H, Hkv, Nq, Nk, D, scale, cap, window, sinks, dtype, None)


def bwd(lib, Nq=300, Nk=300, D=64, window=100, sinks=4, ws=FAKE, ws_bytes=None, dtype=0):
    need = lib.fa_bwd_sinks_workspace_size(1, 2, 1, Nq, Nk, D, window, sinks) if ws_bytes is None else ws_bytes
    return lib.fa_bwd_sinks(*[FAKE] * 9, ws, need, 1, 2, 1, Nq, Nk, D, 0.125, 0.0, window, sinks, dtype, None)


def paged(lib, window=100, sinks=4, D=64, page=16, splits=1, ws=None, ws_bytes=0, dtype=0, max_pages=40):
    return lib.fa_fwd_paged_sinks(*[FAKE] * 5, None, FAKE, FAKE, ws, ws_bytes, 2, 2, 1, 1, D, 50, page, max_pages, splits, 0.125,
                                  0.0, window, sinks, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(sinks=-1), _native.FA_ERR_INVALID_ARG),
    (dict(window=-1), _native.FA_ERR_INVALID_ARG),
    (dict(window=0), _native.FA_ERR_INVALID_ARG),
    (dict(dtype=2), _native.FA_ERR_INVALID_ARG),
    (dict(D=96), _native.FA_ERR_UNSUPPORTED),
    (dict(Nq=301), _native.FA_ERR_UNSUPPORTED),
])
def test_refusals(lib, kw, code):
    assert fwd(lib, **kw) == code
    assert bwd(lib, ws_bytes=1 << 40, **kw) == code
    if "Nq" not in kw:
        assert paged(lib, **kw) == code


def test_more_refusals(lib):
    assert fwd(lib, q=None) == _native.FA_ERR_INVALID_ARG
    assert fwd(lib, cap=-1.0) == _native.FA_ERR_INVALID_ARG
    assert fwd(lib, cap=5000.0) == _native.FA_ERR_UNSUPPORTED
    assert fwd(lib, scale=0.0) == _native.FA_ERR_INVALID_ARG
    assert paged(lib, page=24) == _native.FA_ERR_UNSUPPORTED
    assert paged(lib, splits=2) == _native.FA_ERR_WORKSPACE
    assert paged(lib, splits=-1, ws=FAKE, ws_bytes=1 << 40) == _native.FA_ERR_INVALID_ARG


def test_workspace_sizes(lib):
    base = lib.fa_bwd_ex_workspace_size(1, 2, 1, 300, 300, 64, 1)
    assert lib.fa_bwd_sinks_workspace_size(1, 2, 1, 300, 300, 64, 100, 0) == base
    assert lib.fa_bwd_sinks_workspace_size(1, 2, 1, 300, 300, 64, 300, 4) == base  # hides nothing
    # one far unit of a tile past the first's window: 128 rows and 4 more, of 2 D fp32
    assert lib.fa_bwd_sinks_workspace_size(1, 2, 1, 300, 300, 64, 100, 4) == base + (128 + 4) * 2 * 64 * 4
    assert lib.fa_bwd_sinks_workspace_size(1, 2, 1, 300, 300, 64, 0, 4) == 0
    assert lib.fa_bwd_sinks_workspace_size(1, 2, 1, 300, 300, 64, 100, -4) == 0
    assert fa.bwd_workspace_size(1, 2, 300, 64, True, Hkv=1, window=100, sinks=4) == base + (128 + 4) * 2 * 64 * 4
    assert fa.bwd_workspace_size(1, 2, 300, 64, True, Hkv=1, window=1 << 40, sinks=4) == base
    # many sinks: bounded by 64 far units and two per key tile, not by keys times queries
    Nk = 32768
    most = lib.fa_bwd_ex_workspace_size(1, 2, 1, Nk, Nk, 128, 1) + (64 + 2 * 128) * 128 * 2 * 128 * 4
    assert lib.fa_bwd_sinks_workspace_size(1, 2, 1, Nk, Nk, 128, 64, 16384) <= most


def test_split_count_without_a_gpu(lib):
    assert lib.fa_fwd_paged_sinks_split_count(0, 2, 1, 1, 64, 16, 40, 100, 4) == 1
    assert lib.fa_fwd_paged_sinks_split_count(2, 2, 1, 1, 64, 16, 40, 0, 4) == 1
    assert lib.fa_fwd_paged_sinks_split_count(2, 2, 1, 1, 64, 16, 40, 100, -4) == 1


def test_python_refusals_come_before_the_device():
    x = torch.zeros((1, 2, 8, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fwd_scored(x, x, x, causal=True, window=4, sinks=2)
    from attention_sm_flashattention_gb300.scored import _check_sinks
    for bad in (dict(sinks=-1, window=4, causal=True, slopes=None), dict(sinks=2, window=0, causal=True, slopes=None),
                dict(sinks=2, window=4, causal=False, slopes=None), dict(sinks=2, window=4, causal=True, slopes=x),
                dict(sinks=2, window=4, causal=True, slopes=None, key_ranges=x)):
        with pytest.raises(ValueError, match="sinks"):
            _check_sinks(**bad)
