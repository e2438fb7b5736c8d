"""Windows with sinks: what keys that no query sees hold does not change a bit of any result."""

import pytest
import torch

import attention_sm_flashattention_gb300 as fa
from attention_sm_flashattention_gb300.inputs import make_inputs, make_paged_inputs

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("Nq,window,sinks", [(40, 150, 5), (200, 60, 130), (1, 1, 1)])
def test_dense(Nq, window, sinks, cap, D):
    q, k, v, do = (t.cuda() for t in make_inputs(2, 4, Nq, D, 51, Hkv=2, Nk=900))
    how = dict(causal=True, softcap=cap, window=window, sinks=sinks)

    def run(k, v):
        o, lse = fa.fwd_scored(q, k, v, **how)
        return (o, lse) + tuple(fa.bwd_scored(q, k, v, o, do, lse, **how))
    clean = run(k, v)
    unseen = slice(sinks, 900 - Nq - window + 1)
    for a, b in ((NAN, INF), (INF, NAN), (NAN, NAN)):
        ks, vs = k.clone(), v.clone()
        ks[:, :, unseen], vs[:, :, unseen] = a, b
        for name, x, y in zip(("o", "lse", "dq", "dk", "dv"), clean, run(ks, vs)):
            assert torch.equal(x, y), (name, a, b)
    assert all((g[:, :, unseen] == 0).all() for g in clean[3:]) and fa.device_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("Nq", [1, 90])
@pytest.mark.parametrize("splits", [1, 4])
def test_paged(splits, Nq, cap, D):
    page, lens, window, sinks = 16, [700, 411], 60, 21
    q, kc, vc, table, ctx = make_paged_inputs(2, 4, 2, Nq, lens, D, page, 52)

    def run(kc, vc):
        return fa.fwd_paged_scored(*(t.cuda() for t in (q, kc, vc, table, ctx)), softcap=cap, window=window, sinks=sinks,
                                   splits=splits)
    clean = run(kc, vc)
    for b, n in enumerate(lens):
        for p in list(range(sinks, n - Nq + 1 - window)) + list(range(n, -(-n // page) * page)):
            kc[table[b, p // page], p % page], vc[table[b, p // page], p % page] = NAN, INF
    assert all(torch.equal(x, y) for x, y in zip(clean, run(kc, vc)))
