"""GPU parity of every kernel that expert_combine and expert_combine_bwd choose
between, by rows, columns and entries per token."""
import numpy as np
import pytest

import expert_refs as er
import layer_refs as lr
from gemv_gemm_f32_amd import binding as bd
from gpu_util import dev, host, torch
from test_experts import _combine_inputs

pytestmark = pytest.mark.gpu


# four spans of 256 columns per wave: from 4,096 runs of 1,024 columns on, with
# rows that end in each of the spans
@pytest.mark.parametrize("missing", [0.0, 0.3])
@pytest.mark.parametrize("weighted,residual", [(False, False), (True, True)])
@pytest.mark.parametrize("T,k,K", [(4096, 1, 129), (4100, 2, 300), (4097, 3, 767), (4097, 1, 1024), (2100, 3, 1029), (1400, 9, 2050)])
def test_combine_on_four_spans(T, k, K, weighted, residual, missing):
    Y, pos, w, R, _ = _combine_inputs(T, k, K, missing=missing)
    w, R = (w if weighted else None), (R if residual else None)
    out = bd.expert_combine(dev(Y), dev(pos), weights=None if w is None else dev(w),
                            residual=None if R is None else dev(R))
    lr.within(host(out), *er.combine(Y, pos, w, R))


def _check(dY, dw, Y, pos, w, dO):
    """dY is one product, exactly rounded; dw a sum of K products over at most
    K/64 additions in a lane and a tree."""
    t, j = np.nonzero(pos >= 0)
    p = pos[t, j]
    if dY is not None:
        assert np.array_equal(dY[p], dO[t] if w is None else w[t, j][:, None] * dO[t])
    if dw is not None:
        m = dO[t].astype(np.float64) * Y[p]
        assert np.all(np.abs(dw[t, j] - m.sum(1)) <= (Y.shape[1] / 64 + 20) * lr.U * np.abs(m).sum(1) + 1e-44)
        assert not dw[pos < 0].any()


# one wave per token (up to 256 columns, or up to 1,023 where tokens are many) and
# four, each with 1, 2, 4 and 8 entries at a time, the last run of them cut or whole
ONE_WAVE = [(9, 1, 200), (1030, 1, 513), (5, 2, 256), (1024, 2, 1023), (6, 3, 129), (1030, 4, 257), (7, 9, 255),
            (1030, 8, 513), (8, 5, 130), (1100, 16, 300)]
FOUR_WAVES = [(9, 1, 300), (1025, 1, 1024), (5, 2, 257), (300, 2, 1500), (6, 3, 1030), (1023, 4, 1023), (7, 9, 600),
              (40, 8, 1024), (3, 17, 2000)]


@pytest.mark.parametrize("missing", [0.0, 0.3])
@pytest.mark.parametrize("T,k,K", ONE_WAVE + FOUR_WAVES)
def test_combine_bwd_on_every_kernel(T, k, K, missing):
    Y, pos, w, _, dO = _combine_inputs(T, k, K, missing=missing)
    full = torch().full((T * k, K), 7.0, device="cuda")
    dY, dw = bd.expert_combine_bwd(dev(dO), dev(pos), Y=dev(Y), weights=dev(w), dY=full)
    _check(host(dY), host(dw), Y, pos, w, dO)
    unnamed = np.setdiff1d(np.arange(T * k), pos[pos >= 0])
    assert np.all(host(dY)[unnamed] == 7)
    only, none = bd.expert_combine_bwd(dev(dO), dev(pos), want=("dY",))
    assert none is None
    _check(host(only), None, Y, pos, None, dO)
    none, dw2 = bd.expert_combine_bwd(dev(dO), dev(pos), Y=dev(Y), weights=dev(w), want=("dw",))
    assert none is None and np.array_equal(host(dw2), host(dw))
