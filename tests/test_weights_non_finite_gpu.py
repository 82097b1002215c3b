"""pa_decode_weights on logits that are not finite: NaN, or +infinity, makes a head's softmax NaN, and so the head's
output and the totals of its kv head at every position; a logit of -infinity is a weight of zero.  Other heads and
sequences keep their bits.
"""

import numpy as np
import pytest
import torch

import oracle
from test_cache_drop_gpu import batch, f64, ready

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from paged_kv_cache_382_b200 import build

    build.build()
    from paged_kv_cache_382_b200 import pa as binding

    return binding


HQ, HKV, D, B, P = 6, 2, 64, 16, 64
CTX = [50, 200, 64 * 40 + 9, 33]      # one partition, a few (merged with the totals), many, one


def place(kc, tables, s, h, positions, value, column=None):
    for p in positions:
        row = kc[int(tables[s, p // B]), h, p % B]
        row[slice(None) if column is None else column] = value


# what is put where: (sequence, positions) of K of kv head 1, or a query head's q
KINDS = {
    "nan key": lambda kc, q, t: [place(kc, t, s, 1, [p], float("nan"), 3) for s, p in ((0, 7), (1, 130), (2, 1999))],
    "a partition of nan keys": lambda kc, q, t: [place(kc, t, s, 1, r, float("nan")) for s, r in ((0, range(50)), (1, range(64, 128)),
                                                                                                  (2, range(64, 128)))],
    "nothing but nan": lambda kc, q, t: [place(kc, t, s, 1, range(CTX[s]), float("nan")) for s in (0, 1, 2)],
    "nan query": lambda kc, q, t: q[:3, 4].fill_(float("nan")),
    "infinite key": lambda kc, q, t: [place(kc, t, s, 1, [p], float("inf"), 3) for s, p in ((0, 0), (1, 199), (2, 2000))],
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", KINDS)
def test_totals_and_output_of_non_finite_logits(pa, kind, dtype):
    step = batch(CTX, HQ, HKV, D, B, dtype, P=P)
    kc, vc, tables, lens = ready(pa, step)
    q = step.q.clone()
    stride = tables.shape[1] * B

    def run(q, kc):
        w_in = torch.linspace(0, 1, stride, device="cuda").expand(len(CTX), HKV, stride).contiguous()
        w, out = torch.zeros_like(w_in), torch.empty(len(CTX), HQ, D, dtype=torch.float32, device="cuda")
        pa.decode_weights(out, w, q, kc, vc, tables, lens, step.scale, weights_in=w_in, partition_size=P)
        torch.cuda.synchronize()
        return w, out, w_in

    clean_w, clean_out, w_in = run(q, kc)
    KINDS[kind](kc, q, tables)
    w, out, _ = run(q, kc)
    k64, v64, q64 = f64(kc), f64(vc), f64(q)
    bad = 0
    for s, c in enumerate(CTX):
        for h in range(HKV):
            keys = oracle.gather_kv(k64, step.block_tables[s], c, h)
            values = oracle.gather_kv(v64, step.block_tables[s], c, h)
            exact = np.zeros(c)
            for n in range(h * 3, h * 3 + 3):
                with np.errstate(invalid="ignore"):
                    x = float(np.float32(step.scale)) * (keys @ q64[s, n])
                    e = np.exp(x - (x.max() if not np.isnan(x).all() else 0.0))
                    p = e / e.sum()
                exact += p
                if np.isnan(p).any():
                    bad += 1
                    assert np.isnan(p).all() and torch.isnan(out[s, n]).all(), (s, n)
                elif np.isneginf(x).any():
                    assert np.abs(f64(out[s, n]) - p @ values).max() <= (1e-5 if dtype == torch.float32 else 2e-3)
                else:
                    assert torch.equal(out[s, n], clean_out[s, n]), (s, n)
            got, before = f64(w[s, h, :c]), f64(w_in[s, h, :c])
            if np.isnan(exact).any():
                assert np.isnan(got).all(), (s, h)
            else:
                assert np.all(np.abs(got - before - exact) <= 6e-4 * exact + 2.0 ** -22 * (before + exact)), (s, h)
                if h == 0 or s == 3:
                    assert torch.equal(w[s, h], clean_w[s, h])
    assert bad >= 3
