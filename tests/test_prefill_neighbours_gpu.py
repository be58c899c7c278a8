"""A tile of new tokens reads 128 rows, past its request's end into the rows of the next request or into
the padding behind the last one.  Whatever stands there - NaN, infinities, the largest values - the
request's results are those of the same rows alone, bit for bit, and nothing is reported."""
import numpy as np
import pytest
import torch

from paged_gqa_attention_head_gb300 import inputs

pytestmark = pytest.mark.gpu

KINDS = ["plain", "noncausal", "bf16", "fp8", "int8"]
JUNK = [float("nan"), float("inf"), float("-inf"), 3e38, 2.0 ** 22]


def _call(sa, p, kind, dev):
    c = p.prefix
    cu, sk = p.cu_seqlens.to(dev), None if p.sinks is None else p.sinks.to(dev)
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device=dev)

    def run(q, k, v):
        if kind == "plain":
            o = sa.prefill(q, k, v, cu, sk, p.scale, workspace_buf=ws)
        elif kind == "noncausal":
            o = sa.prefill_noncausal(q, k, v, cu, sk, p.scale, workspace_buf=ws)
        else:
            pages, at = (c.k_pages.to(dev), c.v_pages.to(dev)), (c.block_table.to(dev), c.lens.to(dev))
            if kind == "bf16":
                o = sa.prefill(q, k, v, cu, sk, p.scale, *pages, *at, workspace_buf=ws)
            elif kind == "fp8":
                o = sa.prefill_fp8(q, k, v, cu, sk, p.scale, *pages, c.k_scale.to(dev), c.v_scale.to(dev), *at, workspace_buf=ws)
            else:
                o = sa.prefill_int8(q, k, v, cu, *pages, c.kv_scales.to(dev), *at, sk, p.scale, workspace_buf=ws)
        return o, sa.get_status(ws)

    return run


def _make(kind, new, pre, D):
    if kind in ("plain", "noncausal"):
        return inputs.make_prefill(new, 8, 2, D, seed=D)
    return inputs.make_prefill(new, 8, 2, D, seed=D, prefix_lens=pre, prefix_kv_dtype=kind)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("last", [1, 31, 33, 70, 128])
def test_padding_behind_the_last_request(sa, cuda_dev, kind, D, last):
    p = _make(kind, [200, last], [40, 300], D)
    run = _call(sa, p, kind, cuda_dev)
    rows = [x.to(cuda_dev) for x in (p.q, p.k, p.v)]
    (out, lse), status = run(*rows)
    assert status == 0
    T, pad = p.q.shape[0], 140
    for i, junk in enumerate(JUNK):
        wide = [torch.cat([x, torch.full((pad, *x.shape[1:]), junk, dtype=x.dtype, device=cuda_dev)]) for x in rows]
        wide[2][T:, :, i::3] = 1.0
        (o, m), status = run(*wide)
        assert status == 0, junk
        assert torch.equal(o[:T], out) and torch.equal(m[:T], lse), junk


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
def test_values_of_another_request(sa, cuda_dev, kind, D):
    new = [70, 40, 130, 5]
    p = _make(kind, new, [40, 0, 300, 129], D)
    run = _call(sa, p, kind, cuda_dev)
    rows = [x.to(cuda_dev) for x in (p.q, p.k, p.v)]
    (out, lse), status = run(*rows)
    assert status == 0
    cu = np.concatenate([[0], np.cumsum(new)])
    for hit, junk in ((1, float("nan")), (2, float("inf")), (3, 3e38)):
        v = rows[2].clone()
        v[cu[hit]:cu[hit + 1], :, 3] = junk
        (o, m), status = run(rows[0], rows[1], v)
        assert status == sa.STATUS_VALUE_RANGE
        for i in range(len(new)):
            if i != hit:
                at = slice(int(cu[i]), int(cu[i + 1]))
                assert torch.equal(o[at], out[at]) and torch.equal(m[at], lse[at]), (hit, i)
