"""Decode over an INT8 cache whose values lie near the ends of what its scales may be, 2^-100 to 2^100: the
partial states of split sequences hold sums of up to 2^17 such values, each with its probability."""
import pytest
import torch

from paged_gqa_attention_head_gb300 import inputs
from test_decode_int8_gpu import _dev, _ref, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 8), (128, 1, 16)])
@pytest.mark.parametrize("e", [-100, 60, 100])
@pytest.mark.parametrize("sms", [0, 1])
def test_sums_of_large_and_small_values(sa, cuda_dev, D, Hkv, G, e, sms):
    """All values of one sign and near the largest; the first page's scores 7 (log2) below the others',
    within the slack of the running maximum, so that every later probability is at its largest."""
    w = inputs.make_decode([30000, 130, 3], 3, Hkv * G, Hkv, D, seed=D, kv_dtype="int8")
    c = w.cache
    c.kv_scales[:, :, 1] = 2.0 ** e
    c.v_pages[:] = 127
    c.v_pages[:, :, :, ::2] = 120
    w.q[:] = 1.0
    c.k_pages[:] = 100
    c.kv_scales[:, :, 0] = 7.0 / (1.4426950408889634 * w.scale * 100 * D)
    c.k_pages[c.block_table[0, 0].long()] = 0
    out, lse = sa.decode_int8(*_dev(w, cuda_dev), max_sms=sms)
    check(out, lse, _ref(w))
