"""Decode over a 4-bit cache whose V scales are below any that the append writes."""
import pytest
import torch

from oracle import plain
from paged_gqa_attention_head_gb300 import inputs
from test_int4_gpu import _dev, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G", [(64, 8), (64, 16), (128, 1), (128, 16)])
@pytest.mark.parametrize("word", [0x0010, 0x0040, 0x0080, 0x0D00])
@pytest.mark.parametrize("ordinary", [0, 20])
def test_v_scales_below_two_to_the_minus_100(sa, cuda_dev, D, G, word, ordinary):
    """Subnormal ones too (2^-129, 2^-127; 2^-126, 2^-101): they count as 0, alone and beside ordinary tokens."""
    lens = [5000, 40, 16]
    w = inputs.make_decode(lens, len(lens), 2 * G, 2, D, seed=41, poison=False)
    c = w.cache
    kv = inputs.pack_int4(c.k_pages, c.v_pages)
    words = kv.view(torch.int16)[:, :, 1, 8].view(c.num_pages, 2, D // 32, 16)
    keep = words.clone()
    words[:] = (words & 15) | word
    for b in range(len(lens)):  # the first tokens of each sequence stay as they were
        for j in range(ordinary if lens[b] > ordinary else 0):
            p = int(c.block_table[b, j // 16])
            words[p, :, :, j % 16] = keep[p, :, :, j % 16]
    a = list(_dev(w, cuda_dev))
    a[1] = kv.to(cuda_dev)
    ref = plain.attend_int4(w.q, kv, c.block_table, c.lens, w.sinks, w.scale)
    out, lse = sa.decode_int4(*a)
    # 15 scales below 2^-100 are off by 2^-96 at most where they are all that there is
    check(out, lse, (ref[0], ref[1], ref[2] + 2.0 ** -96 * 2.0 ** 11))
    assert sa.default_status() == 0
