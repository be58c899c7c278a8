"""Status bits of the INT8 attention calls that are given no workspace: default_status has them, of eager
calls and of captured ones."""
import pytest
import torch

from paged_gqa_attention_head_gb300 import inputs

pytestmark = pytest.mark.gpu


def _decode(dev):
    w = inputs.make_decode([3000, 100], 2, 16, 2, 64, seed=1, kv_dtype="int8")
    c = w.cache
    return [x.to(dev) for x in (w.q, c.k_pages, c.v_pages, c.kv_scales, c.block_table, c.lens)], 4


def _prefill(new, pre):
    def make(dev):
        p = inputs.make_prefill(new, 8, 1, 64, seed=2, prefix_lens=pre, prefix_kv_dtype="int8")
        c = p.prefix
        return [x.to(dev) for x in (p.q, p.k, p.v, p.cu_seqlens, c.k_pages, c.v_pages, c.kv_scales, c.block_table, c.lens)], 7
    return make


@pytest.mark.parametrize("name,make", [("decode_int8", _decode), ("prefill_int8", _prefill([17], [4000])),
                                       ("prefill_int8", _prefill([300, 2000, 1500, 900], [0, 70, 33, 500]))])
def test_bad_pages_of_default_calls(sa, cuda_dev, name, make):
    """In parts and whole; the table's entry goes bad and good again between replays."""
    f = getattr(sa, name)
    args, at = make(cuda_dev)
    table = args[at]
    good = table.clone()
    sa.default_status(cuda_dev)
    alone = f(*args)
    assert sa.default_status() == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = f(*args)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()

    def eager():
        f(*args)

    def on_another_stream():
        with torch.cuda.stream(other):
            f(*args)

    for run in (eager, on_another_stream, g.replay):
        table[1 if table.shape[0] > 1 else 0, 1] = -5
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert sa.default_status(cuda_dev) == sa.STATUS_BAD_PAGE
        table.copy_(good)
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert sa.default_status(cuda_dev) == 0
    assert torch.equal(out, alone[0]) and torch.equal(lse, alone[1])


def test_a_given_workspace_keeps_its_own_bits(sa, cuda_dev):
    args, at = _decode(cuda_dev)
    args[at][1, 1] = -5
    sa.default_status()
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=cuda_dev)
    sa.decode_int8(*args, workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_PAGE
    assert sa.default_status() == 0


def test_a_workspace_elsewhere_is_refused(sa, cuda_dev):
    """By every call of the INT8 cache and by the preparation, before anything is launched."""
    host = torch.zeros(1 << 24, dtype=torch.uint8)
    decode, _ = _decode(cuda_dev)
    prefill, _ = _prefill([17], [40])(cuda_dev)
    q, k, v, cu, kp, vp, sc, bt, lens = prefill
    with pytest.raises(ValueError, match="workspace_buf is on cpu"):
        sa.decode_int8(*decode, workspace_buf=host)
    with pytest.raises(ValueError, match="workspace_buf is on cpu"):
        sa.prefill_int8(*prefill, workspace_buf=host)
    with pytest.raises(ValueError, match="workspace_buf is on cpu"):
        sa.append_kv_int8(k, v, cu, bt, lens, kp, vp, sc, workspace_buf=host)
    with pytest.raises(ValueError, match="workspace_buf is on cpu"):
        sa.qk_norm_rope(q, k, workspace_buf=host)
