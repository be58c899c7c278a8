"""Host side of the INT8 cache's calls: which scratch and which status word a call gets (no GPU needed)."""
import ctypes
import threading
import weakref

import pytest
import torch


@pytest.fixture
def host_scratch(sa, monkeypatch):
    """The default scratch as host memory, outside any capture."""
    real = torch.zeros
    monkeypatch.setattr(sa.torch, "zeros", lambda *size, dtype=None, device=None: real(*size, dtype=dtype))
    monkeypatch.setattr(sa, "_capturing", lambda: False)
    monkeypatch.setattr(sa, "_current_device", lambda: 0)
    monkeypatch.setattr(sa, "_scratch", sa._Scratch())  # nothing of it stays for tests on a GPU
    return sa


def test_threads_on_one_stream_do_not_share_scratch(host_scratch):
    """A call is a split kernel and a merge: with one buffer, another thread's split kernel could
    overwrite the partial states between the two."""
    sa, got = host_scratch, {}

    def call(name):
        got[name] = [sa._stream_workspace(n, 0, 0, tag) for n, tag in ((1000, "decode"), (500, "decode"), (500, "prefill"))]

    call("main")
    threads = [threading.Thread(target=call, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for mine in got.values():
        assert mine[0] is mine[1]  # a thread keeps its own
        assert mine[2] is not mine[0]
    assert len({id(mine[0]) for mine in got.values()}) == 3
    assert host_scratch._stream_workspace(500, 0, 7, "decode") is not got["main"][0]  # another stream


def test_outgrown_scratch_is_let_go(host_scratch):
    """No captured call uses the eager scratch, so nothing needs the smaller buffer any more."""
    ws = host_scratch._stream_workspace(1000, 0, 9, "decode")
    old = weakref.ref(ws)
    del ws
    assert host_scratch._stream_workspace(1001, 0, 9, "decode").numel() == 2000
    assert old() is None


def test_report_entry_points_check_their_arguments(sa):
    """Before any CUDA work: missing or misaligned pointers, the status word's among them; empty calls."""
    lib = sa.load()
    desc = lambda n: ctypes.byref(sa.paged_desc(n, 8, 2, 64, 10, 4))  # noqa: E731
    buf = (ctypes.c_uint8 * 4096)()
    p = (ctypes.addressof(buf) + 255) // 256 * 256
    decode = lambda ptr, status, n=4: lib.sinkattn_decode_int8_report(  # noqa: E731
        p, ptr, p, p, p, p, None, 0.125, p, None, desc(n), p, 256, status, None)
    prefill = lambda ptr, status, n=4, tokens=8: lib.sinkattn_prefill_int8_report(  # noqa: E731
        p, p, p, p, tokens, ptr, p, p, p, p, None, 0.125, p, None, desc(n), p, 256, status, None)
    for call in (decode, prefill):
        assert call(None, None) == sa.ERR_INVALID_ARG
        assert call(p, p + 2) == sa.ERR_INVALID_ARG
        assert call(None, None, n=0) == sa.OK
    assert prefill(None, None, tokens=0) == sa.OK


def test_the_shared_status_word_during_a_capture(host_scratch, monkeypatch):
    """Before the word exists a captured call says that it will not report."""
    sa = host_scratch
    monkeypatch.setattr(sa, "_workspaces", {})
    monkeypatch.setattr(sa, "_capturing", lambda: True)
    with pytest.warns(RuntimeWarning, match="default_status"):
        assert sa._status_buffer(0) is None
    word = sa._workspaces[torch.device("cuda", 0), "append"] = torch.zeros(256, dtype=torch.uint8)
    assert sa._status_buffer(0) is word


def test_a_capture_on_another_device_than_the_current_one(host_scratch, monkeypatch):
    """It is the tensors' device whose stream is asked, not the current one's."""
    sa, current, calls = host_scratch, [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    real = torch.empty
    monkeypatch.setattr(sa.torch, "empty", lambda *size, dtype=None, device=None: real(*size, dtype=dtype))
    monkeypatch.setattr(sa.torch.cuda, "device", Device)
    monkeypatch.setattr(sa, "_current_device", lambda: current[0])
    monkeypatch.setattr(sa, "_capturing", lambda: current[0] == 1)
    monkeypatch.setattr(sa, "_call", lambda index, what, *args: calls.append((index, what)))
    eager = [sa._stream_workspace(1000, 0, 5, "prefill") for _ in range(2)]
    captured = [sa._stream_workspace(1000, 1, 5, "prefill") for _ in range(2)]
    assert eager[0] is eager[1] and captured[0] is not captured[1]
    assert calls == [(1, "sinkattn_workspace_init")] * 2 and current == [0]


def test_workspaces_that_are_not_the_calls_to_write(sa):
    """On another device, or with elements that do not lie one after the other."""
    with pytest.raises(ValueError, match="is on cpu"):
        sa._workspace_args(torch.zeros(256, dtype=torch.uint8), 0)
    with pytest.raises(TypeError):
        sa._workspace_args(4096, 0)
    here = torch.zeros(256, dtype=torch.int32).get_device()
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(512, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            sa._workspace_args(bad, here)
    ws = torch.zeros(256, dtype=torch.int32)
    assert sa._workspace_args(ws, here) == (ws.data_ptr(), 1024)


def test_the_status_word_is_zero_before_others_see_it(host_scratch, monkeypatch):
    """Made once, whichever thread comes first, and published after its memory is cleared."""
    sa, seen, made = host_scratch, [], []
    words = {}

    class Stream:
        def synchronize(self):
            seen.append(dict(words))

    fake = sa.torch.zeros
    monkeypatch.setattr(sa, "_workspaces", words)
    monkeypatch.setattr(sa.torch, "zeros", lambda *a, **k: made.append(1) or fake(*a, **k))
    monkeypatch.setattr(sa.torch.cuda, "current_stream", lambda index: Stream())
    got = []
    threads = [threading.Thread(target=lambda: got.append(sa._status_buffer(0))) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert seen == [{}] and len(made) == 1 and all(w is got[0] for w in got) and len(got) == 8
