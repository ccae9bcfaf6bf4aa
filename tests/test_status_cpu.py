"""Which status word a call writes and which words get_error reads, with the
library and the device stubbed (no GPU)."""
import pytest
import torch


class FakeLib:
    """Records the words that are polled; `set` holds those that report a timeout."""

    def __init__(self):
        self.polled, self.set = [], set()

    def qlora_get_error(self, ptr, stream):
        self.polled.append(ptr.value)
        if ptr.value in self.set:
            self.set.discard(ptr.value)
            return 7
        return 0

    def qlora_noalloc_get_error(self, stream):
        self.polled.append("fixed")
        if "fixed" in self.set:
            self.set.discard("fixed")
            return 7
        return 0

    def qlora_status_string(self, code):
        return b"timeout"


@pytest.fixture()
def q(monkeypatch):
    import bit_nf4_quantized_20_b200 as q
    fake, zeros = FakeLib(), torch.zeros
    monkeypatch.setattr(q, "lib", lambda: fake)
    monkeypatch.setattr(q._lib, "lib", lambda: fake)
    monkeypatch.setattr(q, "_WS", {})
    monkeypatch.setattr(q, "_STATUS", {})
    monkeypatch.setattr(q, "_FIXED", set(), raising=False)
    monkeypatch.setattr(q, "_stream", lambda dev: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k))
    q.fake = fake
    yield q
    del q.fake


@pytest.mark.parametrize("made", ["cuda", "cuda:1", torch.device("cuda"), 1])
@pytest.mark.parametrize("asked", ["cuda", "cuda:1", torch.device("cuda"), None, 1])
def test_a_recorded_failure_is_found_however_the_device_is_named(q, made, asked):
    """Every name of the current device means the same workspace."""
    dev = torch.device("cuda", made) if isinstance(made, int) else made
    ws = q.workspace(dev, 4096)
    assert q.workspace(torch.device("cuda", 1), 4096) is ws
    q.fake.set.add(ws.data_ptr())
    with pytest.raises(q.QLoraError) as e:
        q.get_error(asked)
    assert e.value.status == 7
    q.get_error(asked)
    assert q.fake.polled == [ws.data_ptr()] * 2


def test_another_device_has_a_word_of_its_own(q):
    ws = q.workspace("cuda:0", 4096)
    q.fake.set.add(ws.data_ptr())
    q.get_error("cuda")            # device 1: nothing recorded there
    with pytest.raises(q.QLoraError):
        q.get_error("cuda:0")


def test_a_first_use_inside_a_capture_is_reported(q, monkeypatch):
    """No word can be made while a graph is captured.  The call then records in
    the library's fixed array (a null word), and get_error reads that as well."""
    from contextlib import nullcontext
    dev = torch.device("cuda", 1)
    monkeypatch.setattr(torch.cuda, "device", lambda d: nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    assert q._status(dev) is None
    q.fake.set.add("fixed")
    q.get_error("cuda:0")                  # another device: not its array
    assert q.fake.polled == []
    with pytest.raises(q.QLoraError) as e:
        q.get_error()
    assert e.value.status == 7
    q.get_error()
    # a word made later does not hide what the graph's replays record
    word = torch.zeros(256, dtype=torch.uint8)
    q._STATUS[dev] = word
    assert q._status(dev) == word.data_ptr()
    q.fake.set.add("fixed")
    with pytest.raises(q.QLoraError):
        q.get_error()
