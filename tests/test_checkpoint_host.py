"""The checkpoint store without a GPU: its launches are made with the table block's device current, and bytes of another
device are refused before anything is launched (the coder is replaced by one that records)."""
import pytest

torch = pytest.importorskip("torch")
from lossless_entropy_coding_fixed_b200 import hx  # noqa: E402
from lossless_entropy_coding_fixed_b200.checkpoint import CheckpointStore  # noqa: E402


@pytest.fixture
def calls(monkeypatch):
    seen, current = [], [None]

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, current[0] = current[0], self.device

        def __exit__(self, *exc):
            current[0] = self.before

    def encode(tables, x, scratch=None, hist=None, kind=0):
        seen.append(("encode", current[0]))
        return x.clone(), torch.zeros(1, dtype=torch.int32)

    def decode(tables, stream, n, out=None, status=None, kind=0):
        seen.append(("decode", current[0]))
        out.copy_(stream)
        return out, status

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(hx, "encode", encode)
    monkeypatch.setattr(hx, "decode", decode)
    return seen


def test_launches_on_the_tables_device(calls):
    tables = torch.zeros(hx.TABLES_BYTES, dtype=torch.uint8)
    store = CheckpointStore(tables)
    data, scale = torch.arange(12, dtype=torch.uint8).view(3, 4), torch.ones(3)
    got, s = store.take(store.put(data, scale))
    assert torch.equal(got, data) and s is scale
    assert calls == [("encode", tables.device), ("decode", tables.device)]


def test_bytes_of_another_device_are_refused(calls):
    store = CheckpointStore(torch.zeros(hx.TABLES_BYTES, dtype=torch.uint8))
    with pytest.raises(ValueError):
        store.put(torch.zeros(3, 4, dtype=torch.uint8, device="meta"), torch.ones(3))
    assert not calls and len(store) == 0
