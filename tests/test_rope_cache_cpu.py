"""The kept RoPE tables without a GPU: a table is found by other calls only once it is written, and never
when its kernel has only been captured.  A stand-in for torch's CUDA calls records what happens."""
import contextlib
import threading
import types

import pytest


class FakeStream:
    cuda_stream = 0

    def __init__(self, torch):
        self.torch = torch

    def synchronize(self):
        self.torch.waits += 1
        if self.torch.on_wait:
            self.torch.on_wait()
        for t in self.torch.tables:
            t.written = True


@pytest.fixture
def fake(monkeypatch):
    """api.py on a stand-in: tables are objects that count as written after a synchronisation."""
    from static_offset_sparse_gb300 import api

    t = types.SimpleNamespace(tables=[], waits=0, capturing=False, on_wait=None, float32=None, api=api)

    class Table:
        def __init__(self, shape):
            self.shape, self.written = shape, False

        def data_ptr(self):
            return 4096

        def __getitem__(self, rows):
            part = Table((rows.stop,) + tuple(self.shape[1:]))
            part.whole = self
            return part

    def empty(shape, dtype=None, device=None):
        t.tables.append(Table(shape))
        return t.tables[-1]

    t.empty = empty
    t.device = lambda kind, index=0: types.SimpleNamespace(index=index)
    t.cuda = types.SimpleNamespace(device=lambda d: contextlib.nullcontext(), current_device=lambda: 0, current_stream=lambda *a: FakeStream(t),
                                   is_current_stream_capturing=lambda: t.capturing)
    monkeypatch.setattr(api, "_torch", lambda: t)
    monkeypatch.setattr(api, "_lib", lambda: types.SimpleNamespace(sfa_rope_table=lambda *a: 0))
    monkeypatch.setattr(api, "_ROPE_CACHE", {})
    if hasattr(api, "_ROPE_WHOLE"):
        monkeypatch.setattr(api, "_ROPE_WHOLE", {})
    return t


def _written(table):
    return getattr(table, "whole", table).written


def test_a_table_is_kept_when_it_is_written(fake):
    seen = []
    fake.on_wait = lambda: seen.append(dict(fake.api._ROPE_CACHE))
    tab = fake.api.rope_table(100, 1e4)
    assert seen == [{}] and _written(tab)
    assert all(_written(x) for x in fake.api._ROPE_CACHE.values())
    assert fake.api.rope_table(100, 1e4) is tab and fake.waits == 1


def test_a_captured_table_is_not_kept(fake):
    fake.capturing = True
    tab = fake.api.rope_table(100, 1e4)
    assert tab.shape == (100, 32, 2) and not fake.api._ROPE_CACHE and fake.waits == 0
    fake.capturing = False
    tab = fake.api.rope_table(100, 1e4)
    assert _written(tab)
    fake.capturing = True  # one that is there serves captures too
    assert fake.api.rope_table(100, 1e4) is tab


def test_a_second_thread_waits_for_the_table(fake):
    """A thread that asks while another waits for the table gets it when it is written, and makes none itself."""
    got, inside = [], threading.Event()

    def ask():
        inside.set()
        got.append(_written(fake.api.rope_table(100, 1e4)))

    other = threading.Thread(target=ask)

    def on_wait():
        fake.on_wait = None
        other.start()
        inside.wait()
        other.join(0.2)  # the synchronisation takes a while; the thread must not come back meanwhile
        assert not got

    fake.on_wait = on_wait
    assert _written(fake.api.rope_table(100, 1e4))
    other.join()
    assert got == [True] and len(fake.tables) == 1


def test_widths_share_a_table(fake):
    """A table for every width of a block table that grows by pages is a few tables, not one a width."""
    for pages in range(1, 1001):
        tab = fake.api.rope_table(64 * pages, 1e4)
        assert tab.shape == (64 * pages, 32, 2) and _written(tab)
    sizes = [t.shape[0] for t in fake.tables]
    assert len(sizes) <= 11 and sum(sizes) < 4 * 64000 and fake.waits == len(sizes)
    assert fake.api.rope_table(64, 1e4) is fake.api.rope_table(64, 1e4)
    fake.api.rope_table(64, 500.0)  # another theta has its own
    assert fake.waits == len(sizes) + 1
    fake.capturing = True  # a new width that a kept table covers, inside a capture
    before = len(fake.tables)
    assert fake.api.rope_table(63000, 1e4).shape == (63000, 32, 2) and len(fake.tables) == before
    fake.api.rope_table(1 << 17, 1e4)  # one that none covers
    assert fake.tables[-1].shape == (1 << 17, 32, 2) and fake.waits == len(sizes) + 1
