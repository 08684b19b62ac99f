"""The sections of rotary positions with several axes, as several threads give them (no GPU).

A call passes the address of a host array that the library reads, so the array has to outlive the call whatever other threads do.
"""
import threading

import torch

from compressed_linear_amd import serving


def test_threads_get_an_array_that_stays(monkeypatch):
    """Two first calls with the same sections, neither of which has seen the other's: both get the array that is kept."""
    both = threading.Barrier(2)

    class Sections(dict):
        def get(self, key):
            found = super().get(key)
            both.wait(20)
            return found

    sections = Sections()
    monkeypatch.setattr(serving, "_i32", torch.int32)
    monkeypatch.setattr(serving, "_sections", sections)
    positions = torch.zeros(3, 2, dtype=torch.int32)
    got = []

    def call():
        got.append(serving._axes(positions, 2, (4, 3, 1), positions.device))

    threads = [threading.Thread(target=call) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    (pairs, kept), = sections.values()
    assert list(pairs) == [4, 3, 1] and kept == pairs.buffer_info()[0]
    assert [axes for _, axes, _ in got] == [3, 3]
    assert [address for _, _, address in got] == [kept, kept]
