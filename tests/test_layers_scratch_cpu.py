"""The network operators' scratch memory without a GPU: a stand-in takes the place of the library's
calls, host memory that of the GPU's."""
from __future__ import annotations

import threading
import time

import pytest
import torch

from learned_image_compression_amd import layers as L

REFUSED = L._E_WORKSPACE
HOST = torch.device("cpu")


@pytest.fixture(autouse=True)
def empty(monkeypatch):
    monkeypatch.setattr(L, "_workspaces", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)


class Call:
    """A call of several launches: who is inside with which memory, and whether two ever were."""

    def __init__(self):
        self.guard, self.inside, self.mixed, self.done = threading.Lock(), {}, [], 0

    def __call__(self, need):
        def call(address, nbytes):
            if nbytes < need:
                return REFUSED
            with self.guard:
                self.mixed += [address] if address in self.inside.values() else []
                self.inside[threading.get_ident()] = address
            time.sleep(0.002)  # the interpreter's lock is free here, as within a foreign call
            with self.guard:
                del self.inside[threading.get_ident()]
                self.done += 1
            return 0
        return call


def in_threads(jobs):
    failed = []

    def work(job):
        try:
            job()
        except BaseException as e:  # noqa: BLE001 - reported by the test
            failed.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not failed and not any(t.is_alive() for t in threads)


def test_threads_of_one_stream_take_turns():
    call = Call()

    def job(i):
        for turn in range(20):
            need = (1 << 20) + 4096 * (turn if i else 0)  # some of them grow the memory
            L._with_workspace(HOST, 0, call(need), lambda: need, "stand-in")

    in_threads([lambda i=i: job(i) for i in range(4)])
    assert call.done == 80 and call.mixed == []


def test_streams_have_memory_of_their_own():
    seen = {}

    def job(stream):
        def call(address, nbytes):
            if nbytes == 0:
                return REFUSED
            seen.setdefault(stream, set()).add(address)
            return 0

        for _ in range(5):
            L._with_workspace(HOST, stream, call, lambda: 10, "stand-in")

    in_threads([lambda s=s: job(s) for s in range(4)])
    assert all(len(v) == 1 for v in seen.values()) and len(set.union(*seen.values())) == 4


def test_a_call_from_within_a_call_does_not_wait_for_itself():
    def inner(address, nbytes):
        return 0 if nbytes else REFUSED

    def size():  # as a finalizer that the allocation runs
        L._with_workspace(HOST, 0, inner, lambda: 1 << 21, "inner")
        return 64

    done = []
    in_threads([lambda: done.append(L._with_workspace(HOST, 0, inner, size, "outer"))])
    assert done == [None]


def test_a_refused_call_leaves_the_lock():
    with pytest.raises(RuntimeError):
        L._with_workspace(HOST, 0, lambda a, n: -1, lambda: 10, "stand-in")
    in_threads([lambda: L._with_workspace(HOST, 0, lambda a, n: 0, lambda: 10, "stand-in")])


def test_scratch_memory_can_be_given_back():
    import weakref

    def call(address, nbytes):
        return 0 if nbytes else REFUSED

    for stream in (0, 1):
        L._with_workspace(HOST, stream, call, lambda: 1 << 22, "stand-in")
    kept = [weakref.ref(w.held[2]) for w in L._workspaces.values()]
    assert len(kept) == 2 and all(k() is not None for k in kept)
    L.release_workspaces()
    assert all(k() is None for k in kept)
    L._with_workspace(HOST, 0, call, lambda: 1 << 22, "stand-in")  # and taken again
    assert L._workspaces[(None, 0)].held[1] == 1 << 22
