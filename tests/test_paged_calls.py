"""The paged calls on the CPU: what their wrappers hand to the library, with the library and the device
replaced by recorders, and refusals before any CUDA call."""
import contextlib
import ctypes

import pytest
import torch

from sparse_attention_kv_echo_gb300 import _lib as L


class _Recorder:
    """Stands in for the loaded library: keeps every call's arguments and succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("_size") else L.ECHO_OK
        return call


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def host(monkeypatch):
    """CPU tensors pass for the current device's (get_device() of both is -1); the current stream and every
    torch.empty made under it are recorded."""
    rec = _Recorder()
    rec.current, rec.taken = _Stream(1), []

    @contextlib.contextmanager
    def use(s):
        before = rec.current
        rec.current = before if s is None else s
        try:
            yield
        finally:
            rec.current = before

    empty = torch.empty

    def recorded(*a, **kw):
        t = empty(*a, **kw)
        rec.taken.append((t.data_ptr(), rec.current.cuda_stream))
        return t
    monkeypatch.setattr(L, "load", lambda *a, **kw: rec)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: rec.current)
    monkeypatch.setattr(L, "_raw_stream", None)
    monkeypatch.setattr(torch, "empty", recorded)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda *a: None)
    return rec


def _weigh(**kw):
    off = torch.tensor([0, 10])
    pages = L.KVPages(torch.zeros(1, dtype=torch.int32), torch.zeros((16, 576), dtype=torch.bfloat16), 16)
    mass = torch.zeros(10)
    L.mla_mass(off, torch.zeros((10, 2, 576), dtype=torch.bfloat16), torch.zeros((10, 2)), off, 10, pages, 0.1, mass, mass,
               torch.zeros(1, dtype=torch.int32), **kw)


@pytest.mark.parametrize("stream", [None, 7])
def test_a_workspace_taken_for_a_call_belongs_to_its_stream(host, stream):
    # a block of another stream's pool may still be in use there when it is handed out
    _weigh(stream=None if stream is None else _Stream(stream))
    (name, args), = [c for c in host.calls if c[0] == "echo_mla_mass"]
    ws, used_on = args[-4], args[-1]
    assert used_on == (1 if stream is None else stream)
    assert (ws, used_on) in host.taken


def test_a_stream_handle_needs_a_workspace(host):
    with pytest.raises(ValueError):
        _weigh(stream=7)
    _weigh(stream=7, ws=torch.zeros(4096, dtype=torch.uint8))


def test_victims_of_residents_check_their_arguments():
    from sparse_attention_kv_echo_gb300 import build
    build.build()
    lib, d = L.load(), ctypes.c_void_p(0x1000)

    def evict(B=1, off=d, n=10, s2t=d, fb=d, C=64, m=d, keep=1, sinks=0, recent=0, et=d, es=d, ec=d, st=d):
        return lib.echo_evict_select_resident(B, off, None, n, s2t, fb, C, m, keep, sinks, recent, et, es, ec, st, None)
    for bad in (dict(B=0), dict(off=None), dict(n=-1), dict(s2t=None), dict(C=0), dict(m=None), dict(keep=-1),
                dict(sinks=-1), dict(recent=-1), dict(et=None), dict(es=None), dict(ec=None), dict(st=None)):
        assert evict(**bad) == L.ECHO_EINVAL, bad
    assert evict(B=L.MAX_REQUESTS + 1) == L.ECHO_EUNSUPPORTED and evict(C=(1 << 19) + 32) == L.ECHO_EUNSUPPORTED
    assert evict(C=48) == L.ECHO_ECAPACITY


@pytest.mark.parametrize("words", [1, 3])
def test_victims_refuse_free_bits_of_another_size(host, words):
    i = torch.zeros((1, 64), dtype=torch.int32)
    with pytest.raises(ValueError):
        L.evict_select(torch.tensor([0, 10]), 10, i, torch.zeros(10), 1, i, i, i[0, :1], i[0, :1],
                       freebits=torch.zeros(words, dtype=torch.int32))


@pytest.mark.parametrize("page,req_rows", [(0, 0), (-1, 0), (2 ** 31, 0), (2 ** 32 + 16, 0), (16, -1), (16, 2 ** 64 + 1)])
def test_pages_refuse_sizes_the_struct_does_not_hold(host, page, req_rows):
    tab, kv = torch.zeros(1, dtype=torch.int32), torch.zeros((16, 576), dtype=torch.bfloat16)
    L.KVPages(tab, kv, 2 ** 31 - 1, 0)
    with pytest.raises(ValueError):
        L.KVPages(tab, kv, page, req_rows)


def test_victims_of_no_requests_are_refused_by_the_library(host):
    i = torch.zeros((0, 64), dtype=torch.int32)
    with pytest.raises(ValueError):      # (no ZeroDivisionError: the tables fit no request)
        L.evict_select(torch.tensor([0]), 10, torch.zeros(64, dtype=torch.int32), torch.zeros(10), 1, i, i, i[:, 0], i[:, 0])
