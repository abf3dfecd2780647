"""Host threads that call one operator at two sizes at once: a kernel's limit of
shared memory belongs to the kernel, so no call may leave it below what another's
launch takes."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROUNDS = 3000


class Recorder:
    """The library, keeping the calls made of it."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        f = getattr(self.lib, name)

        def call(*args):
            if f.restype is ctypes.c_int32:
                self.calls.append((f, args))
            return f(*args)

        return call


def check(rp, monkeypatch, calls):
    """The library's calls behind each of `calls`, over and over from a thread of its own
    with as little Python between them as there can be; every one of them goes through
    and the results stay what they were."""
    lib, scratch, recorded, results = Recorder(rp.load()), [], [], []
    take = rp._workspace
    with monkeypatch.context() as m:
        m.setattr(rp, "load", lambda: lib)
        m.setattr(rp, "_workspace", lambda *a: scratch.append(take(*a)) or scratch[-1])
        for c in calls:
            lib.calls = []
            results.append(c())
            recorded.append(lib.calls)
    torch.cuda.synchronize()
    want = [[t.clone() for t in r if t is not None] for r in results]
    assert all(r for r in recorded)
    refused, start = [], threading.Barrier(len(calls))

    def run(i):
        torch.cuda.set_device(0)
        start.wait()
        for _ in range(ROUNDS):
            for f, args in recorded[i]:
                rc = f(*args)
                if rc:
                    refused.append((i, f.__name__, rc))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, (len(refused), refused[:5])
    for w, r in zip(want, results):
        assert all(torch.equal(a, b) for a, b in zip(w, [t for t in r if t is not None]))


def randn(*shape, seed=1):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def test_log_probabilities_of_long_rows(rp, monkeypatch):
    """Above 6.6 million columns a row's sums pass 48 KB: 50 and 111 KB here."""
    a, b = randn(1, 7_200_000).bfloat16(), randn(1, 16_000_000).bfloat16()
    check(rp, monkeypatch, [lambda: rp.token_logprobs(a, top=2), lambda: rp.token_logprobs(b, top=2)])


def test_heads_of_two_widths(rp, monkeypatch):
    """The backward of heads of 160 takes 50 KB a CTA, of 512 132 KB."""
    calls = []
    for dim in (160, 512):
        x, dy, gain = randn(64, 3 * dim), randn(64, 3 * dim, seed=2), randn(dim, seed=3)
        calls.append(lambda x=x, dy=dy, g=gain: rp.head_norm_rope_backward(dy, x, 2, 1, q_gain=g, k_gain=g))
    check(rp, monkeypatch, calls)
