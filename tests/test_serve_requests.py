"""The serving example's check of requests, before anything reaches a GPU: token ids index the model's tensors."""

import types

import pytest

pytest.importorskip("torch")


@pytest.fixture()
def server():
    from paged_expert_moe_gb300.serve import Server
    s = object.__new__(Server)  # no model, no cache
    s.shape, s.seats, s.rows, s.longest, s.max_biases = types.SimpleNamespace(vocab=500), 2, 16, 40, 3
    s.seated, s.read, s.ended = [None, None], [0, 0], []
    return s


def request(**change):
    from paged_expert_moe_gb300.serve import Request
    return Request(**{"prompt": [0, 499, 7], "tokens": 5, **change})


BAD = [(dict(prompt=[3, 500]), "prompt: token 500"), (dict(prompt=[-1]), "prompt: token -1"), (dict(prompt=[1 << 40]), "prompt"),
       (dict(prompt=[]), "prompt"), (dict(tokens=0), "token"), (dict(prompt=[1] * 36), "36 \\+ 5 tokens"),
       (dict(biases={500: 1.0}), "biases: token 500"), (dict(biases={-1: 1.0}), "biases: token -1"),
       (dict(biases={1: 0.5, 2: 0.5, 3: 0.5, 4: 0.5}), "4 biases"), (dict(allowed=[1, 512]), "allowed: token 512"),
       (dict(allowed=[-2]), "allowed: token -2"), (dict(allowed=[]), "allowed"), (dict(output=[4]), "output")]


@pytest.mark.parametrize("change,what", BAD)
def test_requests_are_refused_before_they_are_seated(server, change, what):
    bad = request(**change)
    waiting = [request(), bad]
    with pytest.raises(AssertionError, match=what):
        server.run(list(waiting))
    assert server.seated == [None, None]
    with pytest.raises(AssertionError, match=what):  # steps by hand
        server.plan(waiting)
    assert waiting == [bad] and server.seated[1] is None


def test_good_requests_are_seated(server):
    waiting = [request(), request(prompt=[1] * 30, biases={0: 1.0, 499: -1.0}, allowed=[0, 499]), request()]
    work = server.plan(waiting)
    assert work == {0: [0, 499, 7], 1: [1] * 13} and len(waiting) == 1
