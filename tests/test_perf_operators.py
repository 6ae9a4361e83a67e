"""The plans that perf/operators.py keeps for its decode calls (CPU; the library's
plan calls are stand-ins)."""
import gc
import types

import pytest
import torch

import perf.operators as operators
import split_kv_paged_gqa_gb300 as fd


@pytest.fixture
def world(monkeypatch):
    w = types.SimpleNamespace(device=0, stream=11, alive={}, used=[], n=0)

    def create(device, *geometry):
        w.n += 1
        w.alive[w.n] = (device,) + geometry
        return w.n

    monkeypatch.setattr(fd, "fd_latent_plan_create", create)
    monkeypatch.setattr(fd, "fd_plan_destroy", lambda plan: w.alive.pop(plan))
    monkeypatch.setattr(fd, "fd_set_plan", w.used.append)
    monkeypatch.setattr(fd, "fd_decode_latent", lambda *a, **k: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: w.device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=w.stream))
    monkeypatch.setattr(operators, "own", True)
    return w


def state(B=2, Tq=1, H=4, P=16):
    return dict(op="decode", B=B, Tq=Tq, H=H, P=P, **{k: None for k in ("q", "cache", "table", "lens", "out", "lse")})


def test_one_plan_for_a_geometry_a_device_and_a_stream(world):
    a, b, c, d = (state() for _ in range(4))
    operators.run(a)
    operators.run(b)
    operators.run(a)
    world.stream = 12           # another stream: the calls may overlap, so no shared workspace
    operators.run(c)
    world.device, world.stream = 1, 11
    operators.run(d)
    assert world.used == [1, 1, 1, 2, 3]
    assert [world.alive[k][0] for k in (1, 2, 3)] == [0, 0, 1]
    operators.run(state(H=8))
    assert world.used[-1] == 4


def test_plans_end_with_the_states_that_use_them(world):
    states = [state(B=1 + k) for k in range(20)]
    for s in states:
        operators.run(s)
    assert len(world.alive) == 20
    keep = states[3:5]
    del states, s
    gc.collect()
    assert sorted(world.alive) == [4, 5]
    operators.run(keep[0])
    assert world.used[-1] == 4 and world.n == 20
