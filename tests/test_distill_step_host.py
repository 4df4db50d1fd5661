"""The distillation example's refusals: on the device an index past the sequences' buffer would end
the process's context, so the host counts the room."""
import importlib.util
import os
import sys

import pytest
import torch

_DIR = os.path.join(os.path.dirname(__file__), os.pardir, "examples")
sys.path.insert(0, _DIR)
_SPEC = importlib.util.spec_from_file_location("distill_step", os.path.join(_DIR, "distill_step.py"))
example = importlib.util.module_from_spec(_SPEC)
_SPEC.loader.exec_module(example)


class Student:
    head = torch.zeros(10, 4)                 # on the CPU: a launch would fail in another way


@pytest.mark.parametrize("room", [0, -1])
def test_a_rollout_without_room(room):
    with pytest.raises(ValueError, match="room"):
        example.Rollout(Student(), torch.zeros(2, 3, dtype=torch.int64), room, 4)


def test_a_call_more_than_there_is_room():
    class Graph:
        replays = 0

        def replay(self):
            self.replays += 1

    rollout = example.Rollout.__new__(example.Rollout)
    rollout.left, rollout.graph = 2, Graph()
    rollout.x, rollout.uniforms = torch.zeros(2, 4), torch.zeros(2)
    rollout.lengths = torch.tensor([3, 3])
    rollout.out = (torch.zeros(2, dtype=torch.int64), torch.zeros(2))
    for _ in range(2):
        rollout(torch.ones(2, 4), torch.ones(2))
    with pytest.raises(RuntimeError, match="full"):
        rollout(torch.ones(2, 4), torch.ones(2))
    assert rollout.graph.replays == 2 and rollout.lengths.tolist() == [5, 5]


@pytest.mark.parametrize("steps", [0, -3])
def test_a_run_without_steps(steps):
    with pytest.raises(ValueError, match="steps"):
        example.run(steps=steps, log=None)
    with pytest.raises(ValueError, match="steps"):
        example.main(["--steps", str(steps)])
