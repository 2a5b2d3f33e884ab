"""Refusals of the orthogonalised step that its ranges and its buffers ask for: on the host, before a launch (CPU)."""
import pytest
import torch

from test_blocks_refusals import B, P, muon_hyper, muon_table, status  # noqa: F401


def test_floor(B):  # noqa: F811
    run = lambda floor: status(B, "moe_muon_step_floor", muon_hyper(B), muon_table(B), 1, floor, P, 1 << 30, None, P)  # noqa: E731
    for floor in (-1e-9, float("nan"), float("inf"), 1e39):
        assert run(floor) == 1, floor
    assert status(B, "moe_muon_step_floor", muon_hyper(B), muon_table(B, batch=-1), 1, 1e-7, P, 1 << 30, None, P) == 1
    assert B.moe_muon_step_floor(muon_hyper(B), muon_table(B), 0, 1e-7, None, 0, None, P, stream=0) == 0
