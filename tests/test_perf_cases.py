"""The cases of perf/operators.py as calls of the library, on the CPU with the
entry points replaced: which operands the calls get."""
import importlib

import pytest
import torch

import associative_algebra_block_amd as aa

SMALL = [
    {"op": "norm_bwd", "M": 40, "d": 48, "x": "bf16", "dy": "f32", "ds": True},
    {"op": "attn", "B": 2, "H": 4, "Hkv": 2, "D": 16, "page": 16, "lo": 1, "hi": 2000, "q": "f32", "o": "bf16"},
    {"op": "moe", "n": 3, "law": "Qq", "q": 2, "D": 64, "F": 32, "E": 4, "k": 2, "norm": True, "y": "f32", "pos": 1},
]
CALLS = {"norm_bwd": ("aa_layernorm_bwd", 9), "attn": ("aa_attn_decode", 7), "moe": ("aa_moe_ffn_fwd", 12)}


@pytest.fixture
def cases(monkeypatch):
    m = importlib.import_module("perf.operators")
    monkeypatch.setattr(m, "DEV", "cpu")
    monkeypatch.setattr(m, "own", True)
    return m


def needed(c):
    if c["op"] == "norm_bwd":
        return aa.aa_layernorm_bwd_workspace(c["M"], c["d"])
    if c["op"] == "attn":
        return aa.aa_attn_decode_workspace(c["B"], c["H"], c["Hkv"], c["D"], c["page"], -(-c["hi"] // c["page"]))
    up = aa.aa_plan_create(c["law"], c["q"], c["D"], c["F"])
    down = aa.aa_plan_create(c["law"], c["q"], c["F"], c["D"], out_dtype=c["y"])
    return aa.aa_moe_ffn_workspace(up, down, c["E"], c["k"], c["n"])


@pytest.mark.parametrize("case", SMALL, ids=lambda c: c["op"])
def test_states_have_workspaces_of_their_own(cases, monkeypatch, case):
    """Calls that share a workspace must not overlap in time, and two states may
    be run on two streams."""
    got = []
    name, at = CALLS[case["op"]]
    monkeypatch.setattr(aa, "aa_kv_append", lambda *a, **k: None)
    monkeypatch.setattr(aa, name, lambda *a, **k: got.append(a[at]))
    states = [cases.prepare(case, seed) for seed in (1, 2)]
    assert needed(case) > 0
    for s in states + states:
        cases.run(s)
    assert all(w.dtype == torch.uint8 and w.numel() >= needed(case) for w in got)
    at = [w.data_ptr() for w in got]
    assert at[0] != at[1] and at[:2] == at[2:]


@pytest.mark.parametrize("case", SMALL, ids=lambda c: c["op"])
def test_a_state_prepared_for_the_plain_form_serves_both(cases, monkeypatch, case):
    got = []
    name, at = CALLS[case["op"]]
    monkeypatch.setattr(aa, "aa_kv_append", lambda *a, **k: None)
    monkeypatch.setattr(aa, name, lambda *a, **k: got.append(a[at]))
    monkeypatch.setattr(cases, "own", False)
    s = cases.prepare(case, 3)
    cases.run(s)
    assert not got
    monkeypatch.setattr(cases, "own", True)
    cases.run(s)
    cases.run(s)
    assert got[0].numel() >= needed(case) and got[0] is got[1]
