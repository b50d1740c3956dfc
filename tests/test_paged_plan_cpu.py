"""Rotary plans as Python objects: what a module that holds one may do with it."""

import copy
import ctypes
import gc
import pickle

import pytest

import certified_quantized_kv_gb300 as kvq


def _fields(p):
    return p.head_dim, p.rotary_dim, p.interleaved, p.magnitude, list(p.step)


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda p: pickle.loads(pickle.dumps(p)),
                                   lambda p: copy.deepcopy({"layers": [p]})["layers"][0]])
def test_copies_of_a_plan_hold_their_own_struct(again):
    plan = kvq.RopePlan(128, rotary_dim=96, layout="interleaved", scaling="yarn", factor=16.0, original_ctx=4096)
    want, at = _fields(plan.plan), plan.address
    other = again(plan)
    assert type(other) is kvq.RopePlan and other.head_dim == 128
    assert other.address == ctypes.addressof(other.plan) != at
    ctypes.memset(plan.address, 0, ctypes.sizeof(plan.plan))      # what the original holds does not matter any more
    assert _fields(other.plan) == want
    assert _fields(kvq.kvq_rope_plan.from_address(other.address)) == want
    del plan
    gc.collect()
    assert _fields(kvq.kvq_rope_plan.from_address(other.address)) == want


def test_an_attribute_of_the_user_goes_along():
    plan = kvq.RopePlan(64)
    plan.name = "layers 0 to 3"
    assert copy.deepcopy(plan).name == plan.name and plan.address == ctypes.addressof(plan.plan)
